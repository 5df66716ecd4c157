"""The top k of gdn_logprobs where a CTA finds few hundred candidates: as many as a CTA has threads, or as its list holds,
and a few more or less. Ids are compared exactly; output buffers are filled beforehand, so that a place that is not written is seen.

Tolerances of the values as in test_gpu_logprobs.py, the sum being serial over at most ceil(V / 256) terms of a thread and
then over 8 + 4 levels: the log of the sum is off by e = 2^-22 (3 + H2) + (V / 256 + 16) 2^-24, the entropy by (2 + H) e."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_logprobs import TYPES, run

pytestmark = pytest.mark.gpu


def check(x, k):
    """Two calls, alike and equal to the restatement."""
    N, V = x.shape
    tokens = (torch.arange(N, device=x.device) * 7 % V).to(torch.int32)
    got, again = run(x, tokens, k), run(x, tokens, k)
    rows = slice(None) if N <= 16 else slice(0, N, N // 8)
    lp, ent, ids, top = O.logprobs(x[rows].float().cpu().numpy(), tokens[rows].cpu().numpy(), k)
    order = torch.sort(x.cpu().double(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(got[2].cpu().long(), order)
    assert np.array_equal(got[2][rows].cpu().numpy(), ids)
    e = 2.0 ** -22 * (3 + np.nan_to_num(ent) / np.log(2)) + (V / 256 + 16) * 2.0 ** -24
    for a, b, tol in ((got[0], lp, e), (got[1], ent, (2 + np.nan_to_num(ent)) * e), (got[3], top, e[:, None])):
        a = a[rows].cpu().numpy()
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b))
        with np.errstate(invalid="ignore"):
            ok = np.abs(a - b) <= tol + 2.0 ** -22 * np.abs(b)
        assert ok[np.isfinite(b)].all()
    for a, b in zip(got, again):
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num()), "two calls differ"


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [255, 256, 257, 300, 384, 511, 512, 513])
def test_equal_rows(cuda_device, V, dtype):
    x = torch.full((3, V), 0.25)
    x[1] = float("-inf")
    x[2] = -7.5
    for k in (1, 16, 32):
        check(x.to(TYPES[dtype]).to(cuda_device), k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V", [257, 300, 384, 511, 512, 513, 30011])
def test_masks_that_leave_few_tokens(cuda_device, V, dtype):
    """-inf and the type's lowest value as masks that leave 0, 1, k - 1, k and 60 tokens."""
    k = 16
    g = torch.Generator().manual_seed(V)
    rows = []
    for mask in (float("-inf"), torch.finfo(TYPES[dtype]).min):
        for left in (0, 1, k - 1, k, 60):
            x = torch.full((V,), mask)
            x[torch.randperm(V, generator=g)[:left]] = torch.randn(left, generator=g) * 3
            rows.append(x)
    check(torch.stack(rows).to(TYPES[dtype]).to(cuda_device), k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [1, 1024])
@pytest.mark.parametrize("ties", [255, 300, 400, 500, 512, 513])
def test_ties_at_the_top(cuda_device, ties, N, dtype):
    """Values cut off at a cap, from one CTA per row to a cluster of sixteen."""
    V = 32000
    g = torch.Generator().manual_seed(ties)
    x = torch.randn(V, generator=g).clamp(max=2.0)
    x[torch.randperm(V, generator=g)[:ties]] = 6.0
    x = x.to(TYPES[dtype]).to(cuda_device)
    check(torch.stack([x.roll(37 * i) for i in range(N)]), 8)


def test_close_values(cuda_device):
    """fp32 logits that lie so close that hundreds share the upper 16 bits of the threshold."""
    g = torch.Generator().manual_seed(5)
    check((200 + torch.randn(1024, 16384, generator=g)).to(cuda_device), 32)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_unaligned_rows(cuda_device, dtype):
    g = torch.Generator().manual_seed(6)
    buf = torch.full((6, 420), float("nan"))
    buf[:, 3:403] = torch.randint(0, 2, (6, 400), generator=g).float()
    buf[0, 3:403] = float("-inf")
    buf[0, 300:305] = torch.tensor([1.0, 3.0, 2.0, 3.0, 1.0])
    check(buf.to(TYPES[dtype]).to(cuda_device)[:, 3:403], 32)
