"""gdn_logprobs on the GPU against its fp64 restatement.

Tolerances. An exponential is within 2^-22 and its argument, kept in base 2, within 2^-23 of its size: with
z the distance to the maximum in base 2, a term of the sum is off by (2^-22 + |z| 2^-23) of itself, which averages to at
most 2^-22 (1 + H2 + 1) over the distribution (H2 its entropy in bits). The sum itself is fp32, serial over
at most ceil(V / 512) terms of a thread and then over 9 + 4 levels. So the log of the sum is off by
e = 2^-22 (3 + H2) + (V / 512 + 16) 2^-24, a log probability by that and 2^-22 of its own size, the
entropy by (2 + H) e."""
import numpy as np
import pytest
import torch

from oracle import operators as O

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def run(x, tokens, k):
    import gated_deltanet_linear_step_gb300 as g

    N, dev = x.shape[0], x.device
    lp, ent = (torch.full((N,), 5.0, device=dev) for _ in range(2))
    ids = torch.full((N, k), -7, dtype=torch.int32, device=dev)
    top = torch.full((N, k), 5.0, device=dev)
    g.gdn_logprobs(x, tokens, lp, ent, ids if k else None, top if k else None)
    return lp, ent, ids, top


def check(x, tokens, k, got):
    V = x.shape[1]
    lp, ent, ids, top = O.logprobs(x.float().cpu().numpy(), tokens.cpu().numpy(), k)
    g_lp, g_ent, g_ids, g_top = (t.cpu().numpy() for t in got)
    assert np.array_equal(g_ids, ids)
    e = 2.0 ** -22 * (3 + np.nan_to_num(ent) / np.log(2)) + (V / 512 + 16) * 2.0 ** -24

    def near(a, b, tol):
        assert np.array_equal(np.isnan(a), np.isnan(b))
        ok = (a == b) | np.isnan(b) | (np.abs(a - np.where(np.isinf(b), 0, b)) <= tol)
        assert ok.all(), (a[~ok][:4], b[~ok][:4])

    with np.errstate(invalid="ignore"):
        near(g_lp, lp, e + 2.0 ** -22 * np.abs(lp))
        near(g_ent, ent, (2 + ent) * e)
        near(g_top, top, e[:, None] + 2.0 ** -22 * np.abs(top))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N,V,k", [(1, 1, 1), (2, 5, 5), (3, 33, 0), (1, 4096, 32), (7, 1001, 8), (2, 65537, 20), (1, 200001, 32),
                                   (700, 2049, 3), (64, 32000, 12)])
def test_matches_restatement(cuda_device, N, V, k, dtype):
    g = torch.Generator().manual_seed(N * V)
    x = (torch.randn(N, V, generator=g) * 3).to(TYPES[dtype]).to(cuda_device)
    tokens = torch.randint(0, V, (N,), generator=g, dtype=torch.int32).to(cuda_device)
    got = run(x, tokens, k)
    check(x, tokens, k, got)
    for a, b in zip(got, run(x, tokens, k)):
        assert torch.equal(a, b), "two calls differ"


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_apart_and_unaligned(cuda_device, dtype):
    """Rows of a padded vocabulary, starting at any element: what lies between them is not read."""
    g = torch.Generator().manual_seed(1)
    buf = torch.full((5, 4007), float("nan"))
    buf[:, 3:3 + 4001] = torch.randn(5, 4001, generator=g)
    buf = buf.to(TYPES[dtype]).to(cuda_device)
    x = buf[:, 3:3 + 4001]
    tokens = torch.tensor([0, 4000, 17, 2000, 3999], dtype=torch.int32, device=cuda_device)
    check(x, tokens, 9, run(x, tokens, 9))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_masks_ties_and_rows_without_a_distribution(cuda_device, dtype):
    V, k = 30011, 16
    g = torch.Generator().manual_seed(2)
    x = torch.randn(12, V, generator=g)
    x[0] = float("-inf")
    x[0, 29000] = -3.0                        # one token left
    x[1] = float("-inf")                      # none left
    x[2] = 0.25                               # all equal: the lowest indices
    x[3] = float("-inf")
    x[3, torch.arange(5) * 6000 + 1] = 1.5    # fewer left than asked for, equal
    x[4, 777] = float("nan")
    x[5, 100] = float("inf")
    x[6] = torch.where(torch.rand(V, generator=g) < 0.9, float("-inf"), x[6])
    x[7] = torch.finfo(TYPES[dtype]).min      # a mask of the type's lowest value
    x[7, 5:9] = torch.tensor([2.0, 1.0, 2.0, 0.0])
    x[8] = torch.linspace(-5, 9, V)           # rising: every element is the largest so far
    x[9] = torch.linspace(9, -5, V)
    x[10] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    x[11] = x[11] * 1e4 if dtype != "fp16" else x[11] * 1e3  # one token takes all
    x = x.to(TYPES[dtype]).to(cuda_device)
    tokens = torch.tensor([29000, 3, 2, 1, 5, 100, 9, 6, V - 1, 0, 4, -1], dtype=torch.int32, device=cuda_device)
    got = run(x, tokens, k)
    check(x, tokens, k, got)
    assert got[0][0].item() == 0.0 and got[1][0].item() == 0.0
    assert torch.isnan(got[0][11]) and torch.isnan(got[0][4]) and torch.isnan(got[1][1])
    tokens.fill_(V)
    assert torch.isnan(run(x, tokens, k)[0]).all()


def test_outputs_are_optional_and_graphs_replay(cuda_device):
    import gated_deltanet_linear_step_gb300 as g

    x = torch.randn(9, 5003, device=cuda_device)
    tokens = torch.arange(9, dtype=torch.int32, device=cuda_device)
    want = run(x, tokens, 4)
    ent = torch.empty(9, device=cuda_device)
    g.gdn_logprobs(x, entropy=ent)
    assert torch.equal(ent, want[1])
    lp = torch.empty(9, device=cuda_device)
    g.gdn_logprobs(x, tokens, lp)
    assert torch.equal(lp, want[0])
    graph = torch.cuda.CUDAGraph()
    lp.zero_()
    with torch.cuda.graph(graph):
        g.gdn_logprobs(x, tokens, lp)
    x.mul_(0.5)
    graph.replay()
    assert torch.equal(lp, run(x, tokens, 0)[0]) and not torch.equal(lp, want[0])
