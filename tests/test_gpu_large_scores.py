"""Attention whose finite scores are far beyond what a model has, of either sign: a row's softmax is then its largest score alone (or its ties).

Queries and keys are small whole numbers, so q . k is exact and two different ones are at least 1e6 apart once they are scaled: every other key's
probability is 0, and the output is the mean of the values of the keys that share the largest q . k. A query of zeros, which shares a warp with the others,
sees all keys alike. Tolerance: the output's rounding, the probabilities' (half a step of 16-bit inputs; 2^-20 covers two parts of 11 bits and the
exponential) and the fp32 sums over n keys (n 2^-24), in units of the mean of |v|."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests import test_gpu_prompt as prompt
from tests.test_gpu_kv4 import TYPES, Cache, host, values
from tests.test_gpu_shared_prefix import Shared

pytestmark = pytest.mark.gpu

SCALES = [1.1e6, 1.3e9, 3.3e30]


def whole(shape, dtype, dev, seed, sign=1):
    """Whole numbers that the cache holds exactly: each 16 of a row have a 6."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0])[torch.randint(0, 5, shape, generator=g)]
    x[..., ::16] = 6.0
    return (sign * x).to(TYPES[dtype]).to(dev)


def expect(q, k, v, last):
    """Means of the values of the keys 0 .. last[i] whose q . k is the largest, and of their sizes."""
    s = q @ k.T
    s = np.where(np.arange(k.shape[0])[None, :] > np.asarray(last)[:, None], -np.inf, s)
    p = (s == s.max(1, keepdims=True)).astype(np.float64)
    p /= p.sum(1, keepdims=True)
    return p @ v, p @ np.abs(v)


def close(got, q, k, v, last, dtype, what):
    info = torch.finfo(TYPES[dtype])
    half, least = info.eps / 2, info.smallest_normal * info.eps / 2
    o, size = expect(q, k, v, last)
    assert np.isfinite(got).all(), what
    tol = half * np.abs(o) + least + ((half if dtype != "fp32" else 0.0) + 2.0 ** -20 + k.shape[0] * 2.0 ** -24) * size
    assert (np.abs(got - o) <= tol).all(), (what, float((np.abs(got - o) / tol).max()))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_prompts(cuda_device, dtype, D, sign, scale):
    lens = [1, 300, 2, 131]
    N, off = sum(lens), prompt.packed(lens)
    q, k = whole((N, 4, D), dtype, cuda_device, 1), whole((N, 2, D), dtype, cuda_device, 2, sign)
    q[:, 1] = 0.0
    v = values((N, 2, D), dtype, cuda_device, 3)
    out = host(prompt.attend(q, k, v, off, scale=scale))
    for b in range(len(lens)):
        rows = slice(off[b], off[b + 1])
        for h in range(4):
            close(out[rows, h], host(q[rows, h]), host(k[rows, h // 2]), host(v[rows, h // 2]), np.arange(lens[b]), dtype, (b, h))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [1, 4, 70])  # by single columns, by two tiles of columns, on the tensor cores
def test_cached(cuda_device, T, dtype, D, sign, scale):
    B, H, start = 3, 2, [0, 130, 700]
    c = Cache(cuda_device, B, 1, H, D, 32, 700 + T)
    k = whole((B, 1, 700 + T, H, D), dtype, cuda_device, 4, sign)
    v = whole((B, 1, 700 + T, H, D), dtype, cuda_device, 5)
    c.append(k, v, [0] * B)
    q = whole((B, 1, T, 4, D), dtype, cuda_device, 6)
    q[:, :, :, 1] = 0.0
    out = host(c.attend(q, start, scale=scale))
    assert c.g.gdn_read_device_error() == 0
    for b in range(B):
        for h in range(4):
            kh, vh = (host(x[b, 0, :start[b] + T, h // 2]) for x in (k, v))
            close(out[b, 0, :, h], host(q[b, 0, :, h]), kh, vh, start[b] + np.arange(T), dtype, (b, h))


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp32", 128), ("bf16", 256)])
@pytest.mark.parametrize("B", [2, 40])  # a few rows over the prefix, and 80: on the tensor cores
def test_shared(cuda_device, B, dtype, D, sign, scale):
    H, far, own = 2, 900, 5
    c = Shared(cuda_device, [far], [0, B], B, 1, H, D, 32, own + 1)
    k, v = whole((1 + B, 1, far, H, D), dtype, cuda_device, 7, sign), whole((1 + B, 1, far, H, D), dtype, cuda_device, 8)
    c.fill(k, v, [own + 1] * B, B)
    q = whole((B, 1, 1, 4, D), dtype, cuda_device, 9)
    q[:, :, :, 1] = 0.0
    out = host(c.shared(q, [own] * B, scale=scale))
    assert c.g.gdn_read_device_error() == 0
    for b in (0, B // 2, B - 1):
        for h in range(4):
            kh, vh = (np.concatenate([host(x[0, 0, :, h // 2]), host(x[1 + b, 0, :own + 1, h // 2])]) for x in (k, v))
            close(out[b, 0, :, h], host(q[b, 0, :, h]), kh, vh, [far + own], dtype, (b, h))


def near(got, q, k, v, last, scale, dtype):
    """Rows over the keys that are not far below the others, within the tolerance of an ordinary call (the larger of the two kinds')."""
    info = torch.finfo(TYPES[dtype])
    half, least = info.eps / 2, info.smallest_normal * info.eps / 2
    o, size, qk, s = O.attention_rows(q, k, v, last, scale)
    step, parts = (2.0 ** -21, 2.0 ** -20) if dtype == "fp32" else (half, 0.0)
    rel = 2 * (step + ((q.shape[-1] + 8) * 2.0 ** -24 + parts) * qk + 2.0 ** -22 * (2 + s) + k.shape[0] * 2.0 ** -24)
    assert (np.abs(got - o) <= half * np.abs(o) + least + rel * size).all()


def far_then_near(shape, dtype, dev, seed, far):
    """Queries whose first element meets -49152 in the first `far` keys and 0 in the others."""
    N, Hq, H, D = shape
    q, k, v = (values((N, h, D), dtype, dev, seed + i) for i, h in enumerate((Hq, H, H)))
    q[..., 0] = 40000.0
    k[..., 0] = 0.0
    k[:far] = 0.0
    k[:far, :, 0] = -49152.0
    return q, k, v


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_prompts_rise_out_of_the_far_range(cuda_device, dtype, D):
    """The first tiles' scores are -2e9 times the scale, the others' ordinary: nothing of the former is left in the rows that see one of the latter."""
    n, far = 600, 200
    q, k, v = far_then_near((n, 4, 2, D), dtype, cuda_device, 11, far)
    out = host(prompt.attend(q, k, v, [0, n]))
    for h in range(4):
        qh, kh, vh = host(q[:, h]), host(k[:, h // 2]), host(v[:, h // 2])
        close(out[:far, h], qh[:far], kh[:far], vh[:far], np.arange(far), dtype, h)
        near(out[far:, h], qh[far:], kh[far:], vh[far:], np.arange(n - far), D ** -0.5, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [1, 4, 70])
def test_cached_rows_rise_out_of_the_far_range(cuda_device, T, dtype, D):
    n, far = 600, 200
    q, k, v = far_then_near((n, 4, 2, D), dtype, cuda_device, 14, far)
    c = Cache(cuda_device, 1, 1, 2, D, 32, n)
    c.append(k[None, None].contiguous(), v[None, None].contiguous(), [0])
    q = q[n - T:][None, None].contiguous()
    out = host(c.attend(q, [n - T]))
    for h in range(4):
        kh, vh = O.kv4_read(c.t_cache.cpu().numpy(), c.table, 0, 0, h // 2, n, 32, D)
        near(out[0, 0, :, h], host(q[0, 0, :, h]), kh[far:], vh[far:], n - T + np.arange(T) - far, D ** -0.5, dtype)
