"""Attention over the 4-bit cache, and its calls, at the ends of their ranges. Helpers and tolerances are those of
test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_kv4 import TYPES, Cache, check_attention, host, values

pytestmark = pytest.mark.gpu


def one_sequence(c, b):
    """Sequence b of the cache alone."""
    one = Cache.__new__(Cache)
    one.__dict__.update(c.__dict__)
    one.table, one.B = c.table[b:b + 1], 1
    return one


@pytest.mark.parametrize("T,D", [(1, 64), (4, 128), (2, 256), (12, 64), (9, 128), (11, 256)])
def test_small_probabilities_of_fp32_calls(cuda_device, T, D):
    """Rows that are nearly all one key's, whose value is 0 in half of the dimensions, so that the outputs there are sums of
    small probabilities. To the tolerance of test_gpu_kv4.py comes what fp16's smallest step leaves of a probability that
    is kept as hi + lo relative to 2^9 at the largest: half of it, 2^-25 / 2^9 = 2^-34 of the largest."""
    B, H, keys = 16, 8, 14
    c = Cache(cuda_device, B, 1, H, D, 16, keys)
    k, v = (values((B, 1, keys, H, D), "fp32", cuda_device, s) for s in (51, 52))
    v[:, :, 0, :, ::2] = 0.0
    c.append(k, v, [0] * B)
    first = k[:, :, :1].repeat_interleave(2, 3)
    q = 15 * D ** 0.5 * first / first.square().sum(-1, keepdim=True) + 0.1 * values((B, 1, T, 2 * H, D), "fp32", cuda_device, 53)
    start = keys - T
    out = c.attend(q, [start] * B)
    cache, worst = c.t_cache.cpu().numpy(), 0.0
    for b in range(B):
        for h in range(H):
            hk, hv = O.kv4_read(cache, c.table, b, 0, h, keys, 16, D)
            for i in (2 * h, 2 * h + 1):
                last = start + np.arange(T)
                o, size, qk, s = O.attention_rows(host(q)[b, 0, :, i], hk, hv, last, D ** -0.5)
                rel = 2.0 ** -22 + 2 * ((D + 8) * 2.0 ** -24 * qk + 2.0 ** -22 * (2 + s)) + 2 * keys * 2.0 ** -24
                seen = np.arange(keys) <= last[:, None]
                tol = 2.0 ** -24 * np.abs(o) + 2.0 ** -150 + rel * size + 2.0 ** -34 * (seen @ np.abs(hv))
                worst = max(worst, float((np.abs(host(out)[b, 0, :, i] - o) / tol).max()))
    print("largest error %.3f of the tolerance" % worst)
    assert worst <= 1.0
