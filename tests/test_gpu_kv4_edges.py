"""Attention over the 4-bit cache, and its calls, at the ends of their ranges. Helpers are those of test_gpu_kv4.py, and so are the
tolerances, with one term more: a probability is kept in fp16 (fp32 calls: hi + lo) relative to 2^9 at the row's largest, and
fp16's smallest step leaves half of it, 2^-25 / 2^9 = 2^-34 of the largest, of each key's."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_kv4 import TYPES, Cache, host, values

pytestmark = pytest.mark.gpu


def check(c, b, q, out, start, dtype, scale):
    """The rows q and out [T][heads][D] of sequence b from position start on, against the restatement; the largest error in tolerances."""
    T, Hq, D = q.shape
    G = Hq // c.H
    cache, got, qh = c.t_cache.cpu().numpy(), host(out), host(q)
    info = torch.finfo(TYPES[dtype])
    last, worst = start + np.arange(T), 0.0
    for h in range(c.H):
        k, v = O.kv4_read(cache, c.table, b, 0, h, start + T, c.page, D)
        seen = (np.arange(start + T) <= last[:, None]) @ np.abs(v)
        for i in range(h * G, h * G + G):
            o, size, qk, s = O.attention_rows(qh[:, i], k, v, last, scale)
            rel = (2.0 ** -22 if dtype == "fp32" else 2.0 ** -12) + 2 * ((D + 8) * 2.0 ** -24 * qk + 2.0 ** -22 * (2 + s)) + 2 * (start + T) * 2.0 ** -24
            tol = info.eps / 2 * np.abs(o) + info.smallest_normal * info.eps / 2 + rel * size + 2.0 ** -34 * seen
            assert np.isfinite(got[:, i]).all()
            worst = max(worst, float((np.abs(got[:, i] - o) / tol).max()))
    assert worst <= 1.0, worst
    return worst


@pytest.mark.parametrize("dtype", list(TYPES))
def test_positions_before_the_table_are_missing(cuda_device, dtype):
    """A negative kv_start: its tokens before position 0 are reported, not written, and read as zeros; the others are where they belong."""
    B, T, H, D, page = 4, 6, 2, 64, 16
    c = Cache(cuda_device, B, 1, H, D, page, 32)
    k, v = (values((B, 1, T, H, D), dtype, cuda_device, s) for s in (1, 2))
    start, n = [-2, 0, -2 ** 31, -7], [6, 6, 6, 0]
    want = c.bytes.copy()
    for b, s in enumerate(start):
        skip = min(-min(s, 0), T)
        kb, vb = host(k)[b:b + 1, :, skip:n[b]], host(v)[b:b + 1, :, skip:n[b]]
        if kb.shape[2] > 0:
            O.kv4_append(kb, vb, want, c.table[b:b + 1], [max(s, 0)], page)
    c.append(k, v, start, n)
    assert c.g.gdn_read_device_error() == 2
    assert np.array_equal(c.t_cache.cpu().numpy(), want)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    c.g.gdn_kv4_read(c.t_cache, c.t_table, c.i32(start), ko, vo, page, seq_len=c.i32(n))
    assert c.g.gdn_read_device_error() == 2
    for x, o in ((k, ko), (v, vo)):
        q = O.kv4_dequantise(*O.kv4_quantise(host(x)))
        assert (host(o)[0, :, :2] == 0).all() and np.array_equal(host(o)[0, :, 2:], q[0, :, 2:])
        assert np.array_equal(host(o)[1], q[1])
        assert (host(o)[2] == 0).all() and (host(o)[3] == 7.0).all()
    # a window of no tokens needs no position
    c.append(k, v, [-1] * B, [0] * B)
    assert c.g.gdn_read_device_error() == 0


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,Hq,H,D", [(1, 4, 1, 128), (4, 8, 2, 64), (3, 5, 1, 256), (12, 16, 2, 128), (70, 4, 2, 64), (9, 4, 2, 256)])
def test_queries_before_the_table_see_nothing(cuda_device, T, Hq, H, D, dtype):
    """Rows before position 0 are zeros, whatever the cache's bytes hold (scales of 255 are NaN); the others see
    the keys up to their own position. Sequences with such rows lie between ones without."""
    start = [40, -T, 3, -1, -T - 5, 0, -2 ** 31, T, 1 - T]
    B, page = len(start), 16
    c = Cache(cuda_device, B, 1, H, D, page, max(40, T) + T)
    c.t_cache.fill_(255)
    total = [max(s + T, 0) for s in start]
    k, v = (values((B, 1, max(total), H, D), dtype, cuda_device, s) for s in (1, 2))
    c.append(k, v, [0] * B, total)
    assert c.g.gdn_read_device_error() == 0
    q = values((B, 1, T, Hq, D), dtype, cuda_device, 3)
    out = c.attend(q, start)
    assert c.g.gdn_read_device_error() == 2
    for b, s in enumerate(start):
        before = min(-min(s, 0), T)
        assert (out[b, :, :before] == 0).all(), b
        if before < T:
            check(c, b, q[b, 0, before:], out[b, 0, before:], max(s, 0), dtype, D ** -0.5)
    assert torch.equal(out, c.attend(q, start)), "two calls differ"
    assert c.g.gdn_read_device_error() == 2


@pytest.mark.parametrize("T,D", [(1, 64), (4, 128), (2, 256), (12, 64), (9, 128), (11, 256)])
def test_small_probabilities_of_fp32_calls(cuda_device, T, D):
    """Rows that are nearly all one key's, whose value is 0 in half of the dimensions, so that the outputs there are sums of
    small probabilities."""
    B, H, keys = 16, 8, 14
    c = Cache(cuda_device, B, 1, H, D, 16, keys)
    k, v = (values((B, 1, keys, H, D), "fp32", cuda_device, s) for s in (51, 52))
    v[:, :, 0, :, ::2] = 0.0
    c.append(k, v, [0] * B)
    first = k[:, :, :1].repeat_interleave(2, 3)
    q = 15 * D ** 0.5 * first / first.square().sum(-1, keepdim=True) + 0.1 * values((B, 1, T, 2 * H, D), "fp32", cuda_device, 53)
    start = keys - T
    out = c.attend(q, [start] * B)
    print("largest error %.3f of the tolerance" % max(check(c, b, q[b, 0], out[b, 0], start, "fp32", D ** -0.5) for b in range(B)))
