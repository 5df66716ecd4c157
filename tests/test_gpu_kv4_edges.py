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


@pytest.mark.parametrize("dtype,G,D,keys", [("fp16", 4, 64, 1 << 20), ("fp16", 8, 128, 1 << 20), ("fp16", 16, 64, 1 << 20), ("fp16", 12, 256, 1 << 19),
                                            ("bf16", 4, 64, 1 << 22), ("fp32", 2, 64, 1 << 19)])
def test_sums_of_very_long_rows(cuda_device, dtype, G, D, keys):
    """Single tokens over up to four million keys, values that are all alike in each dimension, and so many sequences that none is
    split: every output is that value, up to its rounding (or half the type's smallest step), the probabilities' (2^-12,
    fp32: 2^-22), what matrix instructions cut off (1024 steps of up to 2^-23 each before the sums start afresh), and the
    fp32 additions that follow: a sum for every 65536 keys, 4 warps', and a lane's 2048 probabilities in each, of
    either sign (four standard deviations). fp32 calls, which add each step's products with fp32 instructions, have 2 x 1024
    such roundings instead of cuts. All positions lie in four pages, which every sequence shares."""
    H, B, page = 16, 57, 256  # 912 units: as many for each CTA, with 456 CTAs or 304
    c = Cache(cuda_device, 1, 1, H, D, page, 4 * page, spare=0)
    k = values((1, 1, 4 * page, H, D), dtype, cuda_device, 41)
    v = values((D,), dtype, cuda_device, 42)
    c.append(k, v.expand(k.shape).contiguous(), [0])
    c.t_table = c.t_table.view(1, -1).repeat(B, keys // (4 * page)).contiguous()
    q = values((B, 1, 1, H * G, D), dtype, cuda_device, 43)
    out = c.attend(q, [keys - 1] * B).double()
    assert c.g.gdn_read_device_error() == 0
    want = torch.from_numpy(O.kv4_dequantise(*O.kv4_quantise(host(v)))).to(cuda_device)
    info = torch.finfo(TYPES[dtype])
    cuts = 1024 * 2**-23 if dtype != "fp32" else 4 * 2048 ** 0.5 * 2**-24
    tolerance = info.eps / 2 + (2**-22 if dtype == "fp32" else 2**-12) + cuts + (keys / 65536 + 8) * 2**-24 + 4 * 2048 ** 0.5 * 2**-24
    error = (out - want).abs()
    print("largest error %.2e, %.2f of the tolerance" % ((error / want.abs()).nan_to_num().max().item(),
                                                         (error / (tolerance * want.abs() + info.smallest_normal * info.eps / 2)).max().item()))
    assert (error <= tolerance * want.abs() + info.smallest_normal * info.eps / 2).all()


@pytest.mark.parametrize("dtype,D", [("fp32", 64), ("fp16", 128), ("bf16", 256), ("fp32", 256)])
@pytest.mark.parametrize("order", ["rising", "falling", "first missing"])
def test_very_long_rows_whose_maxima_move(cuda_device, order, dtype, D):
    """The sums that start afresh and the partial sums of several CTAs meet other maxima than their own: quarters of a row with
    larger and larger keys, or smaller and smaller, or a row whose first half has no pages. As every page occurs as often as the others, the
    outputs are those of one of each. Tolerances as in test_sums_of_very_long_rows and, for the scores, in check()."""
    H, G, B, page, keys = 8, 4, 67, 256, 1 << 18  # 536 units: some for one CTA, some for two
    c = Cache(cuda_device, 1, 1, H, D, page, 4 * page, spare=0)
    k, v = (values((1, 1, 4 * page, H, D), dtype, cuda_device, s) for s in (44, 45))
    k = (k.float() * torch.tensor([0.2, 0.4, 0.7, 1.0], device=cuda_device).repeat_interleave(page).view(1, 1, -1, 1, 1)).to(TYPES[dtype])
    c.append(k, v, [0])
    pages = torch.from_numpy(c.table[0].copy()).to(cuda_device)
    table = (pages.flip(0) if order == "falling" else pages).repeat_interleave(keys // (4 * page))
    if order == "first missing":
        table[:table.numel() // 2] = -1
    c.t_table = table.repeat(B, 1).contiguous()
    q = values((B, 1, 1, H * G, D), dtype, cuda_device, 46)
    out = c.attend(q, [keys - 1] * B)
    assert c.g.gdn_read_device_error() == (2 if order == "first missing" else 0)
    bytes_, info = c.t_cache.cpu().numpy(), torch.finfo(TYPES[dtype])
    cuts = 1024 * 2**-23 if dtype != "fp32" else 4 * 2048 ** 0.5 * 2**-24
    fixed = (2**-22 if dtype == "fp32" else 2**-12) + cuts + (keys / 65536 + 12) * 2**-24 + 4 * 2048 ** 0.5 * 2**-24
    worst = 0.0
    for h in range(H):
        hk, hv = O.kv4_read(bytes_, c.table, 0, 0, h, 4 * page, page, D)
        if order == "first missing":
            hk, hv = hk[2 * page:], hv[2 * page:]
        for i in range(h * G, h * G + G):
            o, size, qk, s = O.attention_rows(host(q)[:, 0, 0, i], hk, hv, [4 * page] * B, D ** -0.5)
            rel = fixed + 2 * ((D + 8) * 2.0 ** -24 * qk + 2.0 ** -22 * (2 + s))
            tol = info.eps / 2 * np.abs(o) + info.smallest_normal * info.eps / 2 + rel * size + 2.0 ** -34 * np.abs(hv).sum(0)
            worst = max(worst, float((np.abs(host(out)[:, 0, 0, i] - o) / tol).max()))
    print("largest error %.3f of the tolerance" % worst)
    assert worst <= 1.0


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_largest_finite_queries(cuda_device, dtype, T):
    """Rows whose largest element is the type's largest, with a scale that brings the scores back."""
    c = Cache(cuda_device, 1, 1, 2, 64, 16, 70 + T)
    k, v = (values((1, 1, 70 + T, 2, 64), dtype, cuda_device, s) for s in (4, 5))
    c.append(k, v, [0])
    most = torch.finfo(TYPES[dtype]).max
    q = (values((1, 1, T, 4, 64), "fp32", cuda_device, 6) * 1e37).to(TYPES[dtype])
    q[..., 3], q[..., 40] = most, -most
    scale = 2.0 ** -126
    out = c.attend(q, [70], scale=scale)
    check(c, 0, q[0, 0], out[0, 0], 70, dtype, scale)


@pytest.mark.parametrize("T", [1, 20])
def test_the_largest_scale(cuda_device, T):
    """A scale near the largest number and queries as small: neither overflows on its own."""
    c = Cache(cuda_device, 1, 1, 2, 64, 16, 70 + T)
    k, v = (values((1, 1, 70 + T, 2, 64), "fp32", cuda_device, s) for s in (4, 5))
    c.append(k, v, [0])
    scale = float(np.float32(3e38))
    q = values((1, 1, T, 4, 64), "fp32", cuda_device, 6) * 2.0 ** -120
    out = c.attend(q, [70], scale=2.0 ** 118)
    check(c, 0, q[0, 0], out[0, 0], 70, "fp32", 2.0 ** 118)
    q = q * 2.0 ** -10
    out = c.attend(q, [70], scale=scale)
    check(c, 0, q[0, 0], out[0, 0], 70, "fp32", scale)


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


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,H,page", [(1, 16, 2, 16), (8, 1, 1, 64), (4, 4, 2, 32), (9, 2, 2, 16), (3, 6, 2, 128), (1, 9, 1, 32), (1, 32, 2, 16),
                                         (16, 1, 1, 64), (4, 8, 2, 256)])
def test_rows_of_the_single_token_kernel(cuda_device, T, Hq, H, page, D, dtype):
    """Eight, nine and sixteen query rows per kv head: one full column tile, one row of a second, two full ones; as heads, as
    tokens and as both, windows cut short among them."""
    start, n = [0, 300, 31, 64], [T, max(T - 1, 1), T, 1]
    c = Cache(cuda_device, 4, 1, H, D, page, 300 + T)
    k, v = (values((4, 1, 300 + T, H, D), dtype, cuda_device, s) for s in (61, 62))
    c.append(k, v, [0] * 4, [s + m for s, m in zip(start, n)])
    q = values((4, 1, T, Hq, D), dtype, cuda_device, 63)
    out = c.attend(q, start, n)
    assert c.g.gdn_read_device_error() == 0
    for b in range(4):
        assert out[b, :, n[b]:].isnan().all(), "a row past the window was written"
        check(c, b, q[b, 0, :n[b]], out[b, 0, :n[b]], start[b], dtype, D ** -0.5)
