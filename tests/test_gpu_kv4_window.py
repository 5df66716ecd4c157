"""Attention over the 4-bit cache for windows with many query rows per kv head, which run on the tensor cores,
against the fp64 restatement; helpers, cache and tolerances are those of test_gpu_kv4.py."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_kv4 import TYPES, Cache, check_attention, host, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,T,Hq,H,D,page,start,n", [
    (1, 1, 17, 1, 1, 64, 16, [0], None),                     # one row more than the other kernel takes, no cache before it
    (1, 1, 1, 17, 1, 128, 16, [0], None),                    # seventeen heads and a single key
    (1, 1, 64, 2, 1, 128, 64, [0], None),                    # exactly 128 rows, one whole tile
    (1, 1, 129, 1, 1, 128, 64, [63], None),                  # 129 rows: a second block with one of them
    (2, 1, 43, 6, 2, 64, 128, [191, 1], None),               # 129 rows of six heads: rows of a token in two blocks
    (1, 1, 300, 4, 2, 128, 32, [100], None),                 # units of 256 rows, the last of 88
    (3, 2, 9, 20, 4, 128, 16, [250, 0, 33], [9, 0, 2]),      # a ragged window, an empty one, short pages
    (2, 1, 40, 8, 2, 256, 16, [70, 0], [40, 33]),            # D = 256: two blocks
    (1, 1, 5, 16, 4, 128, 256, [6000], None),                # one long sequence over many CTAs
    (1, 2, 20, 1, 1, 64, 256, [3000], None),                 # the same at D = 64
    (20, 1, 3, 12, 2, 128, 64, [7 * i * i for i in range(20)], [1 + i % 3 for i in range(20)]),  # short and long units in a CTA
])
def test_windows_match_restatement(cuda_device, B, L, T, Hq, H, D, page, start, n, dtype):
    c = Cache(cuda_device, B, L, H, D, page, max(start) + T, seed=T)
    total = [s + (T if n is None else n[b]) for b, s in enumerate(start)]
    k, v = (values((B, L, max(total), H, D), dtype, cuda_device, s) for s in (1, 2))
    c.append(k, v, [0] * B, total)
    q = values((B, L, T, Hq, D), dtype, cuda_device, 3)
    out = c.attend(q, start, n)
    assert c.g.gdn_read_device_error() == 0
    print(check_attention(c, q, out, start, n, dtype))
    again = c.attend(q, start, n)
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(again)), "two calls differ"


@pytest.mark.parametrize("dtype,D,T", [("bf16", 128, 12), ("fp32", 128, 70), ("fp16", 64, 70), ("bf16", 256, 12)])
def test_what_is_masked_does_not_matter(cuda_device, dtype, D, T):
    """Bytes of 255 past each sequence's end, a huge last token, NaN and infinite queries: rows that do not see
    them keep their bits."""
    c = Cache(cuda_device, 2, 1, 1, D, 16, 100 + T)
    total = [30 + T, 77 + T]
    k, v = (values((2, 1, 77 + T, 1, D), dtype, cuda_device, s) for s in (7, 8))
    start = [30, 77]
    q = values((2, 1, T, 4, D), dtype, cuda_device, 9)
    c.append(k, v, [0, 0], total)
    want = c.attend(q, start)
    check_attention(c, q, want, start, None, dtype)
    c.t_cache = torch.full_like(c.t_cache, 255)
    c.append(k, v, [0, 0], total)
    assert torch.equal(c.attend(q, start), want)
    big = k[:, :, :1].clone()
    big[..., ::3], big[..., 1::3], big[..., 2::3] = float("nan"), float("inf"), torch.finfo(TYPES[dtype]).min
    c.append(big, big, [s + T - 1 for s in start])
    got = c.attend(q, start)
    assert torch.equal(got[:, :, :T - 1], want[:, :, :T - 1]) and torch.isfinite(got).all()
    bad = q.clone()
    bad[0, 0, 1, 2, 5], bad[1, 0, T - 1, 3, 0] = float("nan"), float("inf")
    got2 = c.attend(bad, start)
    same = torch.ones(2, 1, T, 4, dtype=torch.bool, device=cuda_device)
    same[0, 0, 1, 2] = same[1, 0, T - 1, 3] = False
    assert torch.equal(got2[same], got[same]) and torch.isnan(got2[0, 0, 1, 2]).all()


@pytest.mark.parametrize("gain", [1e-20, 3e6])
def test_queries_of_any_size(cuda_device, gain):
    c = Cache(cuda_device, 1, 1, 2, 128, 16, 120)
    k, v = (values((1, 1, 120, 2, 128), "fp32", cuda_device, s) for s in (4, 5))
    c.append(k, v, [0])
    q = values((1, 1, 20, 4, 128), "fp32", cuda_device, 6) * gain
    out = c.attend(q, [100], scale=128 ** -0.5 / gain)
    check_attention(c, q, out, [100], None, "fp32", scale=128 ** -0.5 / gain)


@pytest.mark.parametrize("page,D", [(16, 128), (32, 64), (64, 256), (128, 128)])
def test_missing_pages_take_no_part(cuda_device, page, D):
    tokens = 4 * page
    c = Cache(cuda_device, 1, 1, 1, D, page, tokens)
    k, v = (values((1, 1, tokens, 1, D), "fp32", cuda_device, s) for s in (10, 11))
    c.append(k, v, [0])
    q = values((1, 1, 10, 2, D), "fp32", cuda_device, 12)
    table = c.table.copy()
    table[0, 1], table[0, 2] = -1, c.t_cache.shape[1]
    c.t_table = torch.from_numpy(table).to(cuda_device)
    start = tokens - 10
    out = c.attend(q, [start])
    assert c.g.gdn_read_device_error() == 2
    hk, hv = O.kv4_read(c.t_cache.cpu().numpy(), c.table, 0, 0, 0, tokens, page, D)
    keep = np.r_[0:page, 3 * page:tokens]
    for h in range(2):
        o, size, _, _ = O.attention_rows(host(q)[0, 0, :, h], hk[keep], hv[keep], len(keep) - 10 + np.arange(10), D ** -0.5)
        assert np.abs(host(out)[0, 0, :, h] - o).max() <= 1e-4 * size.max()
    # a window past the table's end, and no page at all
    assert torch.isfinite(c.attend(q, [tokens - 3])).all() and c.g.gdn_read_device_error() == 2
    c.t_table = torch.full_like(c.t_table, -1)
    assert (c.attend(q, [start]) == 0).all() and c.g.gdn_read_device_error() == 2


def test_graph_replays_as_lengths_advance(cuda_device):
    import gated_deltanet_linear_step_gb300 as g

    B, T, H, Hq, D, page = 3, 6, 2, 8, 128, 32
    a, d = (Cache(cuda_device, B, 1, H, D, page, 240) for _ in range(2))
    k, v = (values((B, 1, T, H, D), "bf16", cuda_device, s) for s in (16, 17))
    q = values((B, 1, T, Hq, D), "bf16", cuda_device, 18)
    pre_k, pre_v = (values((B, 1, 200, H, D), "bf16", cuda_device, s) for s in (19, 20))
    start0 = [120, 0, 199]
    for c in (a, d):
        c.append(pre_k, pre_v, [0] * B, start0)
    ws = torch.empty(g.gdn_kv4_attention_workspace_size(B, 1, T, Hq, H, D), dtype=torch.uint8, device=cuda_device)
    out = torch.empty_like(q)
    start = a.i32(start0)

    def step():
        g.gdn_kv4_append(k, v, a.t_cache, a.t_table, start, page)
        g.gdn_kv4_attention(q, a.t_cache, a.t_table, start, out, ws, page, H)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        start += i  # the first replay repeats the call above
        graph.replay()
        now = start.tolist()
        d.append(k, v, now)
        assert torch.equal(out, d.attend(q, now)), i
    assert g.gdn_read_device_error() == 0


@pytest.mark.parametrize("T,D", [(20, 64), (150, 64), (20, 128), (8, 64), (8, 128)])
def test_long_fp32_sums_are_not_cut_off(cuda_device, T, D):
    """Values that are all alike: every output is that value (one, as the cache holds it), up to what the fp32 sums over 16000 keys lose. Matrix
    instructions cut a sum off, by up to 2^-23 of it each: 64 of them before the sums start afresh (512 keys, 16 at
    a time, probabilities in two parts). Then 32 such sums, rounded; and as many roundings in each partial sum of
    the probabilities as it has tiles, 250, of either sign (four standard deviations). Enough heads that no
    sequence is split."""
    heads, keys = 320, 16000
    c = Cache(cuda_device, 1, 1, heads, D, 64, keys)
    k = values((1, 1, keys, 1, D), "bf16", cuda_device, 21).expand(1, 1, keys, heads, D).contiguous()
    c.append(k, torch.ones_like(k), [0])
    q = values((1, 1, T, heads, D), "fp32", cuda_device, 22)
    out = c.attend(q, [keys - T]).double()
    one = O.kv4_dequantise(*O.kv4_quantise(np.ones(D)))[0]
    error = (out / float(one) - 1).abs().max().item()
    print("largest error %.2e" % error)
    assert error <= 64 * 2**-23 + 32 * 2**-24 + 4 * (32 + 250) ** 0.5 * 2**-24 + 2**-22


@pytest.mark.parametrize("dtype,T,D", [("fp16", 20, 64), ("bf16", 150, 64), ("fp16", 150, 128)])
def test_long_16_bit_sums(cuda_device, dtype, T, D):
    """The same for 16-bit calls over 40000 keys, with another value in each dimension: the output's rounding (or half
    the type's smallest step), the probabilities' (2^-12), 1024 steps before the sums start afresh, and what adds up
    two more such sums and 625 tiles' probabilities."""
    heads, keys = 320, 40000
    c = Cache(cuda_device, 1, 1, heads, D, 64, keys)
    k = values((1, 1, keys, 1, D), dtype, cuda_device, 23).expand(1, 1, keys, heads, D).contiguous()
    v = values((D,), dtype, cuda_device, 24)
    c.append(k, v.expand(k.shape).contiguous(), [0])
    q = values((1, 1, T, heads, D), dtype, cuda_device, 25)
    out = c.attend(q, [keys - T]).double()
    want = torch.from_numpy(O.kv4_dequantise(*O.kv4_quantise(host(v)))).to(cuda_device)
    info = torch.finfo(TYPES[dtype])
    tolerance = info.eps / 2 + 2**-12 + 1024 * 2**-23 + 3 * 2**-24 + 4 * 625 ** 0.5 * 2**-24
    error = (out - want).abs()
    print("largest error %.2e" % (error / want.abs()).nan_to_num().max().item())
    assert (error <= tolerance * want.abs() + info.smallest_normal * info.eps / 2).all()


@pytest.mark.parametrize("dtype,T,D", [("fp32", 20, 64), ("fp32", 33, 128), ("fp32", 17, 256), ("bf16", 150, 64)])
def test_maxima_that_rise_over_long_rows(cuda_device, dtype, T, D):
    """Keys that grow with their position, so that the maximum rises after the sums were started afresh, and enough
    heads that a sequence is not split; against fp64 over the values that the cache gives back. Tolerances as in
    test_gpu_kv4.py, from each row's own largest score and sum |q k|; and, as these rows are nearly all one key's, half
    of fp16's smallest step for each probability relative to 2^-8 of the largest: 2^-33."""
    heads, keys = 310, 1700
    c = Cache(cuda_device, 1, 1, heads, D, 32, keys)
    ramp = (0.1 + torch.arange(keys, device=cuda_device) / 800).view(1, 1, keys, 1, 1)
    k = (values((1, 1, keys, heads, D), "fp32", cuda_device, 31) * ramp).to(TYPES[dtype])
    v = values((1, 1, keys, heads, D), dtype, cuda_device, 32)
    c.append(k, v, [0])
    q = values((1, 1, T, heads, D), dtype, cuda_device, 33)
    out = c.attend(q, [keys - T])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    c.g.gdn_kv4_read(c.t_cache, c.t_table, c.i32([0]), ko, vo, c.page)
    q, k, v, out = (x[0, 0].transpose(0, 1).double() for x in (q, ko, vo, out))  # [head][token][dim]
    scale = D ** -0.5
    seen = torch.arange(keys, device=cuda_device) <= keys - T + torch.arange(T, device=cuda_device).view(T, 1)
    s = (scale * q @ k.transpose(1, 2)).masked_fill(~seen, -float("inf"))
    p = s.softmax(-1)
    want, amount = p @ v, p @ v.abs()
    products = (scale * q.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0).amax(-1, keepdim=True)
    largest = s.masked_fill(~seen, 0).abs().amax(-1, keepdim=True)
    rounding = 2**-22 if dtype == "fp32" else 2**-12
    score = (D + 8) * 2**-24 * products + 2**-22 * (2 + largest)
    tolerance = torch.finfo(TYPES[dtype]).eps / 2 * want.abs() + amount * (rounding + 2 * score + 2 * keys * 2**-24)
    tolerance = tolerance + 2**-33 * (seen.double() @ v.abs())
    ratio = ((out - want).abs() / tolerance).max().item()
    print("largest error %.3f of the tolerance" % ratio)
    assert ratio <= 1
