"""The 4-bit key/value cache and attention over it on the GPU against their fp64 restatement.

Tolerances. The cache's bytes and values are exact. An attention output may be off by its own rounding,
eps(type)/2 of the value or half the type's smallest step, and, in units of A = sum_j p_j |v_j| of its dimension (what a relative error of every
probability moves it by), by the probability's rounding (2^-12 for 16-bit calls; hi + lo leave 2^-22 for fp32
ones), the fp32 evaluation of a score and its exponential (a sum of D products, at most (D + 8) 2^-24 of
scale sum |q k|, and 2^-22 (2 + |s|) for the argument and the approximation, twice: numerator and sum), and
the fp32 sum over n keys (n 2^-24, twice)."""
import numpy as np
import pytest
import torch

from oracle import operators as O

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Cache:
    """A cache filled with random bytes, shuffled pages, and the calls on it."""

    def __init__(self, dev, B, L, H, D, page, tokens, seed=0, spare=3):
        import gated_deltanet_linear_step_gb300 as g

        self.g, self.dev, self.B, self.L, self.H, self.D, self.page = g, dev, B, L, H, D, page
        maxp = (tokens + page - 1) // page
        n = B * maxp + spare
        rng = np.random.default_rng(seed)
        self.table = rng.permutation(n)[:B * maxp].reshape(B, maxp).astype(np.int32)
        self.bytes = rng.integers(0, 256, (L, n, g.gdn_kv4_page_bytes(H, D, page)), dtype=np.uint8)
        self.t_cache = torch.from_numpy(self.bytes.copy()).to(dev)
        self.t_table = torch.from_numpy(self.table).to(dev)

    def i32(self, v):
        return None if v is None else torch.tensor(v, dtype=torch.int32, device=self.dev)

    def append(self, k, v, start, n=None):
        self.g.gdn_kv4_append(k, v, self.t_cache, self.t_table, self.i32(start), self.page, seq_len=self.i32(n))

    def attend(self, q, start, n=None, out=None, scale=None):
        B, L, T, Hq, D = q.shape
        out = torch.full_like(q, float("nan")) if out is None else out
        ws = torch.full((self.g.gdn_kv4_attention_workspace_size(B, L, T, Hq, self.H, D),), 255, dtype=torch.uint8, device=self.dev)
        self.g.gdn_kv4_attention(q, self.t_cache, self.t_table, self.i32(start), out, ws, self.page, self.H, scale=scale,
                                 seq_len=self.i32(n))
        return out


def values(shape, dtype, dev, seed, spread=0.7):
    g = torch.Generator(device="cpu").manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(spread * torch.randn(shape[-1:], generator=g))
    return x.to(TYPES[dtype]).to(dev)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,T,H,page,start,n", [
    (1, 1, 1, 1, 16, [0], None),               # the first token of a cache
    (3, 2, 1, 2, 32, [31, 32, 5], None),         # single tokens at page borders
    (2, 1, 37, 3, 16, [13, 0], [37, 20]),        # windows over several pages, one cut short
    (3, 1, 8, 1, 64, [60, 7, 0], [0, 9, -2]),    # an empty window, a length past T, a negative one
])
def test_append_and_read_are_exact(cuda_device, B, L, T, H, page, start, n, dtype, D):
    c = Cache(cuda_device, B, L, H, D, page, max(start) + T)
    k, v = (values((B, L, T, H, D), dtype, cuda_device, s) * 10.0 ** (s - 2) for s in (1, 3))
    want = c.bytes.copy()
    O.kv4_append(host(k), host(v), want, c.table, start, page, n)
    c.append(k, v, start, n)
    assert np.array_equal(c.t_cache.cpu().numpy(), want)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    c.g.gdn_kv4_read(c.t_cache, c.t_table, c.i32(start), ko, vo, page, seq_len=c.i32(n))
    for x, o in ((k, ko), (v, vo)):
        q = O.kv4_dequantise(*O.kv4_quantise(host(x)))
        for b in range(B):
            m = T if n is None else min(max(n[b], 0), T)
            assert np.array_equal(host(o)[b, :, :m], q[b, :, :m])
            assert (host(o)[b, :, m:] == 7.0).all(), "a row past the window was written"
    assert c.g.gdn_read_device_error() == 0


def test_quantiser_borders(cuda_device):
    """Values next to every tie, far scales, infinities and NaN, bit for bit."""
    s = O.scale_values()[[1, 7, 8, 60, 113, 120, 200, 226]]
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for v in s:
        x = np.float32(mids * v)
        for y in (x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))):
            rows.append(np.concatenate([[6 * v], y, -y, [0.0]]))
    g = O.scale_values()[:-1]
    tie = np.float32((g + O.scale_values()[1:]) / 2 * 6)  # amax / 6 half way between two scales
    for y in (tie, np.nextafter(tie, np.float32(0)), np.nextafter(tie, np.float32(1e9))):
        rows.extend(np.concatenate([[a], np.linspace(-a, a, 15)]) for a in y)
    rows += [np.full(16, np.nan), np.array([np.inf, -np.inf] + [1.0] * 14), np.array([np.nan, 3.0, -1.0] + [0.5] * 13),
             np.array([3e38, -1e-38] + [0.0] * 14), np.full(16, -0.0), np.full(16, 1e-40), np.full(16, 65504.0)]
    x = np.float32(np.stack(rows))
    x = np.concatenate([x, np.zeros((-len(x) % 4, 16), np.float32)]).reshape(-1, 64)
    k = torch.from_numpy(x).to(cuda_device).view(1, 1, -1, 1, 64)
    c = Cache(cuda_device, 1, 1, 1, 64, 16, k.shape[2])
    want = c.bytes.copy()
    O.kv4_append(x.reshape(k.shape).astype(np.float64), x.reshape(k.shape).astype(np.float64), want, c.table, [0], 16)
    c.append(k, k, [0])
    assert np.array_equal(c.t_cache.cpu().numpy(), want)


def check_attention(c, q, out, start, n, dtype, scale=None, rows=None):
    """Compares every row (or the listed (b, l, h) ones) with the restatement."""
    B, L, T, Hq, D = q.shape
    G = Hq // c.H
    scale = D ** -0.5 if scale is None else scale
    cache = c.t_cache.cpu().numpy()
    got, qh = host(out), host(q)
    info = torch.finfo(TYPES[dtype])
    half, least = info.eps / 2, info.smallest_normal * info.eps / 2
    p_step = 2.0 ** -22 if dtype == "fp32" else 2.0 ** -12
    worst = 0.0
    for b in range(B):
        m = T if n is None else min(max(n[b], 0), T)
        assert np.isnan(got[b, :, m:]).all(), "a row past the window was written"
        if m == 0:
            continue
        for l in range(L):
            for h in range(c.H):
                if rows is not None and (b, l, h) not in rows:
                    continue
                k, v = O.kv4_read(cache, c.table, b, l, h, start[b] + m, c.page, D)
                for i in range(h * G, h * G + G):
                    o, size, qk, s = O.attention_rows(qh[b, l, :m, i], k, v, start[b] + np.arange(m), scale)
                    rel = p_step + 2 * ((D + 8) * 2.0 ** -24 * qk + 2.0 ** -22 * (2 + s)) + 2 * (start[b] + m) * 2.0 ** -24
                    tol = half * np.abs(o) + least + rel * size
                    err = np.abs(got[b, l, :m, i] - o)
                    assert np.isfinite(got[b, l, :m, i]).all(), (b, l, i)
                    worst = max(worst, float((err / tol).max()))
    assert worst <= 1.0, worst
    return worst


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,T,Hq,H,D,page,start,n", [
    (1, 1, 1, 1, 1, 64, 16, [0], None),                      # one key
    (1, 1, 1, 4, 4, 128, 16, [1], None),                     # two keys, one query head per kv head
    (2, 1, 1, 5, 1, 128, 32, [30, 31], None),                # up to the page border and past it
    (3, 2, 1, 6, 2, 64, 16, [63, 64, 200], None),            # tiles of four pages, ragged
    (2, 1, 1, 16, 2, 256, 64, [15, 400], None),              # eight query heads per kv head
    (2, 1, 1, 32, 2, 128, 128, [700, 3], None),              # sixteen: two column tiles
    (1, 1, 1, 33, 1, 64, 16, [77], None),                    # thirty-three: two column blocks
    (4, 1, 1, 4, 1, 128, 64, [1, 300, 0, 129], [1, 0, 1, 1]),  # a sequence with no token in the middle
    (3, 2, 8, 10, 2, 128, 32, [250, 0, 33], [8, 3, 5]),      # a ragged verify window of five heads per kv head
    (2, 1, 3, 12, 3, 256, 16, [40, 128], [3, 2]),            # twelve columns at D = 256
    (1, 1, 19, 7, 1, 256, 32, [100], None),                  # several column blocks at D = 256
    (2, 1, 33, 8, 2, 64, 64, [0, 95], [33, 20]),             # a prompt from position 0
    (1, 1, 130, 4, 1, 128, 64, [70], None),                  # a longer prompt
    (1, 1, 1, 4, 1, 128, 64, [5000], None),                  # one sequence over many CTAs
    (40, 1, 1, 2, 1, 64, 16, list(range(0, 400, 10)), None),  # more sequences than a warp has lanes
])
def test_attention_matches_restatement(cuda_device, B, L, T, Hq, H, D, page, start, n, dtype):
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


@pytest.mark.parametrize("dtype,gain", [("fp32", 1e-20), ("fp32", 3e6), ("bf16", 1e-6), ("fp16", 30.0)])
def test_attention_takes_queries_of_any_size(cuda_device, dtype, gain):
    """Queries far outside fp16's range, with a scale that brings the scores back."""
    c = Cache(cuda_device, 2, 1, 2, 128, 16, 90)
    k, v = (values((2, 1, 90, 2, 128), dtype, cuda_device, s) for s in (4, 5))
    c.append(k, v, [0, 0], [90, 41])
    q = (values((2, 1, 1, 4, 128), "fp32", cuda_device, 6) * gain).to(TYPES[dtype])
    scale = 128 ** -0.5 / gain
    out = c.attend(q, [89, 40], scale=scale)
    check_attention(c, q, out, [89, 40], None, dtype, scale=scale)


def test_what_is_masked_does_not_matter(cuda_device):
    """Bytes of 255 (NaN scales) past each row's end, rejected tokens of an earlier window, NaN and
    infinite queries of other rows: the rows that do not see them keep their bits."""
    c = Cache(cuda_device, 2, 1, 1, 128, 16, 100)
    k, v = (values((2, 1, 60, 1, 128), "bf16", cuda_device, s) for s in (7, 8))
    c.append(k, v, [0, 0], [41, 60])
    q = values((2, 1, 3, 4, 128), "bf16", cuda_device, 9)
    want = c.attend(q, [38, 57])
    check_attention(c, q, want, [38, 57], None, "bf16")
    # everything past each sequence's end
    cache = torch.full_like(c.t_cache, 255)
    kept = Cache.__new__(Cache)
    kept.__dict__.update(c.__dict__)
    kept.t_cache = cache
    kept.append(k, v, [0, 0], [41, 60])
    assert torch.equal(kept.attend(q, [38, 57]), want)
    # a later token that only the last row sees holds huge values; a NaN is stored as 0
    big = k[:, :, :1].clone()
    big[..., ::3], big[..., 1::3], big[..., 2::3] = float("nan"), float("inf"), -3e38
    c.append(big, big, [40, 59])
    got = c.attend(q, [38, 57])
    assert torch.equal(got[:, :, :2], want[:, :, :2]) and torch.isfinite(got).all()
    # a NaN query spoils its own row only
    bad = q.clone()
    bad[0, 0, 1, 2, 5] = float("nan")
    bad[1, 0, 0, 0, 0] = float("inf")
    got2 = c.attend(bad, [38, 57])
    same = torch.ones(2, 1, 3, 4, dtype=torch.bool, device=cuda_device)
    same[0, 0, 1, 2] = same[1, 0, 0, 0] = False
    assert torch.equal(got2[same], got[same]) and torch.isnan(got2[0, 0, 1, 2]).all()


def test_missing_pages_are_reported_and_take_no_part(cuda_device):
    """Entries outside [0, n_pages) and positions past the table: the error word's bit 1; such tokens are not
    written, read as zeros, and are left out of the attention."""
    c = Cache(cuda_device, 1, 1, 1, 128, 16, 64)
    k, v = (values((1, 1, 64, 1, 128), "fp32", cuda_device, s) for s in (10, 11))
    c.append(k, v, [0])
    q = values((1, 1, 1, 2, 128), "fp32", cuda_device, 12)
    before = c.t_cache.clone()
    for bad in (-1, c.t_cache.shape[1], 1 << 30):
        table = c.table.copy()
        table[0, 1] = bad
        whole, c.t_table = c.t_table, torch.from_numpy(table).to(cuda_device)
        out = c.attend(q, [60])
        assert c.g.gdn_read_device_error() == 2
        ko, vo = torch.full_like(k, 7.0), torch.full_like(k, 7.0)
        c.g.gdn_kv4_read(c.t_cache, c.t_table, c.i32([0]), ko, vo, 16)
        assert c.g.gdn_read_device_error() == 2
        assert (ko[0, 0, 16:32] == 0).all() and (vo[0, 0, 16:32] == 0).all() and (ko[0, 0, 32:] != 7.0).all()
        c.append(k[:, :, :3], v[:, :, :3], [20])
        assert c.g.gdn_read_device_error() == 2
        c.t_table = whole
        assert torch.equal(c.t_cache, before)
        hk, hv = O.kv4_read(c.t_cache.cpu().numpy(), c.table, 0, 0, 0, 61, 16, 128)
        keep = np.r_[0:16, 32:61]
        o, size, _, _ = O.attention_rows(host(q)[0, 0, 0], hk[keep], hv[keep], [44, 44], 128 ** -0.5)
        assert np.abs(host(out)[0, 0, 0] - o).max() <= 1e-4 * size.max()
    # a window that runs past the table
    c.append(k[:, :, :5], v[:, :, :5], [62])
    assert c.g.gdn_read_device_error() == 2
    out = c.attend(q, [1 << 29])
    assert c.g.gdn_read_device_error() == 2 and torch.isfinite(out).all()
    # no page at all: zeros
    c.t_table = torch.full_like(c.t_table, -1)
    assert (c.attend(q, [60]) == 0).all()
    assert c.g.gdn_read_device_error() == 2


def test_pages_beyond_32_bit_offsets(cuda_device):
    """A cache of over 4 GiB whose used pages lie at its end."""
    import gated_deltanet_linear_step_gb300 as g

    H, D, page = 8, 256, 256
    c = Cache(cuda_device, 1, 1, H, D, 16, 16)
    pb = g.gdn_kv4_page_bytes(H, D, page)
    n = (9 << 29) // pb  # 4.5 GiB
    c.page, c.table = page, np.array([[n - 1, n - 3]], dtype=np.int32)
    c.t_table = torch.from_numpy(c.table).to(cuda_device)
    c.t_cache = torch.empty((1, n, pb), dtype=torch.uint8, device=cuda_device)
    k, v = (values((1, 1, 300, H, D), "bf16", cuda_device, s) for s in (13, 14))
    c.append(k, v, [0])
    q = values((1, 1, 1, H, D), "bf16", cuda_device, 15)
    out = c.attend(q, [299])
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    g.gdn_kv4_read(c.t_cache, c.t_table, c.i32([0]), ko, vo, page)
    assert np.array_equal(host(ko), O.kv4_dequantise(*O.kv4_quantise(host(k))))
    for h in range(H):
        o, size, _, _ = O.attention_rows(host(q)[0, 0, 0, h:h + 1], host(ko)[0, 0, :, h], host(vo)[0, 0, :, h], [299], D ** -0.5)
        assert (np.abs(host(out)[0, 0, 0, h] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -11 * size).all()


def test_graph_and_side_stream(cuda_device):
    """Append and attention captured once and replayed as the lengths advance in device memory, and run on
    another stream, give the bits of direct calls."""
    import gated_deltanet_linear_step_gb300 as g

    B, H, Hq, D, page = 3, 2, 8, 128, 32
    a, d = (Cache(cuda_device, B, 1, H, D, page, 200) for _ in range(2))
    k, v = (values((B, 1, 1, H, D), "bf16", cuda_device, s) for s in (16, 17))
    q = values((B, 1, 1, Hq, D), "bf16", cuda_device, 18)
    pre_k, pre_v = (values((B, 1, 150, H, D), "bf16", cuda_device, s) for s in (19, 20))
    start0 = [120, 0, 149]
    for c in (a, d):
        c.append(pre_k, pre_v, [0] * B, start0)
    ws = torch.empty(g.gdn_kv4_attention_workspace_size(B, 1, 1, Hq, H, D), dtype=torch.uint8, device=cuda_device)
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
    assert torch.equal(out, (d.append(k, v, start0), d.attend(q, start0))[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        start += 1
        graph.replay()
        now = [s + 1 + i for s in start0]
        d.append(k, v, now)
        assert torch.equal(out, d.attend(q, now)), i
    assert torch.equal(a.t_cache, d.t_cache)
    assert g.gdn_read_device_error() == 0
