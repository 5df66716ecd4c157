"""Attention over the 4-bit cache for batches that share prefixes, against the fp64 restatement and against the same keys cached per
sequence; helpers and tolerances are those of test_gpu_kv4.py, with the sum over both parts."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_kv4 import TYPES, Cache, host, values

pytestmark = pytest.mark.gpu


class Shared(Cache):
    """A cache whose first rows of pages are the groups' prefixes and whose others are the sequences'."""

    def __init__(self, dev, prefix, groups, B, L, H, D, page, tokens, seed=0):
        super().__init__(dev, B + len(prefix), L, H, D, page, max(tokens, max(prefix), 1), seed=seed)
        self.prefix, self.groups, self.n = prefix, groups, len(prefix)
        self.t_prefix, self.t_own = self.t_table[:self.n].contiguous(), self.t_table[self.n:].contiguous()

    def fill(self, k, v, start, own):
        """k, v [G + B][L][tokens][H][D]: the prefixes' rows and the sequences'."""
        self.append(k, v, [0] * (self.n + own), [*self.prefix, *start])

    def shared(self, q, start, n=None, out=None, scale=None, prefix=None, groups=None):
        B, L, T, Hq, D = q.shape
        out = torch.full_like(q, float("nan")) if out is None else out
        ws = torch.full((self.g.gdn_kv4_attention_shared_workspace_size(B, L, T, Hq, self.H, D),), 255, dtype=torch.uint8, device=self.dev)
        self.g.gdn_kv4_attention_shared(q, self.t_cache, self.t_prefix, self.i32(prefix or self.prefix), self.i32(groups or self.groups), self.t_own,
                                        self.i32(start), out, ws, self.page, self.H, scale=scale, seq_len=self.i32(n))
        return out

    def check(self, q, out, start, n, dtype, rows=None):
        B, L, T, Hq, D = q.shape
        G, scale = Hq // self.H, D ** -0.5
        cache, got, qh = self.t_cache.cpu().numpy(), host(out), host(q)
        info = torch.finfo(TYPES[dtype])
        half, least = info.eps / 2, info.smallest_normal * info.eps / 2
        p_step = 2.0 ** -22 if dtype == "fp32" else 2.0 ** -12
        worst = 0.0
        for b in range(B):
            m = T if n is None else min(max(n[b], 0), T)
            assert np.isnan(got[b, :, m:]).all(), "a row past the window was written"
            g = max(i for i in range(self.n) if self.groups[i] <= b and self.groups[i] < self.groups[i + 1])
            far = self.prefix[g]
            for l in range(L):
                for h in range(self.H):
                    if m == 0 or (rows is not None and (b, l, h) not in rows):
                        continue
                    pk, pv = O.kv4_read(cache, self.table, g, l, h, far, self.page, D)
                    k, v = O.kv4_read(cache, self.table, self.n + b, l, h, start[b] + m, self.page, D)
                    k, v = np.concatenate([pk, k]), np.concatenate([pv, v])
                    for i in range(h * G, h * G + G):
                        o, size, qk, s = O.attention_rows(qh[b, l, :m, i], k, v, far + start[b] + np.arange(m), scale)
                        # the parts' factors: two more exponentials and roundings
                        rel = p_step + 3 * ((D + 8) * 2.0 ** -24 * qk + 2.0 ** -22 * (2 + s)) + 2 * (far + start[b] + m) * 2.0 ** -24
                        err = np.abs(got[b, l, :m, i] - o)
                        # a probability is off by 2^-34 of the row's largest, which is 1 at most, where that is more than its rounding
                        # (and is 0 below 2^-135 of it): the sum of its values' sizes times that
                        lost = 2.0 ** -34 * np.abs(v[:far + start[b] + m]).sum(0)
                        worst = max(worst, float((err / (half * np.abs(o) + least + rel * size + lost)).max()))
        assert worst <= 1.0, worst
        return worst


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B,L,T,Hq,H,D,page,prefix,groups,start,n", [
    (1, 1, 1, 1, 1, 64, 16, [1], [0, 1], [0], None),                                   # one key each
    (3, 1, 1, 4, 4, 128, 16, [37], [0, 3], [0, 5, 20], None),                           # three rows: no tensor cores
    (5, 1, 1, 20, 4, 128, 32, [200], [0, 5], [3, 0, 40, 31, 32], None),                 # 25 rows over the prefix, single tokens
    (4, 2, 3, 6, 2, 64, 64, [130, 64], [0, 1, 4], [10, 0, 77, 1], [3, 0, 1, 2]),        # two groups, ragged windows
    (6, 1, 8, 8, 1, 128, 16, [100, 0, 33], [0, 2, 2, 6], [9, 1, 0, 2, 3, 50], None),    # an empty group, windows on the tensor cores
    (3, 1, 2, 4, 2, 256, 128, [0, 300], [0, 1, 3], [0, 40, 7], None),                   # a group without a prefix
    (40, 1, 1, 8, 1, 64, 64, [3000], [0, 40], [i for i in range(40)], None),            # 320 rows, a prefix over many CTAs
    (2, 1, 1, 2, 1, 128, 256, [5000], [0, 2], [600, 3], None),                          # few rows over a long prefix
])
def test_matches_restatement(cuda_device, B, L, T, Hq, H, D, page, prefix, groups, start, n, dtype):
    c = Shared(cuda_device, prefix, groups, B, L, H, D, page, max(start) + T)
    tokens = max(max(prefix), max(start) + T)
    k, v = (values((len(prefix) + B, L, tokens, H, D), dtype, cuda_device, s) for s in (1, 2))
    c.fill(k, v, [s + T for s in start], B)
    q = values((B, L, T, Hq, D), dtype, cuda_device, 3)
    out = c.shared(q, start, n)
    assert c.g.gdn_read_device_error() == 0
    print(c.check(q, out, start, n, dtype))
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(c.shared(q, start, n))), "two calls differ"


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("fp16", 64, 32), ("bf16", 64, 256), ("fp16", 128, 128)])
@pytest.mark.parametrize("B,L,T,G,prefix,groups", [
    (17, 1, 1, 1, [128], [0, 17]),                            # one row more than the streaming kernel takes, one whole tile
    (32, 1, 4, 1, [129], [0, 32]),                            # 128 rows, a tile of one key
    (33, 1, 4, 1, [127], [0, 33]),                            # 132 rows: two blocks, the second of four
    (26, 1, 1, 10, [1000], [0, 26]),                          # 260 rows: a unit of 256 and one of four
    (40, 1, 1, 9, [2600], [0, 40]),                           # 360 rows: the second unit of 104
    (60, 2, 1, 5, [40, 700, 0, 3000, 257], [0, 3, 10, 12, 40, 60]),   # units of every kind on one line, a group without a prefix
    (12, 3, 8, 4, [1, 2, 3, 130, 5, 6], [0, 2, 4, 6, 8, 10, 12]),     # short units: many of them in a CTA
    (64, 1, 1, 4, [20000], [0, 64]),                          # one unit over all CTAs
])
def test_many_rows_match_restatement(cuda_device, B, L, T, G, prefix, groups, dtype, D, page):
    start = [(5 * i) % 11 for i in range(B)]
    c = Shared(cuda_device, prefix, groups, B, L, 2, D, page, 11 + T)
    k, v = (values((len(prefix), L, max(prefix), 2, D), dtype, cuda_device, s) for s in (21, 22))
    full = [torch.zeros(len(prefix) + B, *x.shape[1:], dtype=x.dtype, device=cuda_device) for x in (k, v)]
    own = [values((B, L, min(11 + T, max(prefix)), 2, D), dtype, cuda_device, s) for s in (23, 24)]
    if max(prefix) < 11 + T:  # the sequences' own tokens need the longer window
        full = [torch.zeros(len(prefix) + B, L, 11 + T, 2, D, dtype=k.dtype, device=cuda_device) for _ in range(2)]
        own = [values((B, L, 11 + T, 2, D), dtype, cuda_device, s) for s in (23, 24)]
    for f, p_, o in zip(full, (k, v), own):
        f[:len(prefix), :, :p_.shape[2]] = p_
        f[len(prefix):, :, :o.shape[2]] = o
    c.fill(full[0], full[1], [s + T for s in start], B)
    q = values((B, L, T, 2 * G, D), dtype, cuda_device, 25)
    out = c.shared(q, start)
    assert c.g.gdn_read_device_error() == 0
    rows = {(b, l, h) for b in {0, 1, B // 2, B - 2, B - 1} for l in (0, L - 1) for h in range(2)}
    print(c.check(q, out, start, None, dtype, rows=rows))
    for _ in range(5):
        assert torch.equal(out, c.shared(q, start)), "two calls differ"
    assert c.g.gdn_read_device_error() == 0


def test_a_prefix_longer_than_a_run_of_sums(cuda_device):
    """Equal keys and values (0.75, which the cache holds) over 300000 tokens: a CTA has about 300 tiles of a unit and its sums start afresh every
    128. Every output is the value, up to its rounding (2^-12 of 0.75), what matrix instructions cut off of at most 1024 steps of a run
    (2^-23 each) and the fp32 sums of the probabilities (2400 of either sign)."""
    n, B, H = 300000, 3, 20
    for G in (8, 60):  # a unit of up to 128 rows, and one of two blocks
        c = Shared(cuda_device, [n], [0, B], B, 1, H, 64, 256, 8)
        k = torch.full((1, 1, n, H, 64), 0.25, dtype=torch.float16, device=cuda_device)
        c.g.gdn_kv4_append(k, torch.full_like(k, 0.75), c.t_cache, c.t_prefix, c.i32([0]), 256)
        own = torch.full((B, 1, 8, H, 64), 0.25, dtype=torch.float16, device=cuda_device)
        c.g.gdn_kv4_append(own, torch.full_like(own, 0.75), c.t_cache, c.t_own, c.i32([0] * B), 256)
        q = values((B, 1, 1, H * G, 64), "fp16", cuda_device, 26)
        out = c.shared(q, [7] * B)
        assert c.g.gdn_read_device_error() == 0
        worst = float((out.double() - 0.75).abs().max()) / 0.75
        assert worst <= 2.0 ** -11 + 1024 * 2.0 ** -23 + 2400 * 2.0 ** -24, worst


@pytest.mark.parametrize("G", [8, 60])  # a unit of up to 128 rows, and one of two blocks
def test_maxima_that_rise_between_runs_of_sums(cuda_device, G):
    """60 stretches of 10000 tokens of the prefix, each with one key and one value. A stretch's score is 3 (in base 2) above the one's before it, so the
    reference maximum is raised every third, and the last CTA of a unit, which has some 40000 (two blocks) or 80000 tokens, starts its sums
    afresh twice on the way: the earlier ones have to be scaled to the new maximum, and differ in value.

    Keys are exact in the cache: 0.75 a at dim 0 and 0.75 b at dim 16, 16 a + b the number of the stretch. Tolerance, relative (all values are positive): the
    output's rounding, 2^-12 for each probability's (twice: products and sum), 2^-22 of the largest score (180) for the scale's and the exponential's argument,
    twice, what matrix instructions cut off of at most 1024 steps of a run, and the fp32 sums of some 2500 probabilities a row and run."""
    n, B, H, each = 600000, 3, 20, 10000
    c = Shared(cuda_device, [n], [0, B], B, 1, H, 64, 256, 8)
    level = [0.5, 6.0, 1.0, 4.0, 1.5, 3.0, 2.0]
    for s in range(n // each):
        k = torch.zeros((1, 1, each, H, 64), dtype=torch.float16, device=cuda_device)
        k[..., 0], k[..., 16] = 0.75 * (s // 16), 0.75 * (s % 16)
        c.g.gdn_kv4_append(k, torch.full_like(k, level[s % 7]), c.t_cache, c.t_prefix, c.i32([s * each]), 256)
    own = torch.zeros((B, 1, 8, H, 64), dtype=torch.float16, device=cuda_device)
    c.g.gdn_kv4_append(own, own, c.t_cache, c.t_own, c.i32([0] * B), 256)
    q = torch.zeros((B, 1, 1, H * G, 64), dtype=torch.float16, device=cuda_device)
    q[..., 0], q[..., 16] = 16.0, 1.0
    out = c.shared(q, [7] * B, scale=4.0 / np.log2(np.e))
    assert c.g.gdn_read_device_error() == 0
    w = 2.0 ** (3.0 * (np.arange(n // each) - n // each))
    held = [float(O.kv4_dequantise(*O.kv4_quantise(np.full(16, x)))[0]) for x in level]  # (a sixth of 0.5 is no scale of the cache, nor of 4, 1 or 2)
    want = (w * [held[s % 7] for s in range(n // each)]).sum() / w.sum()
    worst = float((out.double() - want).abs().max()) / want
    assert worst <= 2.0 ** -11 + 2 * 2.0 ** -12 + 2 * 2.0 ** -22 * 180 + 1024 * 2.0 ** -23 + 2500 * 2.0 ** -24, worst


@pytest.mark.parametrize("dtype,T", [("fp32", 1), ("bf16", 5)])
def test_what_is_masked_does_not_matter(cuda_device, dtype, T):
    """Bytes of 255 past the prefix, its last page's rest and past the windows; queries that are NaN or infinite."""
    B, start = 6, [3, 0, 30, 16, 15, 1]
    c = Shared(cuda_device, [75, 20], [0, 4, 6], B, 1, 2, 128, 32, 80)
    k, v = (values((B + 2, 1, 80, 2, 128), dtype, cuda_device, s) for s in (4, 5))
    q = values((B, 1, T, 8, 128), dtype, cuda_device, 6)
    c.fill(k, v, [s + T for s in start], B)
    want = c.shared(q, start)
    c.check(q, want, start, None, dtype)
    c.t_cache = torch.full_like(c.t_cache, 255)
    c.fill(k, v, [s + T for s in start], B)
    assert torch.equal(c.shared(q, start), want)
    bad = q.clone()
    bad[1, 0, 0, 2, 5], bad[5, 0, T - 1, 7, 0] = float("nan"), float("inf")
    got = c.shared(bad, start)
    same = torch.ones(q.shape[:4], dtype=torch.bool, device=cuda_device)
    same[1, 0, 0, 2] = same[5, 0, T - 1, 7] = False
    assert torch.equal(got[same], want[same]) and torch.isnan(got[1, 0, 0, 2]).all() and torch.isnan(got[5, 0, T - 1, 7]).all()


@pytest.mark.parametrize("T", [1, 6])
def test_far_apart_parts(cuda_device, T):
    """Scores of one part far above the other's: the other leaves no trace, and nothing overflows."""
    B, start = 3, [8, 8, 8]
    for big in (0, 1):
        c = Shared(cuda_device, [50], [0, B], B, 1, 1, 64, 16, 64)
        k, v = (values((B + 1, 1, 64, 1, 64), "fp32", cuda_device, s) for s in (7, 8))
        k[:1] *= 400.0 if big == 0 else 1e-3
        k[1:] *= 400.0 if big == 1 else 1e-3
        c.fill(k, v, [s + T for s in start], B)
        q = values((B, 1, T, 4, 64), "fp32", cuda_device, 9)
        c.check(q, c.shared(q, start), start, None, "fp32")


def test_missing_pages_and_borders_are_reported(cuda_device):
    B, start = 4, [5, 0, 20, 33]
    c = Shared(cuda_device, [40, 17], [0, 2, 4], B, 1, 1, 64, 16, 48)
    k, v = (values((B + 2, 1, 48, 1, 64), "fp32", cuda_device, s) for s in (10, 11))
    c.g.gdn_read_device_error()
    c.append(k, v, [0] * (B + 2))  # (a length past the prefix reads what is there)
    q = values((B, 1, 1, 2, 64), "fp32", cuda_device, 12)
    want = c.shared(q, start)
    c.check(q, want, start, None, "fp32")
    assert c.g.gdn_read_device_error() == 0
    for prefix in ([40, 1000], [-1, 17]):  # longer than its table, negative
        got = c.shared(q, start, prefix=prefix)
        assert torch.isfinite(got).all() and c.g.gdn_read_device_error() == 2, prefix
    for groups in ([0, 5, 4], [0, -1, 4], [1, 2, 4], [0, 2, 3], [0, 2, 9]):
        got = c.shared(q, start, groups=groups)
        assert torch.isfinite(got).all() and c.g.gdn_read_device_error() == 4, groups
        if groups[1] == 2:  # the ends are taken as 0 and B
            assert torch.equal(got, want)
    c.t_prefix = c.t_prefix.clone()
    c.t_prefix[1, 0] = -1
    got = c.shared(q, start)
    assert torch.equal(got[:2], want[:2]) and not torch.equal(got[2:], want[2:]) and torch.isfinite(got).all() and c.g.gdn_read_device_error() == 2
    c.t_prefix.fill_(-1)
    c.t_own = torch.full_like(c.t_own, 1 << 20)
    assert (c.shared(q, start) == 0).all() and c.g.gdn_read_device_error() == 2


def test_graph_replays_as_lengths_advance(cuda_device):
    B, T = 5, 1
    c = Shared(cuda_device, [100, 64], [0, 3, 5], B, 1, 2, 128, 32, 128)
    k, v = (values((B + 2, 1, 128, 2, 128), "bf16", cuda_device, s) for s in (13, 14))
    c.fill(k, v, [128] * B, B)
    q = values((B, 1, T, 8, 128), "bf16", cuda_device, 15)
    start, plen, groups = c.i32([0, 3, 9, 60, 31]), c.i32([100, 64]), c.i32([0, 3, 5])
    ws = torch.empty(c.g.gdn_kv4_attention_shared_workspace_size(B, 1, T, 8, 2, 128), dtype=torch.uint8, device=cuda_device)
    out = torch.empty_like(q)

    def step():
        c.g.gdn_kv4_attention_shared(q, c.t_cache, c.t_prefix, plen, groups, c.t_own, start, out, ws, 32, 2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        start += i
        plen -= 7 * i
        if i == 2:
            groups[1] = 1
        graph.replay()
        assert torch.equal(out, c.shared(q, start.tolist(), prefix=plen.tolist(), groups=groups.tolist())), i
    assert c.g.gdn_read_device_error() == 0
