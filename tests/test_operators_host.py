"""The operators beside the decode step, on the CPU: their refusals at the C ABI and in the binding, and pins
of their fp64 restatement (number format, page layout, attention, log probabilities)."""
import os

import numpy as np
import pytest
import torch

from oracle import operators as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "gated_deltanet_linear_step_gb300", "libgdn.so")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        from gated_deltanet_linear_step_gb300 import _build

        _build.build()
    import gated_deltanet_linear_step_gb300 as g

    return g.load_library()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake pointers are only passed where no GPU exists")

BASE = 1 << 41
CACHE = dict(B=2, L=3, T=4, kv_heads=4, head_dim=128, n_pages=10, max_pages=3, page_size=64, dtype=0)


def _ptrs(names):
    return {k: BASE + (i << 32) for i, k in enumerate(names)}


def _append(lib, p, **over):
    a = dict(CACHE, **over)
    return lib.gdn_kv4_append(p["k"], p["v"], p["cache"], p["table"], p["start"], p["len"], a["B"], a["L"], a["T"],
                              a["kv_heads"], a["head_dim"], a["n_pages"], a["max_pages"], a["page_size"], a["dtype"], None)


def _read(lib, p, **over):
    a = dict(CACHE, **over)
    return lib.gdn_kv4_read(p["cache"], p["table"], p["start"], p["len"], p["k"], p["v"], a["B"], a["L"], a["T"],
                            a["kv_heads"], a["head_dim"], a["n_pages"], a["max_pages"], a["page_size"], a["dtype"], None)


BAD_SIZES = [dict(B=0), dict(L=0), dict(T=0), dict(T=(1 << 20) + 1), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96),
             dict(head_dim=512), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(n_pages=0), dict(max_pages=0),
             dict(max_pages=1 << 25), dict(B=1 << 20, T=1 << 12), dict(L=-1)]


@no_gpu
@pytest.mark.parametrize("call", [_append, _read])
def test_cache_calls_refuse(lib, call):
    names = ("k", "v", "cache", "table", "start", "len")
    p = _ptrs(names)
    for over in BAD_SIZES:
        assert call(lib, p, **over) == 2, over
    for dtype in (-1, 3):
        assert call(lib, p, dtype=dtype) == 7
        assert b"data type" in lib.gdn_last_error()
    for k in names[:-1]:  # seq_len may be NULL
        assert call(lib, dict(p, **{k: None})) == 1, k
        assert k[:4].encode() in lib.gdn_last_error() or k in ("table", "start")
    for k in ("k", "v", "cache"):
        assert call(lib, dict(p, **{k: p[k] + 8})) == 3, k
    for k in ("table", "start", "len"):
        assert call(lib, dict(p, **{k: p[k] + 2})) == 3, k
    if call is _append:
        assert call(lib, dict(p, k=p["cache"] + 4096)) == 4
        assert call(lib, dict(p, table=p["cache"] + 64)) == 4
    else:
        assert call(lib, dict(p, v=p["k"] + 64)) == 4
        assert call(lib, dict(p, k=p["cache"] + 4096)) == 4
        assert call(lib, dict(p, len=p["v"] + 64)) == 4


@no_gpu
def test_attention_refuses(lib):
    names = ("q", "cache", "table", "start", "len", "out", "ws")
    p = _ptrs(names)
    need = lib.gdn_kv4_attention_workspace_size(2, 3, 4, 20, 4, 128)
    assert need > 0

    def call(p, ws=need, q_heads=20, scale=0.1, **over):
        a = dict(CACHE, **over)
        return lib.gdn_kv4_attention(p["q"], p["cache"], p["table"], p["start"], p["len"], p["out"], p["ws"], ws, a["B"], a["L"],
                                     a["T"], q_heads, a["kv_heads"], a["head_dim"], a["n_pages"], a["max_pages"], a["page_size"],
                                     a["dtype"], scale, None)

    for over in BAD_SIZES:
        assert call(p, **over) == 2, over
    assert call(p, dtype=9) == 7
    for q_heads in (0, 6, -4, 8192):
        assert call(p, q_heads=q_heads) == 2, q_heads
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(p, scale=scale) == 2, scale
    assert call(p, ws=need - 16) == 2
    assert b"workspace" in lib.gdn_last_error()
    for k in names:
        if k != "len":
            assert call(dict(p, **{k: None})) == 1, k
        assert call(dict(p, **{k: p[k] + 2})) == 3, k
    assert call(dict(p, out=p["q"] + 64)) == 4
    assert call(dict(p, out=p["cache"])) == 4
    assert call(dict(p, ws=p["out"] + 64)) == 4


def test_sizes_out_of_range_have_no_bytes(lib):
    assert lib.gdn_kv4_page_bytes(4, 128, 64) == 4 * 2 * 64 * (64 + 8)
    assert lib.gdn_kv4_page_bytes(1, 64, 16) == 2 * 16 * 36
    for args in ((0, 128, 64), (4, 100, 64), (4, 128, 24), (4, 128, 8)):
        assert lib.gdn_kv4_page_bytes(*args) == 0, args
    for args in ((0, 1, 1, 8, 4, 128), (1, 1, 0, 8, 4, 128), (1, 1, 1, 9, 4, 128), (1, 1, 1, 8, 4, 80), (1, 1, 1, 8, 0, 64)):
        assert lib.gdn_kv4_attention_workspace_size(*args) == 0, args


@no_gpu
def test_logprobs_refuses(lib):
    names = ("logits", "tokens", "logprob", "entropy", "ids", "top")
    p = _ptrs(names)

    def call(p, n=3, vocab=1000, ld=1000, k=5, dtype=0):
        return lib.gdn_logprobs(*[p[x] for x in names], n, vocab, ld, k, dtype, None)

    for over in (dict(n=0), dict(n=(1 << 26) + 1), dict(vocab=0), dict(ld=999), dict(vocab=1 << 31, ld=1 << 31), dict(k=33), dict(k=-1),
                 dict(vocab=4, k=5), dict(ld=1 << 40)):
        assert call(p, **over) == 2, over
    assert call(p, dtype=3) == 7
    for k in ("logits", "tokens", "ids", "top"):
        assert call(dict(p, **{k: None})) == 1, k
    for k in names:
        assert call(dict(p, **{k: p[k] + 2})) == 3, k
    assert call(dict(p, logits=p["logits"] + 1), dtype=2) == 3
    assert call(dict(p, logprob=p["logits"] + 8)) == 4
    assert call(dict(p, entropy=p["logprob"] + 4)) == 4
    assert call(dict(p, top=p["ids"] + 4)) == 4


def test_the_binding_refuses_before_any_call(lib):
    import gated_deltanet_linear_step_gb300 as g

    k = torch.zeros(1, 1, 1, 1, 64)
    cache = torch.zeros(1, 2, 1152, dtype=torch.uint8)
    i32 = torch.zeros(1, dtype=torch.int32)
    table = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.gdn_kv4_append(k, k, cache, table, i32, 16)
    with pytest.raises(TypeError, match="k must be"):
        g.gdn_kv4_append(k.double(), k, cache, table, i32, 16)
    with pytest.raises(ValueError, match="head_dim"):
        g.gdn_kv4_read(cache, table, i32, k[0], k[0], 16)
    with pytest.raises(ValueError, match="q must be"):
        g.gdn_kv4_attention(k[0], cache, table, i32, k, cache.view(-1), 16, 1)
    with pytest.raises(TypeError, match="workspace"):
        g.gdn_kv4_attention(k, cache, table, i32, k, k, 16, 1)
    with pytest.raises(ValueError, match="vocab"):
        g.gdn_logprobs(torch.zeros(4))
    with pytest.raises(TypeError, match="logits"):
        g.gdn_logprobs(torch.zeros(4, 4, dtype=torch.int32))


# ------------------------------------------------------------------ the restatement --
def test_format_pins():
    """Hand-computed blocks: the scale of 6 is 1, ties go to the even code, the sign is kept."""
    x = np.zeros(16)
    x[:9] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.1]
    code, byte = O.kv4_quantise(x)
    assert byte[0] == 15 << 3 and O.scale_values()[byte[0]] == 1.0
    assert list(code[:9]) == [7, 0, 2, 2, 4, 4, 6, 6, 15]
    assert np.array_equal(O.kv4_dequantise(code, byte)[:9], [6, 0, 1, 1, 2, 2, 4, 4, -6])
    # saturation and NaN
    x = np.array([np.inf, -np.inf, np.nan, 1e9] + [61440.0] * 12)
    code, byte = O.kv4_quantise(x)
    assert byte[0] == O.MAX_SCALE_BYTE and O.scale_values()[226] == 10240.0
    assert np.array_equal(O.kv4_dequantise(code, byte)[:4], [61440, -61440, 0, 61440])
    # values below half the smallest scale vanish
    code, byte = O.kv4_quantise(np.full(16, 2.0 ** -18 * 6 * 0.999))
    assert byte[0] == 0 and not code.any()
    # the scale grid is the fp16 numbers with the bits b << 7
    half = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(half, O.scale_values())


def test_quantising_twice_changes_nothing():
    x = np.random.default_rng(0).normal(size=(50, 64)) * 10.0 ** np.random.default_rng(1).uniform(-3, 3, (50, 1))
    code, byte = O.kv4_quantise(x)
    y = O.kv4_dequantise(code, byte)
    assert np.array_equal(O.kv4_dequantise(*O.kv4_quantise(y)), y)
    # half a step of e2m1 (2^-2 of the value from 1 on) plus what the scale's rounding (half of 2^-3) cuts off at the top
    blocks = np.abs(y - x).reshape(50, 4, 16).max(-1) / np.abs(x).reshape(50, 4, 16).max(-1)
    assert blocks.max() <= 1.0 / 6.0 + 2.0 ** -4


@pytest.mark.parametrize("D,page", [(64, 16), (128, 32), (256, 16)])
def test_pages_hold_what_was_appended(D, page):
    rng = np.random.default_rng(2)
    B, L, T, H = 2, 2, page + 3, 2
    k, v = rng.normal(size=(2, B, L, T, H, D))
    table = np.array([[3, 0, 5], [1, 4, 2]])
    cache = rng.integers(0, 256, (L, 6, H * 2 * page * (D // 2 + D // 16)), dtype=np.uint8)
    start = np.array([5, 0])
    O.kv4_append(k, v, cache, table, start, page)
    for b in range(B):
        for h in range(H):
            gk, gv = O.kv4_read(cache, table, b, 1, h, start[b] + T, page, D, start[b])
            assert np.array_equal(gk, O.kv4_dequantise(*O.kv4_quantise(k[b, 1, :, h])))
            assert np.array_equal(gv, O.kv4_dequantise(*O.kv4_quantise(v[b, 1, :, h])))


def test_attention_and_logprobs_pins():
    q = np.array([[1.0, 0.0], [0.0, 2.0]])
    k = np.array([[np.log(3.0), 0.0], [0.0, 0.0], [7.0, np.log(2.0) / 2]])
    v = np.array([[4.0, 0.0], [0.0, 8.0], [1.0, 1.0]])
    o = O.attention_rows(q, k, v, [1, 2], 1.0)[0]
    assert np.allclose(o[0], [3.0, 2.0]) and np.allclose(o[1], [1.5, 2.5])
    x = np.log(np.array([[0.5, 0.25, 0.25, 0.0]]) + 1e-300)
    x[0, 3] = -np.inf
    lp, ent, ids, top = O.logprobs(x, [1], 4)
    assert np.allclose(lp, np.log(0.25)) and np.allclose(ent, 1.5 * np.log(2.0))
    assert list(ids[0]) == [0, 1, 2, 3] and top[0, 3] == -np.inf
    lp, ent, ids, top = O.logprobs(np.array([[1.0, np.nan, 3.0], [-np.inf] * 3]), [0, 0], 2)
    assert np.isnan(lp).all() and np.isnan(ent).all() and list(ids[0]) == [1, 2] and list(ids[1]) == [0, 1]
