"""Rotary positions, attention over prompts and over shared prefixes, on the CPU: refusals at the C ABI and in the binding, the table
of frequencies, and pins of the fp64 restatement."""
import ctypes
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_operators_host import BASE, BAD_SIZES, CACHE, _ptrs, lib, no_gpu  # noqa: F401

SCALINGS = [dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="by_turns", factor=8.0, original_len=8192, low=1.0, high=4.0),
            dict(scaling="by_dim", factor=16.0, original_len=4096, low=1.0, high=32.0)]


@pytest.mark.parametrize("r", [4, 64, 122, 128, 512])
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["scaling"])
def test_turns_are_the_frequencies(lib, r, scaling):  # noqa: F811
    """2^-64 of a turn; fp64 powers and logarithms leave a few 2^-53 of a frequency."""
    import gated_deltanet_linear_step_gb300 as g

    for base in (10000.0, 500000.0):
        t = g.gdn_rope_turns(r, base=base, device="cpu", **scaling).numpy().view(np.uint64)
        want = O.rope_frequencies(r, base, **scaling) / (2 * np.pi)
        assert np.abs(t.astype(np.float64) / 2.0 ** 64 / want - 1).max() < 1e-13 + 2.0 ** -65 / want.min()
        assert (t > 0).all() and (t < 2.0 ** 62).all()


def exact_turns(r, base, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Parts of a turn per position with 50 digits."""
    getcontext().prec = 50
    atan = lambda n: sum((-1) ** k * Decimal(1) / ((2 * k + 1) * Decimal(n) ** (2 * k + 1)) for k in range(80))  # noqa: E731
    tau = 2 * (16 * atan(5) - 4 * atan(239))
    d = Decimal
    if scaling == "ntk":
        base = d(base) * (d(factor).ln() * r / (r - 2)).exp()
    f = [(-d(2 * i) / r * d(base).ln()).exp() for i in range(r // 2)]
    if scaling == "by_turns":
        keep = [(d(original_len) * x / tau - d(low)) / (d(high) - d(low)) for x in f]
    elif scaling == "by_dim":
        at = [r * (d(original_len) / (tau * d(n))).ln() / (2 * d(base).ln()) for n in (high, low)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        keep = [1 - d(i - lo) / max(d(hi - lo), d("0.001")) for i in range(r // 2)]
    else:
        keep = [d(0 if scaling == "linear" else 1)] * len(f)
    keep = [min(max(x, d(0)), d(1)) for x in keep]
    return [x * (s + (1 - s) / d(factor)) / tau for x, s in zip(f, keep)]


@pytest.mark.parametrize("r", [4, 64, 122, 512])
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["scaling"])
def test_turns_to_their_last_bits(lib, r, scaling):  # noqa: F811
    """Within 2^-53 of a turn, as stated: a frequency is at most 0.16 of one, a power is off by some 2^-53 of it times (3 + the power's logarithm), and a blend by a few more."""
    import gated_deltanet_linear_step_gb300 as g

    for base in (10000.0, 500000.0):
        t = g.gdn_rope_turns(r, base=base, device="cpu", **scaling).numpy().view(np.uint64)
        err = [abs(Decimal(int(x)) / 2 ** 64 - w) for x, w in zip(t, exact_turns(r, base, **scaling))]
        assert max(err) <= Decimal(2) ** -53, float(max(err)) * 2.0 ** 53


def test_turns_refuse(lib):  # noqa: F811
    out = (ctypes.c_uint64 * 256)()

    def call(p=out, r=64, base=1e4, scaling=0, factor=2.0, original=100.0, low=1.0, high=2.0):
        return lib.gdn_rope_turns(p, r, base, scaling, factor, original, low, high)

    assert call() == 0 and call(scaling=0, factor=0.0, original=0.0) == 0 and call(r=2) == 0
    assert call(p=None) == 1
    for scaling in (-1, 5):
        assert call(scaling=scaling) == 6
    for bad in (dict(r=0), dict(r=3), dict(r=514), dict(r=2, scaling=2), dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")),
                dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("nan")), dict(scaling=1, factor=2.0 ** 21),
                dict(scaling=3, original=0.0), dict(scaling=4, original=float("inf")), dict(scaling=3, low=2.0), dict(scaling=4, low=0.0),
                dict(scaling=4, high=float("nan"))):
        assert call(**bad) == 2, bad
    import gated_deltanet_linear_step_gb300 as g

    with pytest.raises(ValueError):
        g.gdn_rope_turns(64, scaling="other")


ROPE = dict(B=2, L=3, T=4, q_heads=8, kv_heads=2, head_dim=128, r=64, qs=1024, ks=256, gain=1.0, flags=0, dtype=0)


def _rope(lib, p, **over):  # noqa: F811
    a = dict(ROPE, **over)
    return lib.gdn_rope(p["q"], p["k"], p["qo"], p["ko"], p["turns"], p["start"], p["pos"], p["len"], a["B"], a["L"], a["T"], a["q_heads"],
                        a["kv_heads"], a["head_dim"], a["r"], a["qs"], a["ks"], a["gain"], a["flags"], a["dtype"], None)


@no_gpu
def test_rope_refuses(lib):  # noqa: F811
    p = dict(_ptrs(("q", "k", "qo", "ko", "turns", "start", "len")), pos=None)
    for bad in (dict(B=0), dict(L=0), dict(T=0), dict(T=(1 << 20) + 1), dict(q_heads=0), dict(q_heads=4097), dict(kv_heads=-1), dict(head_dim=4),
                dict(head_dim=100), dict(head_dim=520), dict(r=0), dict(r=63), dict(r=130), dict(qs=1023), dict(qs=1026), dict(ks=128), dict(qs=1 << 31),
                dict(gain=float("nan")), dict(gain=float("inf")), dict(B=1 << 20, T=1 << 12)):
        assert _rope(lib, p, **bad) == 2, bad
    assert _rope(lib, p, dtype=3) == 7 and _rope(lib, p, flags=4) == 6
    for k in ("q", "qo", "turns", "k", "ko"):
        assert _rope(lib, dict(p, **{k: None})) == 1, k
    assert _rope(lib, p, kv_heads=0) == 1  # keys without heads
    assert _rope(lib, dict(p, start=None)) == 1 and _rope(lib, dict(p, pos=BASE)) == 1
    for k in ("q", "k", "qo", "ko"):
        assert _rope(lib, dict(p, **{k: p[k] + 8})) == 3, k
    for k in ("turns", "start", "len"):
        assert _rope(lib, dict(p, **{k: p[k] + 2})) == 3, k
    assert _rope(lib, dict(p, qo=p["q"] + 1024)) == 4 and _rope(lib, dict(p, ko=p["q"])) == 4 and _rope(lib, dict(p, ko=p["qo"] + 64)) == 4
    assert _rope(lib, dict(p, turns=p["qo"] + 64)) == 4
    # in place in one projection's output: the keys' rows lie between the queries', but not on them
    f = dict(qs=1536, ks=1536)
    for off, ok in ((1024 * 4, True), (1023 * 4 + 4 - 16, False), (1280 * 4, True), (1296 * 4, False)):
        k = p["q"] + off
        got = _rope(lib, dict(p, qo=p["q"], k=k, ko=k), **f)
        assert (got != 4) == ok, (off, got)  # (a call that is in order fails at the launch: there is no GPU)


PROMPT = dict(B=3, n=100, q_heads=8, kv_heads=2, head_dim=128, qs=1024, ks=256, vs=256, os=1024, dtype=2, scale=0.1)


def _prompt(lib, p, ws=None, **over):  # noqa: F811
    a = dict(PROMPT, **over)
    if ws is None:
        ws = lib.gdn_prompt_attention_workspace_size(3, 100, 8, 2, 128, a["dtype"])
    return lib.gdn_prompt_attention(p["q"], p["k"], p["v"], p["offsets"], p["len"], p["out"], p["ws"], ws, a["B"], a["n"], a["q_heads"],
                                    a["kv_heads"], a["head_dim"], a["qs"], a["ks"], a["vs"], a["os"], a["dtype"], a["scale"], None)


@no_gpu
@pytest.mark.parametrize("dtype", [0, 2])
def test_prompt_refuses(lib, dtype):  # noqa: F811
    p = _ptrs(("q", "k", "v", "offsets", "len", "out", "ws"))
    for bad in (dict(B=0), dict(B=(1 << 20) + 1), dict(n=0), dict(n=(1 << 20) + 1), dict(q_heads=0), dict(q_heads=9), dict(q_heads=8192),
                dict(kv_heads=0), dict(kv_heads=1025, q_heads=1025), dict(head_dim=96), dict(head_dim=32), dict(n=1 << 20, q_heads=2048, kv_heads=1),
                dict(qs=1016), dict(ks=255), dict(vs=258), dict(os=1000), dict(ks=1 << 31), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert _prompt(lib, p, dtype=dtype, **bad) == 2, bad
    assert _prompt(lib, p, dtype=5) == 7
    need = lib.gdn_prompt_attention_workspace_size(3, 100, 8, 2, 128, dtype)
    for k in ("q", "k", "v", "offsets", "out") + (("ws",) if need else ()):
        assert _prompt(lib, dict(p, **{k: None}), dtype=dtype) == 1, k
        assert _prompt(lib, dict(p, **{k: p[k] + 2}), dtype=dtype) == 3, k
    if need:
        assert _prompt(lib, p, ws=need - 1, dtype=dtype) == 2
        assert _prompt(lib, dict(p, ws=p["out"] + 64), dtype=dtype) == 4 and _prompt(lib, dict(p, ws=p["k"]), dtype=dtype) == 4
    assert _prompt(lib, dict(p, out=p["q"]), dtype=dtype) == 4 and _prompt(lib, dict(p, out=p["v"] + 64), dtype=dtype) == 4
    assert _prompt(lib, dict(p, offsets=p["out"] + 64), dtype=dtype) == 4
    for args in ((0, 1, 8, 4, 128, 0), (1, 0, 8, 4, 128, 0), (1, 1, 9, 4, 128, 0), (1, 1, 8, 4, 80, 0), (1, 1, 8, 4, 128, 3)):
        assert lib.gdn_prompt_attention_workspace_size(*args) == 0, args


@no_gpu
def test_shared_refuses(lib):  # noqa: F811
    names = ("q", "cache", "ptable", "plen", "groups", "table", "start", "len", "out", "ws")
    p = _ptrs(names)
    need = lib.gdn_kv4_attention_shared_workspace_size(2, 3, 4, 20, 4, 128)
    assert need > lib.gdn_kv4_attention_workspace_size(2, 3, 4, 20, 4, 128) > 0

    def call(p, ws=need, q_heads=20, scale=0.1, groups=2, far=7, **over):
        a = dict(CACHE, **over)
        return lib.gdn_kv4_attention_shared(p["q"], p["cache"], p["ptable"], p["plen"], p["groups"], p["table"], p["start"], p["len"], p["out"],
                                            p["ws"], ws, a["B"], a["L"], a["T"], groups, q_heads, a["kv_heads"], a["head_dim"], a["n_pages"], far,
                                            a["max_pages"], a["page_size"], a["dtype"], scale, None)

    for over in BAD_SIZES + [dict(groups=0), dict(groups=-1), dict(groups=3), dict(far=0), dict(far=1 << 25), dict(B=1 << 11, T=1 << 10)]:
        assert call(p, **over) == 2, over
    assert call(p, dtype=9) == 7
    for q_heads in (0, 6, -4, 8192):
        assert call(p, q_heads=q_heads) == 2, q_heads
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(p, scale=scale) == 2, scale
    assert call(p, ws=need - 16) == 2
    for k in names:
        if k != "len":
            assert call(dict(p, **{k: None})) == 1, k
        assert call(dict(p, **{k: p[k] + 2})) == 3, k
    assert call(dict(p, out=p["q"] + 64)) == 4 and call(dict(p, out=p["cache"])) == 4 and call(dict(p, ws=p["out"] + 64)) == 4
    assert call(dict(p, plen=p["ws"] + 64)) == 4
    for args in ((0, 1, 1, 8, 4, 128), (1, 1, 0, 8, 4, 128), (1, 1, 1, 9, 4, 128), (1, 1, 1, 8, 4, 80), (1 << 11, 1, 1 << 10, 8, 4, 128)):
        assert lib.gdn_kv4_attention_shared_workspace_size(*args) == 0, args


def test_binding_refuses_on_the_cpu(lib):  # noqa: F811
    import gated_deltanet_linear_step_gb300 as g

    x = torch.zeros(1, 1, 2, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        g.gdn_rope(x, None, torch.zeros(32, dtype=torch.int64), x, None, start=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        g.gdn_prompt_attention(x[0, 0], x[0, 0], x[0, 0], torch.zeros(2, dtype=torch.int32), x[0, 0])
    with pytest.raises(TypeError):
        g.gdn_prompt_attention(x[0, 0].double(), x[0, 0], x[0, 0], torch.zeros(2, dtype=torch.int32), x[0, 0])
    with pytest.raises(ValueError, match=r"\[B\]\[L\]"):
        g.gdn_kv4_attention_shared(x[0], x, x, x, x, x, x, x, x, 16, 4)


def test_restated_rotation():
    """Lengths stay, the inverse undoes it, and products depend on the distance alone."""
    rng = np.random.default_rng(0)
    for interleaved in (False, True):
        f = O.rope_frequencies(24)
        x, y = rng.standard_normal((2, 5, 1, 40))
        a = O.rope(x, np.arange(5) * 7, f, interleaved)
        assert np.allclose((a ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(a[..., 24:], x[..., 24:])
        assert np.allclose(O.rope(a, np.arange(5) * 7, f, interleaved, inverse=True), x)
        dots = [(O.rope(x, np.full(5, p), f, interleaved) * O.rope(y, np.full(5, p + 11), f, interleaved)).sum(-1) for p in (0, 123)]
        assert np.allclose(*dots)
        assert np.allclose(O.rope(x, np.zeros(5), f, interleaved, gain=2.0)[..., :24], 2 * x[..., :24])
