"""Rotary positions on the GPU against their fp64 restatement.

Tolerance of an output a cos - b sin: its own rounding (eps / 2 of it, or half the type's smallest step), and, in units of
gain (|a| + |b|), what cosine and sine are off by (2 ulp of sincospif, 2^-23; the angle's rounding to 24 bits within an eighth of a turn, 0.8 2^-24, and to
2^-32 of a turn; the product with the gain, 2^-24: 2^-22 in all) and two roundings of products and sum (2^-23)."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests.test_gpu_kv4 import TYPES, host, values
from tests.test_prompt_operators_host import SCALINGS, exact_turns

pytestmark = pytest.mark.gpu


def check(x, out, pos, f, dtype, interleaved=False, inverse=False, gain=1.0, valid=None):
    xh, got = host(x), host(out)
    B, L, T = x.shape[:3]
    pos = np.broadcast_to(np.asarray(pos, np.float64).reshape(B, 1, T), (B, L, T))
    want = O.rope(xh, pos, f, interleaved, inverse, gain)
    size = np.zeros_like(xh)
    n = len(f)
    pair = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else (np.arange(n), np.arange(n, 2 * n))
    size[..., pair[0]] = size[..., pair[1]] = abs(gain) * (np.abs(xh[..., pair[0]]) + np.abs(xh[..., pair[1]]))
    info = torch.finfo(TYPES[dtype])
    tol = info.eps / 2 * np.abs(want) + info.smallest_normal * info.eps / 2 + size * (2.0 ** -22 + 2.0 ** -23)
    ok = np.ones(got.shape, bool) if valid is None else np.broadcast_to(np.asarray(valid).reshape(B, 1, T, 1, 1), got.shape)
    assert (np.abs(got - want)[ok] <= tol[ok]).all(), (np.abs(got - want) / tol)[ok].max()
    assert np.array_equal(got[..., 2 * n:][ok[..., 2 * n:]], xh[..., 2 * n:][ok[..., 2 * n:]]), "dims that do not turn changed"


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,L,T,Hq,Hk,D,r", [
    (1, 1, 1, 1, 0, 8, 2),          # the smallest
    (1, 1, 1, 20, 4, 128, 64),
    (3, 2, 5, 4, 1, 64, 64),
    (2, 1, 33, 5, 5, 128, 122),     # 61 pairs
    (1, 3, 7, 16, 2, 256, 96),
    (2, 1, 9, 3, 2, 512, 512),
    (1, 1, 700, 40, 8, 40, 12),
    (1, 36, 1, 20, 4, 128, 128),    # all of a model's layers
])
def test_matches_restatement(cuda_device, B, L, T, Hq, Hk, D, r, interleaved, dtype):
    import gated_deltanet_linear_step_gb300 as g

    q = values((B, L, T, Hq, D), dtype, cuda_device, 1)
    k = values((B, L, T, Hk, D), dtype, cuda_device, 2) if Hk else None
    start = [3 + 100000 * b for b in range(B)]
    pos = np.array(start)[:, None] + np.arange(T)
    f = O.rope_frequencies(r)
    turns = g.gdn_rope_turns(r, device=cuda_device)
    st = torch.tensor(start, dtype=torch.int32, device=cuda_device)
    for inverse, gain in ((False, 1.0), (True, 1.25)):
        qo, ko = torch.full_like(q, 7.0), None if k is None else torch.full_like(k, 7.0)
        g.gdn_rope(q, k, turns, qo, ko, start=st, interleaved=interleaved, inverse=inverse, gain=gain)
        check(q, qo, pos, f, dtype, interleaved, inverse, gain)
        if k is not None:
            check(k, ko, pos, f, dtype, interleaved, inverse, gain)
        # in place, by positions
        q2, k2 = q.clone(), None if k is None else k.clone()
        p = torch.tensor(pos, dtype=torch.int32, device=cuda_device)
        g.gdn_rope(q2, k2, turns, q2, k2, positions=p, interleaved=interleaved, inverse=inverse, gain=gain)
        assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["scaling"])
def test_far_and_negative_positions(cuda_device, scaling, interleaved):
    """Up to the ends of 32 bits: the tables are 2^-53 of a frequency off, 2^31 positions 2^-22 of a turn at most (added to the tolerance by
    comparing with the table's own frequencies)."""
    import gated_deltanet_linear_step_gb300 as g

    r = 128
    turns = g.gdn_rope_turns(r, base=500000.0, device=cuda_device, **scaling)
    t = [int(x) for x in turns.cpu().numpy().view(np.uint64)]
    pos = [0, 1, -1, 4095, 1 << 20, (1 << 24) + 1, 123456789, 2 ** 31 - 1, -2 ** 31]
    q = values((1, 1, len(pos), 2, r), "fp32", cuda_device, 5)
    out = torch.empty_like(q)
    g.gdn_rope(q, None, turns, out, None, positions=torch.tensor([pos], dtype=torch.int32, device=cuda_device), interleaved=interleaved)
    for i, p in enumerate(pos):  # exact integer arithmetic for the angle
        f = np.array([((p * x) % 2 ** 64) / 2.0 ** 64 for x in t]) * 2 * np.pi
        check(q[:, :, i:i + 1], out[:, :, i:i + 1], [[1]], f, "fp32", interleaved)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_angles_against_exact_ones(cuda_device, base):
    """Cosine and sine of positions up to the ends of int32 against angles with 50 digits. Tolerance: the table's 2^-53 of a turn for each position, 2^-28 of a
    turn for the angle's rounding (30 bits to 24) and 2^-32 for its cut, and 2^-22 for cosine, sine and the products with 1 and 0."""
    import gated_deltanet_linear_step_gb300 as g

    r, pos = 128, [0, 1, -1, 12345, 2 ** 24 + 1, 1000000007, -1234567890, 2 ** 31 - 1, -2 ** 31]
    x = torch.zeros((1, 1, len(pos), 1, r), device=cuda_device)
    x[..., :r // 2] = 1.0
    out = torch.empty_like(x)
    g.gdn_rope(x, None, g.gdn_rope_turns(r, base=base, device=cuda_device), out, None, positions=torch.tensor([pos], dtype=torch.int32, device=cuda_device))
    got = host(out)[0, 0, :, 0]
    for t, p in enumerate(pos):
        part = np.array([float(p * w % 1) for w in exact_turns(r, base)]) * 2 * np.pi
        tol = 2 * np.pi * (abs(p) * 2.0 ** -53 + 2.0 ** -28 + 2.0 ** -32) + 2.0 ** -22
        assert np.abs(got[t, :r // 2] - np.cos(part)).max() <= tol and np.abs(got[t, r // 2:] - np.sin(part)).max() <= tol, p


@pytest.mark.parametrize("dtype,r,interleaved", [("bf16", 128, False), ("fp16", 60, False), ("fp32", 128, True)])
def test_one_projections_output_in_place(cuda_device, dtype, r, interleaved):
    """Queries, keys and values of a token next to each other: turned where they lie, values and rows past the window untouched."""
    import gated_deltanet_linear_step_gb300 as g

    B, T, Hq, Hk, D = 3, 11, 6, 2, 128
    x = values((B, 1, T, Hq + 2 * Hk, D), dtype, cuda_device, 3)
    n = [11, 0, 4]
    start = torch.tensor([5, 6, 1000], dtype=torch.int32, device=cuda_device)
    turns = g.gdn_rope_turns(r, device=cuda_device)
    y = x.clone()
    q, k = y[..., :Hq, :], y[..., Hq:Hq + Hk, :]
    g.gdn_rope(q, k, turns, q, k, start=start, seq_len=torch.tensor(n, dtype=torch.int32, device=cuda_device), interleaved=interleaved)
    valid = np.arange(T)[None] < np.array(n)[:, None]
    pos = start.cpu().numpy()[:, None] + np.arange(T)
    check(x[..., :Hq + Hk, :], y[..., :Hq + Hk, :], pos, O.rope_frequencies(r), dtype, interleaved, valid=valid)
    assert torch.equal(y[..., Hq + Hk:, :], x[..., Hq + Hk:, :])
    for b in range(B):
        assert torch.equal(y[b, :, n[b]:], x[b, :, n[b]:]), "a row past the window changed"
    dense = torch.empty(B, 1, T, Hq, D, dtype=TYPES[dtype], device=cuda_device)  # and out of it into a dense one
    g.gdn_rope(x[..., :Hq, :], None, turns, dense, None, start=start, interleaved=interleaved)
    assert torch.equal(dense[0], q[0])


def test_dims_that_do_not_turn_may_hold_anything(cuda_device):
    import gated_deltanet_linear_step_gb300 as g

    for interleaved in (False, True):
        q = values((1, 1, 4, 3, 64), "fp32", cuda_device, 6)
        q[..., 22:][..., ::2], q[..., 22:][..., 1::2] = float("nan"), float("inf")
        out = torch.zeros_like(q)
        g.gdn_rope(q, None, g.gdn_rope_turns(22, device=cuda_device), out, None, interleaved=interleaved,
                   start=torch.zeros(1, dtype=torch.int32, device=cuda_device))
        assert torch.isfinite(out[..., :22]).all()
        assert torch.equal(out[..., 22:].view(torch.int32), q[..., 22:].view(torch.int32))


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(cuda_device, interleaved):
    """<g, rope(x)> has the gradient rope^T(g): against differences of the fp64 restatement, and <rope(x), g> = <x, rope^T(g)>."""
    import gated_deltanet_linear_step_gb300 as g

    r, D = 12, 16
    x, dy = (values((1, 1, 3, 2, D), "fp32", cuda_device, s) for s in (7, 8))
    turns = g.gdn_rope_turns(r, device=cuda_device)
    pos = torch.tensor([[0, 17, 4000]], dtype=torch.int32, device=cuda_device)
    dx, y = torch.empty_like(x), torch.empty_like(x)
    g.gdn_rope(dy, None, turns, dx, None, positions=pos, interleaved=interleaved, inverse=True, gain=1.5)
    g.gdn_rope(x, None, turns, y, None, positions=pos, interleaved=interleaved, gain=1.5)
    f, h = O.rope_frequencies(r), 1e-3
    xh, dyh = host(x), host(dy)
    num = np.zeros_like(xh)
    for i in np.ndindex(xh.shape):
        e = np.zeros_like(xh)
        e[i] = h
        p = pos.cpu().numpy()
        num[i] = (dyh * (O.rope(xh + e, p[:, None], f, interleaved, gain=1.5) - O.rope(xh - e, p[:, None], f, interleaved, gain=1.5))).sum() / (2 * h)
    assert np.abs(host(dx) - num).max() <= 1e-5 * np.abs(dyh).max()  # (linear: differences are exact but for fp64)
    a, b = float((y.double() * dy.double()).sum()), float((x.double() * dx.double()).sum())
    assert abs(a - b) <= 1e-5 * float(y.double().abs().sum() * dy.double().abs().max())


def test_graph_and_other_stream(cuda_device):
    import gated_deltanet_linear_step_gb300 as g

    q, k = (values((4, 1, 3, h, 128), "bf16", cuda_device, h) for h in (8, 2))
    turns = g.gdn_rope_turns(128, device=cuda_device)
    start = torch.tensor([0, 5, 9, 100], dtype=torch.int32, device=cuda_device)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.gdn_rope(q, k, turns, qo, ko, start=start)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gdn_rope(q, k, turns, qo, ko, start=start)
    for i in range(2):
        start += 7 * i
        graph.replay()
        pos = start.cpu().numpy()[:, None] + np.arange(3)
        check(q, qo, pos, O.rope_frequencies(128), "bf16")
        check(k, ko, pos, O.rope_frequencies(128), "bf16")


def test_binding_refuses(cuda_device):
    import gated_deltanet_linear_step_gb300 as g

    q = torch.zeros(2, 1, 3, 4, 64, device=cuda_device)
    turns = g.gdn_rope_turns(64, device=cuda_device)
    st = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    bad = [
        lambda: g.gdn_rope(q, None, turns, q[:1], None, start=st),
        lambda: g.gdn_rope(q, q, turns, q, None, start=st),
        lambda: g.gdn_rope(q, None, turns, q, None),
        lambda: g.gdn_rope(q, None, turns, q, None, start=st, positions=st),
        lambda: g.gdn_rope(q, None, turns.int(), q, None, start=st),
        lambda: g.gdn_rope(q, None, turns, q.transpose(2, 3), None, start=st),
        lambda: g.gdn_rope(q[..., ::2], None, turns[:16], q[..., :32], None, start=st),
        lambda: g.gdn_rope(q, None, turns, torch.zeros(2, 1, 4, 4, 64, device=cuda_device)[:, :, :3], None, start=st),
        lambda: g.gdn_rope(q, None, turns, q.bfloat16(), None, start=st),
        lambda: g.gdn_rope(q, None, turns.cpu(), q, None, start=st),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(g.GdnError):
        g.gdn_rope(q, None, g.gdn_rope_turns(66, device=cuda_device), q, None, start=st)
