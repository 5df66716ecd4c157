"""Ends of the ranges of the prompt operators: rows and pages behind 2^31 elements and 2^32 bytes, calls on two streams at once, windows whose rows
past their length hold anything."""
import numpy as np
import pytest
import torch

from oracle import operators as O
from tests import test_gpu_prompt as prompt, test_gpu_rope as rope
from tests.test_gpu_kv4 import host, values
from tests.test_gpu_shared_prefix import Shared

pytestmark = pytest.mark.gpu


def test_rows_beyond_32_bit_offsets(cuda_device):
    """2.3e9 elements of queries in 1000 sequences of 70 tokens; the last three are checked."""
    import gated_deltanet_linear_step_gb300 as g

    n, B, Hq, H, D = 70, 1000, 256, 2, 128
    N = n * B
    q = values((n, Hq, D), "bf16", cuda_device, 1).repeat(B, 1, 1)
    k, v = (values((N, H, D), "bf16", cuda_device, s) for s in (2, 3))
    turns, f = g.gdn_rope_turns(64, device=cuda_device), O.rope_frequencies(64)
    pos = torch.arange(N, dtype=torch.int32, device=cuda_device).view(1, N)
    was = q[-3 * n:].clone()
    g.gdn_rope(q[None, None], None, turns, q[None, None], None, positions=pos)
    rope.check(was[None, None], q[None, None, -3 * n:], np.arange(N - 3 * n, N), f, "bf16")
    offsets = [i * n for i in range(B + 1)]
    out = prompt.attend(q, k, v, offsets)
    tail = slice(N - 3 * n, None)
    prompt.check(q[tail], k[tail], v[tail], out[tail], [0, n, 2 * n, 3 * n], "bf16", heads=(0, 1, 127, 128, 255))
    assert g.gdn_read_device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_pages_beyond_32_bit_offsets(cuda_device, D):
    """A cache of 4.5 GiB whose last pages are the prefix of 40 rows."""
    H, page, n, B = 8, 256, 600, 10
    c = Shared(cuda_device, [n], [0, B], B, 1, H, D, page, n)
    pb = c.g.gdn_kv4_page_bytes(H, D, page)
    pages = (9 << 29) // pb
    c.table = (pages - 1 - c.table).astype(np.int32)
    c.t_table = torch.from_numpy(c.table).to(cuda_device)
    c.t_prefix, c.t_own = c.t_table[:1].contiguous(), c.t_table[1:].contiguous()
    c.t_cache = torch.zeros((1, pages, pb), dtype=torch.uint8, device=cuda_device)
    k, v = (values((B + 1, 1, n, H, D), "fp16", cuda_device, s) for s in (4, 5))
    start = [3 * b for b in range(B)]
    c.fill(k, v, [s + 1 for s in start], B)
    q = values((B, 1, 1, 4 * H, D), "fp16", cuda_device, 6)
    out = c.shared(q, start)
    assert c.g.gdn_read_device_error() == 0
    # (the restatement reads the used pages alone)
    used = np.arange(pages - 1 - int((pages - 1 - c.table).max()), pages)
    whole, c.t_cache, c.table = c.t_cache, c.t_cache[:, used[0]:].contiguous(), c.table - used[0]
    c.check(q, out, start, None, "fp16", rows={(0, 0, 0), (B - 1, 0, H - 1), (4, 0, 3)})
    del whole


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_borders_that_fall_leave_every_row(cuda_device, dtype):
    """Falling borders may name the same rows any number of times: the call reports them and does nothing, however many there are."""
    import gated_deltanet_linear_step_gb300 as g

    q = values((300, 2, 64), dtype, cuda_device, 16)
    for off in ([30, 20, 64], [0, 300, 0, 300], [0, 300] * 100, [0, 10, 9] + [300] * 200):
        assert (prompt.attend(q, q, q, off) == 7.0).all() and g.gdn_read_device_error() == 4, off[:4]
    prompt.check(q, q, q, prompt.attend(q, q, q, [0, 10, 10, 300]), [0, 10, 10, 300], dtype)
    assert g.gdn_read_device_error() == 0


def test_thousands_of_short_prompts(cuda_device):
    """Sequences of 0 to 3 tokens and a longer one among them; four times as many take some four times as long, not sixteen."""
    import gated_deltanet_linear_step_gb300 as g

    best = {}
    for B in (5000, 20000):
        lens = [(7 * i) % 4 for i in range(B)]
        lens[B // 2] = 700
        off = prompt.packed(lens)
        q, k, v = (values((off[-1], h, 64), "bf16", cuda_device, 17 + i) for i, h in enumerate((4, 2, 2)))
        out = prompt.attend(q, k, v, off)
        if B == 5000:
            prompt.check(q, k, v, out, off, "bf16", heads=[1, 2])
        ws = torch.empty(g.gdn_prompt_attention_workspace_size(B, off[-1], 4, 2, 64, q.dtype), dtype=torch.uint8, device=cuda_device)
        t_off, times = torch.tensor(off, dtype=torch.int32, device=cuda_device), []
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            g.gdn_prompt_attention(q, k, v, t_off, out, ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best[B] = min(times)
    assert best[20000] < 8 * best[5000], best
    assert g.gdn_read_device_error() == 0


def test_calls_on_two_streams_at_once(cuda_device):
    """Each stream has its own workspaces and outputs; every result has the bits that it has alone."""
    import gated_deltanet_linear_step_gb300 as g

    B, Hq, H, D, page, n = 30, 20, 4, 128, 32, 3000
    jobs = []
    for i in range(2):
        c = Shared(cuda_device, [n], [0, B], B, 1, H, D, page, 64, seed=i)
        k, v = (values((1, 1, n, H, D), "bf16", cuda_device, 7 + s + 10 * i) for s in (0, 1))
        c.g.gdn_kv4_append(k, v, c.t_cache, c.t_prefix, c.i32([0]), page)
        own = [values((B, 1, 64, H, D), "bf16", cuda_device, 9 + s + 10 * i) for s in (0, 1)]
        c.g.gdn_kv4_append(*own, c.t_cache, c.t_own, c.i32([0] * B), page)
        q = values((B, 1, 1, Hq, D), "bf16", cuda_device, 11 + 10 * i)
        p = [values((2000, h, D), "bf16", cuda_device, 12 + 10 * i + h) for h in (Hq, H, H)]
        jobs.append(dict(c=c, q=q, p=p, out=torch.empty_like(q), po=torch.empty_like(p[0]), start=c.i32([63] * B), lens=c.i32([n]), groups=c.i32([0, B]),
                         off=c.i32([0, 700, 2000]), stream=torch.cuda.Stream(),
                         ws=torch.empty(g.gdn_kv4_attention_shared_workspace_size(B, 1, 1, Hq, H, D), dtype=torch.uint8, device=cuda_device),
                         pw=torch.empty(g.gdn_prompt_attention_workspace_size(2, 2000, Hq, H, D, torch.bfloat16), dtype=torch.uint8, device=cuda_device)))

    def run(j):
        c = j["c"]
        g.gdn_prompt_attention(*j["p"], j["off"], j["po"], j["pw"])
        g.gdn_kv4_attention_shared(j["q"], c.t_cache, c.t_prefix, j["lens"], j["groups"], c.t_own, j["start"], j["out"], j["ws"], page, H)

    alone = []
    for j in jobs:
        run(j)
        torch.cuda.synchronize()
        alone.append((j["out"].clone(), j["po"].clone()))
    for _ in range(10):
        for j in jobs:
            j["out"].zero_(), j["po"].zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for j in jobs:
                with torch.cuda.stream(j["stream"]):
                    run(j)
        torch.cuda.synchronize()
        for j, (out, po) in zip(jobs, alone):
            assert torch.equal(j["out"], out) and torch.equal(j["po"], po)
    assert g.gdn_read_device_error() == 0


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp32", 128)])
def test_rows_past_a_windows_length_may_hold_anything(cuda_device, dtype, D):
    """NaN and infinities in queries past seq_len do not reach the others, which share the matrix products (in 16 bits they change no bit of them)."""
    B, T, H = 12, 4, 2
    c = Shared(cuda_device, [500, 0], [0, 7, B], B, 1, H, D, 16, 32)
    k, v = (values((B + 2, 1, 500, H, D), dtype, cuda_device, s) for s in (14, 15))
    c.fill(k, v, [28] * B, B)
    n = [(b * 3) % (T + 1) for b in range(B)]
    q = values((B, 1, T, 4 * H, D), dtype, cuda_device, 16)
    want = c.shared(q, [20] * B, n)
    for bad in (float("nan"), float("inf")):
        for b in range(B):
            q[b, :, n[b]:] = bad
        out = c.shared(q, [20] * B, n)
        c.check(q, out, [20] * B, n, dtype)
        if dtype != "fp32":
            assert torch.equal(torch.nan_to_num(out, nan=5.0), torch.nan_to_num(want, nan=5.0))
    assert c.g.gdn_read_device_error() == 0
    c.check(q, want, [20] * B, n, dtype)
