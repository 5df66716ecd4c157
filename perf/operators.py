"""Cases of the operators that stand beside the decode step in a hybrid model: the 4-bit key/value
cache (written and read back), attention over it, and the log probabilities that decide a verify window.

``own`` false: the operators in their plain form (elementary torch operations). ``own`` true: the calls
that a user makes of this package. Both run on what ``prepare`` gives.

The 4-bit cache. A block of 16 values along the head dimension is 16 e2m1 codes (8 bytes, the even value
in the low nibble) and one scale byte b that stands for the fp16 number with the bits b << 7. A page
holds, per kv head, P tokens: [K codes | K scales | V codes | V scales], token by token; block i of token
row r of a page is stored at block i ^ ((8 (r & 1) + 4 (r >> 2 & 1)) & (D/16 - 1)). The cache is
[layers][pages][kv heads][bytes], and block_table[b] lists the pages of sequence b in order.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # halfway between neighbouring e2m1 magnitudes
MAX_SCALE = 10240.0


# ------------------------------------------------------------------ the cases --
def listed():
    return [
        # a decode step of a batch: every sequence appends one token to a layer's cache
        dict(name="append, one token x 64", op="append", dtype="bf16", B=64, L=1, T=1, Hkv=4, D=128, P=64, ctx=8192, ragged=False),
        # a prompt chunk of several sequences, four layers' caches
        dict(name="append, prompts", op="append", dtype="bf16", B=16, L=4, T=1024, Hkv=8, D=128, P=64, ctx=2048, ragged=True),
        # a cached prefix read back in full, e.g. to hand it to another program; odd lengths
        dict(name="read, ragged prefixes", op="read", dtype="fp16", B=5, L=2, T=5001, Hkv=4, D=64, P=16, ctx=0, ragged=True),
        # one conversation, single tokens: latency counts
        dict(name="attention, one short", op="attention", dtype="fp32", B=1, L=1, T=1, Hq=20, Hkv=4, D=128, P=64, ctx=500, ragged=False),
        # ordinary batched decoding at mixed lengths
        dict(name="attention, mixed batch", op="attention", dtype="bf16", B=64, L=1, T=1, Hq=20, Hkv=4, D=128, P=64, ctx=8192, ragged=True),
        # few sequences over a long document
        dict(name="attention, long document", op="attention", dtype="bf16", B=4, L=1, T=1, Hq=16, Hkv=2, D=256, P=64, ctx=131000, ragged=False),
        # a full machine: many long sequences
        dict(name="attention, full batch", op="attention", dtype="fp16", B=64, L=1, T=1, Hq=32, Hkv=8, D=128, P=128, ctx=16384, ragged=False),
        # a speculative verify window of mixed lengths in the framework's own type
        dict(name="attention, verify window", op="attention", dtype="fp32", B=16, L=2, T=8, Hq=20, Hkv=4, D=128, P=32, ctx=4096, ragged=True),
        # a prompt chunk behind a cached prefix
        dict(name="attention, prompt chunk", op="attention", dtype="bf16", B=2, L=1, T=1024, Hq=32, Hkv=8, D=128, P=64, ctx=8000, ragged=False),
        # one sequence's next token: latency counts
        dict(name="logprobs, one row", op="logprobs", dtype="fp32", N=1, V=131072, K=8, masked=0.0),
        # a verify window's rows, an odd vocabulary, a grammar's mask over part of it
        dict(name="logprobs, verify rows", op="logprobs", dtype="fp32", N=128, V=200001, K=20, masked=0.3),
        # scoring prompts
        dict(name="logprobs, prompt rows", op="logprobs", dtype="bf16", N=2048, V=131072, K=4, masked=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "read", "attention", "attention", "attention", "logprobs"))
    dtype = rng.choice(("fp32", "fp16", "bf16"))
    if op == "logprobs":
        V = _log(rng, 1000, 260000)
        return dict(op=op, dtype=dtype, N=_log(rng, 1, min(2048, 100_000_000 // V)), V=V, K=rng.randint(1, 32), masked=rng.choice((0.0, 0.5, 0.99)))
    c = dict(op=op, dtype=dtype, L=rng.choice((1, 1, 2, 3)), Hkv=rng.choice((1, 2, 3, 4, 8)), D=rng.choice((64, 128, 256)),
             P=rng.choice((16, 32, 64, 128)), ragged=rng.random() < 0.6)
    row = c["L"] * c["Hkv"] * c["D"]
    if op != "attention":
        c["T"] = _log(rng, 1, 4096)
        c["B"] = _log(rng, 1, max(1, min(64, 60_000_000 // (c["T"] * row))))
        c["ctx"] = _log(rng, 1, 2048) if op == "append" else 0
        return c
    c["Hq"] = c["Hkv"] * rng.choice((1, 2, 4, 5, 8, 16))
    c["T"] = rng.choice((1, 1, 1, rng.randint(2, 8), _log(rng, 9, 1024)))
    c["ctx"] = _log(rng, 1, 100_000 if c["T"] <= 8 else 8000)
    c["B"] = _log(rng, 1, max(1, min(64, 400_000_000 // ((c["ctx"] + c["T"]) * row), 60_000_000_000 // (c["T"] * (c["ctx"] + c["T"]) * c["L"] * c["Hq"] * c["D"]))))
    return c


# ------------------------------------------------------------------- the data --
def _lengths(case):
    """Start and valid window length of every sequence, from the sizes alone."""
    B, T, ctx = case["B"], case["T"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B, [T] * B
    g = torch.Generator().manual_seed(1000 * B + T + ctx)
    u = torch.rand(B, 2, generator=g).tolist()
    return [int(a * (ctx + 1)) for a, _ in u], [1 + int(b * T) for _, b in u]


def _normal(shape, g, dtype):
    """Values as projected keys, values and queries have them: some channels several times the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    gain = torch.exp(0.7 * torch.randn(shape[-2:], generator=g, device="cuda"))
    return (x * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "logprobs":
        N, V = case["N"], case["V"]
        x = torch.randn(N, V, generator=g, device="cuda") * 2.5
        tokens = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        x[torch.arange(N, device="cuda"), tokens.long()] += 8.0 * torch.rand(N, generator=g, device="cuda")
        if case["masked"]:
            x.masked_fill_(torch.rand(N, V, generator=g, device="cuda") < case["masked"], float("-inf"))
        f = dict(device="cuda", dtype=torch.float32)
        return dict(case=case, logits=x.to(dtype), tokens=tokens, logprob=torch.empty(N, **f), entropy=torch.empty(N, **f),
                    top_ids=torch.empty(N, case["K"], device="cuda", dtype=torch.int32), top_logprobs=torch.empty(N, case["K"], **f))
    B, L, T, Hkv, D, P = (case[k] for k in ("B", "L", "T", "Hkv", "D", "P"))
    start, n = _lengths(case)
    maxp = max((s + T + P - 1) // P for s in start)
    pages = B * maxp
    head = 2 * P * (D // 2 + D // 16)
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(B, maxp)
    cache = torch.randint(0, 256, (L, pages, Hkv * head), generator=g, device="cuda", dtype=torch.uint8)
    s = dict(case=case, cache=cache, table=table, start=torch.tensor(start, dtype=torch.int32, device="cuda"),
             n=torch.tensor(n, dtype=torch.int32, device="cuda") if case["ragged"] else None)
    if case["op"] != "append":  # what was there before, quantised sequence by sequence
        view = cache.view(L, pages, Hkv, head)
        for b in range(B):
            used = start[b] + n[b]
            np_ = (used + P - 1) // P
            for part in range(2):
                x = _normal((np_, P, L, Hkv, D), g, torch.float32).permute(2, 0, 3, 1, 4)  # [L, pages, Hkv, P, D]
                codes, scales = _pack(x, P, D)
                at = part * head // 2
                view[:, table[b, :np_].long(), :, at:at + P * D // 2] = codes.reshape(L, np_, Hkv, -1)
                view[:, table[b, :np_].long(), :, at + P * D // 2:at + head // 2] = scales.reshape(L, np_, Hkv, -1)
    if case["op"] == "attention":
        s["q"] = _normal((B, L, T, case["Hq"], D), g, dtype)
        s["out"] = torch.zeros_like(s["q"])
        if own:
            import gated_deltanet_linear_step_gb300 as gdn

            bytes_ = gdn.gdn_kv4_attention_workspace_size(B, L, T, case["Hq"], Hkv, D)
            s["workspace"] = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
        return s
    s["k_out"] = torch.zeros((B, L, T, Hkv, D), dtype=dtype, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    if case["op"] == "append":
        s["k"] = _normal((B, L, T, Hkv, D), g, dtype)
        s["v"] = _normal((B, L, T, Hkv, D), g, dtype)
    return s


# ------------------------------------------------------------- the plain form --
def _quantise(x):
    """Codes (0..15) and scale bytes of fp32 values whose last dimension is a multiple of 16."""
    x = torch.nan_to_num(x, nan=0.0).clamp(-61440.0, 61440.0).unflatten(-1, (-1, 16))
    a = x.abs().amax(-1) / torch.full((), 6.0, device=x.device)
    up = torch.clamp(torch.floor(torch.log2(a.clamp_min(2.0 ** -14))), -14, 13)
    up = up + (a >= torch.exp2(up + 1)).float() - (a < torch.exp2(up)).float() * (up > -14).float()  # log2 may round over a border
    s = (torch.round(a * torch.exp2(3 - up)) * torch.exp2(up - 3)).clamp_max(MAX_SCALE)
    byte = s.to(torch.float16).view(torch.int16) >> 7
    y = x / torch.where(s > 0, s, torch.full_like(s, float("inf"))).unsqueeze(-1)
    m = y.abs()
    even = torch.tensor(MIDS, device=x.device)
    code = torch.bucketize(m, even)                       # ties go down here ...
    code = code + ((m == even[code.clamp_max(6)]) & (code % 2 == 1)).to(code.dtype)  # ... and to the even code
    code = torch.where(y < 0, code + 8, code)
    return code.flatten(-2).to(torch.uint8), byte.to(torch.uint8)


def _block_order(P, D, device):
    """Where block i of token row r lies: [P, D/16]."""
    r = torch.arange(P, device=device).unsqueeze(1)
    return torch.arange(D // 16, device=device) ^ ((8 * (r & 1) + 4 * ((r >> 2) & 1)) & (D // 16 - 1))


def _pack(x, P, D):
    """Code bytes and scale bytes of whole pages [..., P, D], in the order a page holds them."""
    codes, scales = _quantise(x)
    byte = codes[..., 0::2] | (codes[..., 1::2] << 4)
    blocks = byte.unflatten(-1, (D // 16, 8))
    order = _block_order(P, D, x.device)
    return torch.gather(blocks, -2, order.unsqueeze(-1).expand(blocks.shape)), scales


def _values(s, part):
    """The cache's keys (part 0) or values (part 1) of every sequence, fp32 [B, L, Hkv, S, D]."""
    c = s["case"]
    L, Hkv, D, P = (c[k] for k in ("L", "Hkv", "D", "P"))
    head = 2 * P * (D // 2 + D // 16)
    at = part * head // 2
    pages = s["cache"].view(L, -1, Hkv, head)[:, s["table"].clamp_min(0).long(), :, at:at + head // 2]  # [L, B, maxp, Hkv, bytes]
    blocks = pages[..., :P * D // 2].unflatten(-1, (P, D // 16, 8))
    order = _block_order(P, D, blocks.device)
    blocks = torch.gather(blocks, -2, order.unsqueeze(-1).expand(blocks.shape))
    codes = torch.stack((blocks & 15, blocks >> 4), -1).flatten(-2)                       # [..., P, D/16, 16]
    scale = (pages[..., P * D // 2:].to(torch.int16) << 7).view(torch.float16).float().unflatten(-1, (P, D // 16))
    v = torch.tensor(E2M1, device=codes.device)[codes.int()] * scale.unsqueeze(-1)
    return v.flatten(-2).permute(1, 0, 3, 2, 4, 5).flatten(3, 4)


def _tokens(s):
    """Positions [B, T] of the window's tokens and whether each is valid."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    n = s["n"] if s["n"] is not None else torch.full((c["B"],), c["T"], device="cuda")
    return s["start"].unsqueeze(1).long() + t, t < n.unsqueeze(1)


def _plain_append(s):
    c = s["case"]
    L, Hkv, D, P = (c[k] for k in ("L", "Hkv", "D", "P"))
    head = 2 * P * (D // 2 + D // 16)
    pos, valid = _tokens(s)
    b, t = valid.nonzero(as_tuple=True)
    row = pos[b, t] % P
    page = s["table"][b, pos[b, t] // P].long()
    view = s["cache"].view(L, -1, Hkv, head)
    for part, x in enumerate((s["k"], s["v"])):
        codes, scales = _quantise(x[b, :, t].float())                                     # [n, L, Hkv, D]
        blocks = (codes[..., 0::2] | (codes[..., 1::2] << 4)).unflatten(-1, (D // 16, 8))
        order = _block_order(P, D, x.device)[row][:, None, None, :, None]
        blocks = torch.gather(blocks, -2, order.expand(blocks.shape)).flatten(-2)
        at = part * head // 2
        li = torch.arange(L, device="cuda")[None, :, None, None]
        hi = torch.arange(Hkv, device="cuda")[None, None, :, None]
        pi, ri = page[:, None, None, None], row[:, None, None, None]
        view[li, pi, hi, at + ri * (D // 2) + torch.arange(D // 2, device="cuda")] = blocks
        view[li, pi, hi, at + P * D // 2 + ri * (D // 16) + torch.arange(D // 16, device="cuda")] = scales


def _plain_read(s):
    c = s["case"]
    L, Hkv, D, P = (c[k] for k in ("L", "Hkv", "D", "P"))
    head = 2 * P * (D // 2 + D // 16)
    pos, valid = _tokens(s)
    b, t = valid.nonzero(as_tuple=True)
    row = pos[b, t] % P
    view = s["cache"].view(L, -1, Hkv, head)
    li = torch.arange(L, device="cuda")[None, :, None, None]
    hi = torch.arange(Hkv, device="cuda")[None, None, :, None]
    pi, ri = s["table"][b, pos[b, t] // P].long()[:, None, None, None], row[:, None, None, None]
    order = _block_order(P, D, row.device)[row][:, None, None, :, None]
    for part, name in enumerate(("k_out", "v_out")):
        at = part * head // 2
        blocks = view[li, pi, hi, at + ri * (D // 2) + torch.arange(D // 2, device="cuda")].unflatten(-1, (D // 16, 8))
        blocks = torch.gather(blocks, -2, order.expand(blocks.shape))                      # [n, L, Hkv, D/16, 8]
        codes = torch.stack((blocks & 15, blocks >> 4), -1).flatten(-2)
        byte = view[li, pi, hi, at + P * D // 2 + ri * (D // 16) + torch.arange(D // 16, device="cuda")]
        scale = (byte.to(torch.int16) << 7).view(torch.float16).float()
        x = torch.tensor(E2M1, device="cuda")[codes.int()] * scale.unsqueeze(-1)
        s[name][b, :, t] = x.flatten(-2).to(s[name].dtype)
    return s["k_out"], s["v_out"]


def _plain_attention(s):
    c = s["case"]
    B, L, T, Hq, Hkv, D = (c[k] for k in ("B", "L", "T", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    pos, valid = _tokens(s)
    last = torch.where(valid, pos, -1).amax(1)
    k = _values(s, 0)
    q = s["q"].float().unflatten(3, (Hkv, G)).permute(0, 1, 3, 4, 2, 5).reshape(B, L, Hkv, G * T, D)
    x = torch.matmul(q, k.transpose(-1, -2)) * D ** -0.5                                 # [B, L, Hkv, G T, S]
    j = torch.arange(k.shape[3], device="cuda")
    del k
    see = (j <= pos.unsqueeze(-1)).unsqueeze(1).expand(B, G, T, -1).reshape(B, 1, 1, G * T, -1)
    x = torch.where(see, x, float("-inf"))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _values(s, 1)
    v = torch.where((j <= last.unsqueeze(-1))[:, None, None, :, None], v, 0.0)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    o = o.view(B, L, Hkv, G, T, D).permute(0, 1, 4, 2, 3, 5).reshape(B, L, T, Hq, D).to(s["out"].dtype)
    s["out"].copy_(torch.where(valid[:, None, :, None, None], o, s["out"]))
    return s["out"]


def _plain_logprobs(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    z = x - m
    p = torch.exp(z)
    total = p.sum(-1, keepdim=True)
    log_total = torch.log(total)
    logprob = torch.gather(z, 1, s["tokens"].long().unsqueeze(1)) - log_total
    entropy = log_total - torch.where(p > 0, p * z, 0.0).sum(-1, keepdim=True) / total
    bits = x.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32 - torch.arange(x.shape[1], device="cuda")  # ties: the lowest index
    ids = torch.topk(key, s["case"]["K"], dim=-1).indices
    return logprob.squeeze(1), entropy.squeeze(1), ids.int(), torch.gather(z, 1, ids) - log_total


# ---------------------------------------------------------------------- a pass --
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "append":
            _plain_append(s)
            return _plain_read(s)
        return {"read": _plain_read, "attention": _plain_attention, "logprobs": _plain_logprobs}[op](s)
    import gated_deltanet_linear_step_gb300 as gdn

    if op == "logprobs":
        gdn.gdn_logprobs(s["logits"], s["tokens"], s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"])
        return s["logprob"], s["entropy"], s["top_ids"], s["top_logprobs"]
    P = s["case"]["P"]
    if op == "attention":
        gdn.gdn_kv4_attention(s["q"], s["cache"], s["table"], s["start"], s["out"], s["workspace"], P, s["case"]["Hkv"], seq_len=s["n"])
        return s["out"]
    if op == "append":
        gdn.gdn_kv4_append(s["k"], s["v"], s["cache"], s["table"], s["start"], P, seq_len=s["n"])
    gdn.gdn_kv4_read(s["cache"], s["table"], s["start"], s["k_out"], s["v_out"], P, seq_len=s["n"])
    return s["k_out"], s["v_out"]


def work(case):
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "logprobs":
        N, V, K = case["N"], case["V"], case["K"]
        return {"bytes": N * V * size + N * (12 + 8 * K), "flops": 6 * N * V}
    L, Hkv, D = case["L"], case["Hkv"], case["D"]
    start, n = _lengths(case)
    row = 2 * L * Hkv * D                                      # key and value elements of a token
    if case["op"] == "read":
        return {"bytes": sum(n) * row * (0.5625 + size), "flops": sum(n) * row * 2}
    if case["op"] == "append":                               # in, quantised, read back, out
        return {"bytes": sum(n) * row * (2 * size + 2 * 0.5625), "flops": sum(n) * row * 6}
    Hq = case["Hq"]
    seen = sum(m * a + m * (m + 1) // 2 for a, m in zip(start, n))
    return {"bytes": sum(a + m for a, m in zip(start, n)) * row * 0.5625 + 2 * sum(n) * L * Hq * D * size, "flops": 4 * D * L * Hq * seen}


# ------------------------------------------------------------- in 64 bits --
def _exact_quantised(x):
    """Each value of x (float64) as the 4-bit cache holds it, from the definition."""
    x = torch.where(x.isnan(), 0.0, x).clamp(-61440, 61440).unflatten(-1, (-1, 16))
    grid = [m * 2.0 ** -17 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-14, 14) for m in range(8)]
    grid = [v for v in grid if v <= MAX_SCALE]
    scale = _nearest(x.abs().amax(-1, keepdim=True) / 6, torch.tensor(grid, dtype=torch.float64, device=x.device))
    y = torch.where(scale > 0, x / scale.clamp_min(2.0 ** -30), 0.0)
    code = _nearest(y.abs(), torch.tensor(E2M1[:8], dtype=torch.float64, device=x.device))
    return (torch.sign(y) * code * scale).flatten(-2)


def _nearest(a, grid):
    """The entry of a rising grid that is nearest to a >= 0, at half way the one with the even place."""
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return grid[torch.where(up, hi, hi - 1)]


def _exact_rows(s, b, count):
    """Keys and values of the first `count` tokens of sequence b: two float64 [L, Hkv, count, D]."""
    c = s["case"]
    L, Hkv, D, P = (c[k] for k in ("L", "Hkv", "D", "P"))
    np_ = (count + P - 1) // P
    lut = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    got = []
    pages = s["cache"].view(L, -1, Hkv, 2, P * (D // 2 + D // 16)).index_select(1, s["table"][b, :np_].long())
    for part in range(2):
        x = pages[:, :, :, part].transpose(1, 2)                                           # [L, Hkv, np, bytes]
        code = x[..., :P * D // 2].reshape(L, Hkv, np_ * P, D // 16, 8)[:, :, :count]
        b8 = x[..., P * D // 2:].reshape(L, Hkv, np_ * P, D // 16)[:, :, :count].double()
        e, m = torch.floor(b8 / 8), b8 % 8
        scale = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 15), m * 2.0 ** -17)
        row = torch.arange(count, device="cuda") % P
        turn = (8 * (row & 1) + 4 * ((row >> 2) & 1)) & (D // 16 - 1)
        rows = torch.arange(count, device="cuda")
        v = torch.empty(L, Hkv, count, D // 16, 16, dtype=torch.float64, device="cuda")
        for i in range(D // 16):
            at = code[:, :, rows, i ^ turn].long()
            v[:, :, :, i, 0::2], v[:, :, :, i, 1::2] = lut[at % 16], lut[at // 16]
        got.append((v * scale.unsqueeze(-1)).flatten(-2))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        out = [], [], [], []
        for i in range(case["N"]):
            x = s["logits"][i].double()
            lse = torch.logsumexp(x, 0)
            p = torch.softmax(x, 0)
            out[0].append(x[int(s["tokens"][i])] - lse)
            out[1].append(-torch.special.xlogy(p, p).sum())
            ids = torch.sort(x, descending=True, stable=True).indices[:case["K"]]
            out[2].append(ids.int())
            out[3].append(x[ids] - lse)
        return tuple(torch.stack(o) for o in out)
    start, n = _lengths(case)
    B, L, T, Hkv, D = (case[k] for k in ("B", "L", "T", "Hkv", "D"))
    if case["op"] == "attention":
        G = case["Hq"] // Hkv
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            k, v = _exact_rows(s, b, start[b] + n[b])
            hidden = torch.arange(start[b] + n[b], device="cuda") > start[b] + torch.arange(n[b], device="cuda").unsqueeze(1)
            for h in range(case["Hq"]):
                x = s["q"][b, :, :n[b], h].double() @ k[:, h // G].transpose(-1, -2) / math.sqrt(D)
                o[b, :, :n[b], h] = torch.softmax(x.masked_fill(hidden, float("-inf")), -1) @ v[:, h // G]
        return o
    k = torch.zeros((B, L, T, Hkv, D), dtype=torch.float64, device="cuda")
    v = torch.zeros_like(k)
    for b in range(B):
        if case["op"] == "append":
            k[b, :, :n[b]], v[b, :, :n[b]] = _exact_quantised(s["k"][b, :, :n[b]].double()), _exact_quantised(s["v"][b, :, :n[b]].double())
        else:
            a, c = _exact_rows(s, b, n[b])
            k[b, :, :n[b]], v[b, :, :n[b]] = a.transpose(1, 2), c.transpose(1, 2)
    return k, v
