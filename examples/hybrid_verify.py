"""Speculative decoding of a small hybrid model: Gated DeltaNet layers and an attention layer over a 4-bit cache.

A window of T tokens per sequence (the last accepted token and T - 1 drafted ones) is verified at once:

  gdn_step_inputs, gdn_verify_window   the recurrent layers' outputs, their states only read
  gdn_kv4_append, gdn_kv4_attention    the attention layer: the window's keys and values are cached, then attended to
  gdn_logprobs                         the model's own next token after every token of the window
  gdn_verify_commit                    the recurrent states advance by the tokens that were kept

The cache needs no undoing: tokens that were not kept are overwritten by the next window, whose kv_start says
where. Weights are random; the drafts are the model's own greedy continuation with some tokens spoiled, so the program
can check that verification keeps exactly what greedy decoding would have produced.

    python examples/hybrid_verify.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_deltanet_linear_step_gb300 as gdn  # noqa: E402
from gated_deltanet_linear_step_gb300._binding import CONV_CHANNELS, D_CONV, HEAD_DIM, V_HEADS, VALUE_DIM  # noqa: E402


class HybridModel:
    """One recurrent layer, one attention layer, tied embeddings; random weights."""

    def __init__(self, batch, max_tokens, n_embd=256, vocab=2000, q_heads=8, kv_heads=2, head_dim=128, page=32, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.device = device

        def w(*shape, dtype=torch.float32):
            return (torch.randn(shape, generator=g, device=device) / math.sqrt(shape[-1])).to(dtype)

        self.E, self.B, self.Hq, self.Hkv, self.D, self.page = n_embd, batch, q_heads, kv_heads, head_dim, page
        self.emb = torch.randn(vocab, n_embd, generator=g, device=device)
        # recurrent layer
        self.w_qkv, self.w_gate = (w(1, n, n_embd, dtype=torch.bfloat16) for n in (CONV_CHANNELS, VALUE_DIM))
        self.w_alpha, self.w_beta = (w(1, V_HEADS, n_embd, dtype=torch.bfloat16) for _ in range(2))
        self.dt, self.ssm_a = torch.zeros(1, V_HEADS, device=device), -torch.ones(1, V_HEADS, device=device)
        self.conv_w, self.norm = 0.5 * torch.randn(1, CONV_CHANNELS, D_CONV, generator=g, device=device), torch.ones(1, HEAD_DIM, device=device)
        self.w_out = w(n_embd, VALUE_DIM)
        # attention layer
        self.w_q, self.w_k, self.w_v = (w(h * head_dim, n_embd) for h in (q_heads, kv_heads, kv_heads))
        self.w_o = w(n_embd, q_heads * head_dim)
        self.reset(max_tokens)

    def reset(self, max_tokens):
        f = dict(device=self.device)
        self.conv_state = torch.zeros(self.B, 1, CONV_CHANNELS, D_CONV - 1, **f)
        self.state = torch.zeros(self.B, 1, V_HEADS, HEAD_DIM, HEAD_DIM, **f)
        per_seq = -(-max_tokens // self.page)
        self.cache = torch.empty(1, self.B * per_seq, gdn.gdn_kv4_page_bytes(self.Hkv, self.D, self.page), dtype=torch.uint8, **f)
        self.table = torch.randperm(self.B * per_seq, **f).to(torch.int32).view(self.B, per_seq)
        self.kv_start = torch.zeros(self.B, dtype=torch.int32, **f)

    def window(self, tokens):
        """The model's next token after each token of the window [B][T], its log probability, and what commit() needs."""
        B, T = tokens.shape
        f = dict(device=self.device)
        x = self.emb[tokens.long()]
        # recurrent layer: y from the untouched state
        h = torch.nn.functional.rms_norm(x, (self.E,)).view(B, 1, T, self.E).contiguous()
        qkv, z = torch.empty(B, 1, T, CONV_CHANNELS, **f), torch.empty(B, 1, T, VALUE_DIM, **f)
        gate, beta = (torch.empty(B, 1, T, V_HEADS, **f) for _ in range(2))
        ws = torch.empty(gdn.gdn_in_proj_workspace_size(B, 1, T, self.E), dtype=torch.uint8, **f)
        gdn.gdn_step_inputs(h, self.w_qkv, self.w_gate, self.w_alpha, self.w_beta, self.dt, self.ssm_a, qkv, z, gate, beta, ws)
        y = torch.empty(B, 1, T, VALUE_DIM, **f)
        flags = gdn.FLAG_GATES_READY | gdn.FLAG_NO_STATE_WRITE
        gdn.gdn_decode_step_ex(qkv, z, gate, beta, self.dt, self.ssm_a, self.conv_w, self.norm, self.conv_state, self.state, y, flags=flags)
        x = x + (y.view(B, T, -1) @ self.w_out.T)
        # attention layer over the 4-bit cache
        h = torch.nn.functional.rms_norm(x, (self.E,))
        q = (h @ self.w_q.T).view(B, 1, T, self.Hq, self.D)
        k = (h @ self.w_k.T).view(B, 1, T, self.Hkv, self.D)
        v = (h @ self.w_v.T).view(B, 1, T, self.Hkv, self.D)
        gdn.gdn_kv4_append(k, v, self.cache, self.table, self.kv_start, self.page)
        ws = torch.empty(gdn.gdn_kv4_attention_workspace_size(B, 1, T, self.Hq, self.Hkv, self.D), dtype=torch.uint8, **f)
        o = torch.empty_like(q)
        gdn.gdn_kv4_attention(q, self.cache, self.table, self.kv_start, o, ws, self.page, self.Hkv)
        x = x + o.view(B, T, -1) @ self.w_o.T
        # the next token
        logits = torch.nn.functional.rms_norm(x, (self.E,)).view(B * T, self.E) @ self.emb.T
        top = torch.empty(B * T, 1, dtype=torch.int32, **f)
        top_lp, entropy = torch.empty(B * T, 1, **f), torch.empty(B * T, **f)
        gdn.gdn_logprobs(logits, entropy=entropy, top_ids=top, top_logprobs=top_lp)
        return top.view(B, T), top_lp.view(B, T), (qkv, gate, beta)

    def commit(self, seen, n_keep):
        """Keeps the first n_keep[b] tokens of the window."""
        qkv, gate, beta = seen
        flags = gdn.FLAG_GATES_READY | gdn.FLAG_NO_Y
        gdn.gdn_decode_step_ex(qkv, None, gate, beta, self.dt, self.ssm_a, self.conv_w, None, self.conv_state, self.state, None, seq_len=n_keep,
                               flags=flags)
        self.kv_start += n_keep


def greedy(model, first, steps):
    """Token by token: [B][steps + 1], `first` included."""
    out = [first]
    one = torch.ones_like(model.kv_start)
    for _ in range(steps):
        top, _, seen = model.window(out[-1].view(-1, 1))
        model.commit(seen, one)
        out.append(top[:, 0])
    return torch.stack(out, 1)


def speculate(model, first, drafts, steps, T):
    """The same by windows of T tokens. drafts(b, at) -> the T - 1 tokens guessed to follow position `at` of sequence b.
    Returns the tokens and how many windows it took."""
    out = [[int(t)] for t in first]
    windows = 0
    while min(len(o) for o in out) <= steps:
        window = torch.tensor([[o[-1]] + drafts(b, len(o) - 1)[:T - 1] for b, o in enumerate(out)], dtype=torch.int32, device=model.device)
        top, _, seen = model.window(window)
        # token i + 1 of the window is kept while it is what the model says after token i
        kept = (top[:, :-1] == window[:, 1:]).int().cumprod(1).sum(1)
        n_keep = (kept + 1).int()
        model.commit(seen, n_keep)
        for b, o in enumerate(out):
            o.extend(top[b, :int(n_keep[b])].tolist())
        windows += 1
    return torch.tensor([o[:steps + 1] for o in out], dtype=torch.int32, device=model.device), windows


def main(batch=4, steps=48, T=6):
    model = HybridModel(batch, max_tokens=steps + 2 * T + 2)
    first = torch.arange(batch, dtype=torch.int32, device=model.device) * 17 + 5
    want = greedy(model, first, steps)
    text = want.tolist()

    def drafts(b, at):
        guess = [text[b][min(at + 1 + i, steps)] for i in range(T - 1)]
        spoil = (3 * b + at) % T  # every window but some has a wrong token somewhere
        return [t if i != spoil else (t + 1) % 2000 for i, t in enumerate(guess)]

    model.reset(steps + 2 * T + 2)
    got, windows = speculate(model, first, drafts, steps, T)
    same = int((got == want).all(1).sum())
    print(f"{batch} sequences, {steps} tokens each: {windows} windows of {T} tokens instead of {steps} steps; "
          f"{same} of {batch} sequences equal greedy decoding")
    if gdn.gdn_read_device_error() != 0:
        raise RuntimeError("a kernel reported an error")
    return want, got, windows


if __name__ == "__main__":
    main()
