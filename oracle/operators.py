"""fp64 CPU restatements of the operators beside the decode step: the 4-bit key/value
cache, attention over it, and log probabilities with entropy and top alternatives.

TEST INFRASTRUCTURE, as the rest of this package: written from the definitions in
``include/gdn.h`` and sharing no code with the library. Everything is numpy in
float64; the cache is bytes.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MAX_SCALE_BYTE = 226


def scale_values() -> np.ndarray:
    """What the scale bytes 0 .. 226 stand for, rising."""
    b = np.arange(MAX_SCALE_BYTE + 1)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * 2.0 ** (e - 15.0))


def _nearest(a, grid):
    """Index of the nearest entry of a rising grid to a >= 0; at half way the even index."""
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    below, above = a - grid[hi - 1], grid[hi] - a
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)


def kv4_quantise(x):
    """Codes (uint8 0..15, like x) and scale bytes ([..., D/16]) of values [..., D]."""
    x = np.asarray(x, np.float64)
    x = np.clip(np.where(np.isnan(x), 0.0, x), -61440.0, 61440.0).reshape(*x.shape[:-1], -1, 16)
    byte = _nearest(np.abs(x).max(-1) / 6.0, scale_values())
    s = scale_values()[byte][..., None]
    code = _nearest(np.abs(np.divide(x, s, out=np.zeros_like(x), where=s > 0)), E2M1)
    code = code + np.where(np.signbit(x) & (s > 0), 8, 0)
    return code.reshape(*code.shape[:-2], -1).astype(np.uint8), byte.astype(np.uint8)


def kv4_dequantise(code, byte):
    v = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    return (v.reshape(*byte.shape, 16) * scale_values()[byte][..., None]).reshape(code.shape)


def _row_places(r, h, part, page, D):
    """Byte ranges of token row r of a page, kv head h, K (part 0) or V (part 1): where its code
    blocks (in order) and its scales lie within the page."""
    half = page * (D // 2 + D // 16)
    base = 2 * half * h + half * part
    turn = (8 * (r & 1) + 4 * ((r >> 2) & 1)) & (D // 16 - 1)
    blocks = [base + r * (D // 2) + 8 * (i ^ turn) for i in range(D // 16)]
    return blocks, base + page * (D // 2) + r * (D // 16)


def kv4_append(k, v, cache, block_table, kv_start, page, seq_len=None):
    """Writes k, v [B][L][T][H][D] into cache (uint8 [L][n_pages][bytes], in place)."""
    B, L, T, H, D = k.shape
    for part, x in enumerate((k, v)):
        code, byte = kv4_quantise(x)
        packed = code[..., 0::2] | (code[..., 1::2] << 4)
        for b in range(B):
            for t in range(T if seq_len is None else min(max(int(seq_len[b]), 0), T)):
                pos = int(kv_start[b]) + t
                for l in range(L):
                    row = cache[l, block_table[b, pos // page]]
                    for h in range(H):
                        blocks, at = _row_places(pos % page, h, part, page, D)
                        for i, o in enumerate(blocks):
                            row[o:o + 8] = packed[b, l, t, h, 8 * i:8 * i + 8]
                        row[at:at + D // 16] = byte[b, l, t, h]


def kv4_read(cache, block_table, b, l, h, end, page, D, first=0):
    """Keys and values [end - first][D] of positions first .. end - 1 of sequence b in float64."""
    out = np.zeros((2, end - first, D))
    for part in range(2):
        for pos in range(first, end):
            row = cache[l, block_table[b, pos // page]]
            blocks, at = _row_places(pos % page, h, part, page, D)
            p = np.concatenate([row[o:o + 8] for o in blocks])
            out[part, pos - first] = kv4_dequantise(np.stack([p & 15, p >> 4], -1).reshape(-1), row[at:at + D // 16])
    return out[0], out[1]


def attention_rows(q, k, v, last, scale):
    """Softmax attention of query rows q [n][D], row i over keys 0 .. last[i], and per output the bound
    terms of a rounded evaluation: (out, sum p |v|, max |scale| sum |q k|, max |score|)."""
    s = scale * (q @ k.T)
    hidden = np.arange(k.shape[0])[None, :] > np.asarray(last)[:, None]
    s = np.where(hidden, -np.inf, s)
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    size = np.where(hidden, 0.0, scale * (np.abs(q) @ np.abs(k).T)).max(1, keepdims=True)
    return p @ v, p @ np.abs(v), size, np.abs(np.where(hidden, 0.0, s)).max(1, keepdims=True)


def logprobs(x, tokens, k):
    """(logprob, entropy, top_ids, top_logprobs) of rows x [N][V]; rows without a finite maximum give NaN."""
    x = np.asarray(x, np.float64)
    N = x.shape[0]
    lp, ent, top = np.full(N, np.nan), np.full(N, np.nan), np.full((N, k), np.nan)
    order = np.where(np.isnan(x), np.inf, x)
    # NaN first, then by falling value, then by rising index
    ids = np.stack([np.lexsort((np.arange(x.shape[1]), -order[i], ~np.isnan(x[i])))[:k] for i in range(N)])
    for i in range(N):
        m = x[i].max()
        if not np.isfinite(m):
            continue
        z = x[i] - m
        p = np.exp(z)
        total = p.sum()
        lse = np.log(total)
        if 0 <= tokens[i] < x.shape[1]:
            lp[i] = z[tokens[i]] - lse
        ent[i] = lse - (p[p > 0] * z[p > 0]).sum() / total
        top[i] = z[ids[i]] - lse
    return lp, ent, ids, top
