"""fp64 oracle of the paged key-value cache operators (test infrastructure).

Plain numpy loops over requests and tokens, following the definitions in
include/slora.h; shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np


def plan(table, rows, ctx, new, pages, T, P, num_pages):
    """Writes the opened blocks into `table` [L, 2, rows, blocks]; returns the
    batch arrays.  pages: [block][layer][K, V] flat."""
    L = table.shape[0]
    pages = np.asarray(pages, dtype=np.int64).reshape(-1, L, 2)
    tok_req = np.full(T, -1, np.int32)
    tok_pos = np.full(T, -1, np.int32)
    slots = np.full((L, 2, T), -1, np.int32)
    q_start = np.zeros(len(ctx) + 1, np.int32)
    t = b = 0
    for r, (row, c, n) in enumerate(zip(rows, ctx, new)):
        q_start[r] = t
        for i in range(n):
            pos = c + i
            if pos % P == 0:                     # the token opens a block
                for layer in range(L):
                    for j in (0, 1):
                        page = pages[b, layer, j]
                        table[layer, j, row, pos // P] = page if 0 <= page < num_pages else -1
                b += 1
            page = table[:, :, row, pos // P].astype(np.int64)
            slots[:, :, t] = np.where(page < 0, -1, page * P + pos % P)
            tok_req[t], tok_pos[t] = r, pos
            t += 1
    q_start[len(ctx)] = t
    return {"q_start": q_start, "kv_len": np.asarray(ctx, np.int32) + np.asarray(new, np.int32), "tok_req": tok_req,
            "tok_pos": tok_pos, "slots": slots}


def norm_rotate(x, w, eps, pos, inv_freq, rot, interleaved, mscale):
    """x [heads, d] of one token at position pos, in fp64."""
    x = np.array(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = float(pos) * float(inv_freq[i])
        c, s = mscale * math.cos(ang), mscale * math.sin(ang)
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, a] * s + x[:, b] * c
    return y


def attend(q, keys, values, ctx, scale, softcap):
    """One request: q [n, heads_q, d] at positions ctx + i, keys and values
    [ctx + n, heads_kv, d]; [n, heads_q, d]."""
    n, hq, d = q.shape
    hkv = keys.shape[1]
    out = np.zeros((n, hq, d))
    for h in range(hq):
        k, v = keys[:, h // (hq // hkv)].astype(np.float64), values[:, h // (hq // hkv)].astype(np.float64)
        for i in range(n):
            m = ctx + i + 1
            s = scale * (k[:m] @ q[i, h].astype(np.float64))
            if softcap:
                s = softcap * np.tanh(s / softcap)
            p = np.exp(s - s.max())
            out[i, h] = (p / p.sum()) @ v[:m]
    return out
