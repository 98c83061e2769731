"""fp64 oracle of keys and values held in 4 bits (test infrastructure).

Plain numpy, following the format in include/slora.h; shares no code with the
library.
"""
from __future__ import annotations

import numpy as np

LARGEST = {"f16": 31.0 * 2.0 ** 11, "bf16": 31.0 * 2.0 ** 123}
FINEST = {"f16": 2.0 ** -21, "bf16": 2.0 ** -100}


def groups(d):
    return -(-d // 32)


def row_bytes(heads, d):
    return -(-18 * groups(d) * heads // 16) * 16


def scale(m, dtype):
    """M of a group whose element of largest magnitude is m (finite)."""
    if m == 0:
        return 0.0
    unit = max(2.0 ** (np.frexp(abs(m))[1] - 5), FINEST[dtype])
    return float(np.copysign(min(np.ceil(abs(m) / unit) * unit, LARGEST[dtype]), m))


def quantise(x, dtype):
    """x [heads, d] of one token: k [heads, 32 ng] and M [heads, ng]."""
    heads, d = x.shape
    ng = groups(d)
    y = np.zeros((heads, 32 * ng))
    y[:, :d] = x
    k, M = np.zeros(y.shape, np.int64), np.zeros((heads, ng))
    for h in range(heads):
        for g in range(ng):
            v = y[h, 32 * g: 32 * g + 32]
            if not np.isfinite(v).all():
                M[h, g] = np.nan
                continue
            hi, lo = v.max(), v.min()
            M[h, g] = scale(hi if hi >= -lo else lo, dtype)
            if M[h, g]:
                k[h, 32 * g: 32 * g + 32] = np.clip(np.floor(8 * v / M[h, g] + 0.5), -7, 8)
    return k, M


def values(k, M, d):
    """What codes and scales stand for: [..., heads, d]."""
    return (np.repeat(M, 32, -1) * k / 8)[..., :d]


def _bits(M, dtype):
    """16-bit patterns of numbers that the type holds."""
    if dtype == "f16":
        b = M.astype(np.float16).view(np.uint16)
    else:
        b = (M.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.where(np.isnan(M), 0x7FFF, b).astype(np.uint16)


def _place(e, ng, is_value):
    g, r = e // 32, e % 32
    if is_value:
        return 16 * ((r // 4) * ng + g) + 4 * (r % 4)
    return 32 * ((r // 8) * ng + g) + 16 * (r % 2) + 4 * (r % 8 // 2)


def pack(k, M, dtype, is_value):
    """Token rows as bytes: k [n, heads, 32 ng], M [n, heads, ng] -> [n, row_bytes], padding 0."""
    n, heads, ng = M.shape
    codes = np.zeros((n, heads, 16 * ng), np.uint8)
    for e in range(32 * ng):
        at = _place(e, ng, is_value)
        codes[:, :, at // 8] |= ((k[:, :, e] + 7).astype(np.uint8) << (at % 8)).astype(np.uint8)
    rows = np.zeros((n, -(-18 * ng * heads // 16) * 16), np.uint8)
    rows[:, : 16 * ng * heads] = codes.reshape(n, -1)
    rows[:, 16 * ng * heads: 18 * ng * heads] = _bits(M, dtype).reshape(n, -1).view(np.uint8)
    return rows


def unpack(rows, heads, d, dtype, is_value):
    """The numbers that token rows [n, row_bytes] stand for: [n, heads, d]."""
    n, ng = rows.shape[0], groups(d)
    codes = rows[:, : 16 * ng * heads].reshape(n, heads, 16 * ng)
    k = np.zeros((n, heads, 32 * ng))
    for e in range(32 * ng):
        at = _place(e, ng, is_value)
        k[:, :, e] = (codes[:, :, at // 8] >> (at % 8) & 15).astype(np.float64) - 7
    b = np.ascontiguousarray(rows[:, 16 * ng * heads: 18 * ng * heads]).view(np.uint16).reshape(n, heads, ng)
    M = b.view(np.float16) if dtype == "f16" else (b.astype(np.uint32) << 16).view(np.float32)
    return values(k, M.astype(np.float64), d)
