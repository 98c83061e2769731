"""Rotary frequencies for KVCache.set_rotary / slora_kv_set_rotary.

Pair i of a head's rotated part turns by ``position * inv_freq[i]`` radians
("RoFormer: Enhanced Transformer with Rotary Position Embedding", section 3.4:
base ** (-2 i / rot_dim)).  The scalings stretch a model's positions over a
longer context than it was trained on; each is a choice of frequencies and of
one factor on the rotated vectors, so the kernels need nothing of their own.
"""
from __future__ import annotations

import math
from typing import List, Tuple


def inv_freq(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
             trained_len: int = 0, fast: float = 32.0, slow: float = 1.0) -> Tuple[List[float], float]:
    """(rot_dim / 2 frequencies in radians a position, mscale).

    scaling "none"    the plain frequencies
            "linear"  positions divided by `factor` (position interpolation)
            "base"    the base raised to base * factor ** (rot_dim / (rot_dim - 2)): the
                      lowest frequency is divided by `factor`, the highest unchanged
                      (NTK-aware scaling)
            "parts"   frequencies that turn more than `fast` times over `trained_len`
                      positions unchanged, less than `slow` times divided by `factor`, a
                      linear ramp over the turns' pair index between; mscale
                      0.1 ln(factor) + 1 ("YaRN: Efficient Context Window Extension of
                      Large Language Models", section 3)
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling == "base":
        if rot_dim < 4:
            raise ValueError("scaling 'base' needs rot_dim of at least 4")
        base *= factor ** (rot_dim / (rot_dim - 2))
    plain = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in ("none", "base"):
        return plain, 1.0
    if scaling == "linear":
        return [f / factor for f in plain], 1.0
    if scaling == "parts":
        if trained_len < 1 or not fast > slow > 0:
            raise ValueError("scaling 'parts' needs trained_len and fast > slow > 0")

        def pair_of(turns):   # the (real) pair index that turns so often over the trained length
            return rot_dim * math.log(trained_len / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(pair_of(fast), 0.0), min(pair_of(slow), rot_dim / 2 - 1.0)
        out = []
        for i, f in enumerate(plain):
            stretched = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            out.append(f * (1.0 - stretched) + f / factor * stretched)
        return out, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")
