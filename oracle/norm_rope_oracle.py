"""Oracle for the norm with rotation, per head and as the cache's write side.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this module:
only the tests may call it.  It shares no code with the CUDA library.

In float64, from the definitions: n = x / sqrt(mean(x^2) + eps) * w over a
vector; a pair (a, b) at angle phi becomes (a cos phi - b sin phi,
a sin phi + b cos phi), where cos and sin are the given table's values; pairs
are (2i, 2i + 1) or (i, i + half).
"""
from __future__ import annotations

import numpy as np


def rms_norm(x, weight, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return n if weight is None else n * np.asarray(weight, dtype=np.float64)


def rotate(x, cos_sin_rows, interleaved: bool):
    """x [..., D] rotated by rows [..., D] of the table; also |a| + |b| of each output's pair."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    cs = np.asarray(cos_sin_rows, dtype=np.float64)
    out, mag = np.empty_like(x), np.empty_like(x)
    for j in range(half):
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b, c, s = x[..., ia], x[..., ib], cs[..., j], cs[..., half + j]
        out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
        mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return out, mag


def norm_rope(x, positions, cos_sin, weight, eps: float, norm: bool, rope_offset: int, interleaved: bool):
    """(out, magnitude) of x [T, H, D]; rows whose position is outside the table are zero.

    magnitude: what an error bound of an output element scales with (|a| + |b| of its pair where it is
    rotated, |n| elsewhere)."""
    n = rms_norm(x, weight, eps) if norm else np.asarray(x, dtype=np.float64).copy()
    mag = np.abs(n)
    if cos_sin is None:
        return n, mag
    cs = np.asarray(cos_sin, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.int64)
    ok = (pos >= 0) & (pos < cs.shape[0])
    sl = slice(rope_offset, rope_offset + cs.shape[1])
    rows = cs[np.where(ok, pos, 0)][:, None, :]
    n[..., sl], mag[..., sl] = rotate(n[..., sl], rows, interleaved)
    n[~ok], mag[~ok] = 0.0, 0.0
    return n, mag
