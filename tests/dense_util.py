"""Comparisons of the dense decode that its tests of weights share."""
import numpy as np

from cache_util import bits
from oracle import dense_oracle

# A weight times its block's scale: two E4M3 terms of 4 bits each (2^-9 of it), after four roundings to fp16 (2^-11 each).
WEIGHT = 2.0 ** -8
# fp16's least step, 2^-24, where the row's largest product of weight and scale is at least 2^1.75 (the window's lower end
# less 2^4 for A): half of it, for a weight (times a mantissa below 2), a mantissa (for weights below the largest product)
# and their product: 2^-25.75 + 2^-25 + 2^-26.75.  A reference is at most 2^-16.75 of the largest operand, with steps of
# 2^-9 and as much for the offset: 2^-25.75.  Together below 2^-23.5.
LEAST = 2.0 ** -23.5


def floor_of(rows: int) -> float:
    """The second term has steps of 2^-9 (of 2^-13 for 16 and 32 rows) and takes an offset of up to half a step, so it is off
    by up to a step; a tile's largest operand is above 2^-0.25."""
    return 2.0 ** -8.75 if rows == 64 else 2.0 ** -12.75


def check_weights(out, lse, q, cache, bt, lens, sm_scale, rows):
    """Element by element, and by the root mean square over each block's 128 dims."""
    ref, rl, worst, sigma, e = dense_oracle.dense_errors(bits(q).reshape(q.shape), cache.cpu().numpy(), bt.cpu().numpy(),
                                                         lens.cpu().numpy(), sm_scale, WEIGHT, floor_of(rows), LEAST)
    got, gl = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    full = np.isfinite(rl)
    assert np.array_equal(np.isneginf(gl), ~full) and np.all(got[~full] == 0.0)
    if not full.any():
        return
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert np.all(err <= worst + 1e-300), f"out: {(err / (worst + 1e-300)).max():.3f} of its bound"
    B, H, _ = err.shape
    blocks = lambda x: np.sqrt((x.reshape(B, H, 4, 128) ** 2).mean(-1))
    rms, bound = blocks(err), 1.5 * blocks(sigma)
    assert np.all(rms <= bound + 1e-300), f"rms over a block: {(rms / (bound + 1e-300)).max():.3f} of its bound"
    ltol = e + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(full, rl, 0.0))
    assert np.all(np.abs(gl - rl)[full] <= ltol[full]), "lse"


def block_errors(out, ref):
    """[B, H, 4]: error of each 128-dim block relative to that block's own result."""
    B, H, _ = ref.shape
    d = lambda x: np.sqrt((x.reshape(B, H, 4, 128) ** 2).sum(-1))
    return d(out - ref) / d(ref)
