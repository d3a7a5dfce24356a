"""Comparison of decode results with the oracles of masked_oracle."""
import numpy as np


def check_decode(out, lse, want):
    """Bounds as in cache_util.check_dense, element by element."""
    ref, rl, weighted, floor, e = want[:5]
    got, gl = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty) and np.all(got[empty] == 0.0)
    full = ~empty
    if not full.any():
        return
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * weighted + 2.0 ** -13.75 * floor
    ltol = (want[5] if len(want) == 6 else e) + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(full, rl, 0.0))
    assert np.isfinite(got[full]).all() and np.isfinite(gl[full]).all()
    worst, lworst = (np.abs(got - ref) / np.maximum(tol, 1e-300))[full].max(), (np.abs(gl[full] - rl[full]) / ltol[full]).max()
    assert worst <= 1.0, f"out error {worst:.3f} of its bound"
    assert lworst <= 1.0, f"lse error {lworst:.3f} of its bound"
