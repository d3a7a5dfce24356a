"""Inputs and comparisons shared by the tests of the operators around the paged cache."""
import numpy as np
import torch

from oracle import dense_oracle
from sparse_mla_decode_paged_gb300 import workloads as wl

DEV = "cuda"


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def make_dense(lens, H, s_q=1, seed=0, spare_pages=3, q_scale=1.0, poison=True):
    """CPU inputs of a dense decode: lens[b] per query (s_q queries per request).  With poison, every record that no
    query may read holds NaN codes, infinite scales and NaN rope values."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    R = B // s_q
    need = [max(0, max(lens[r * s_q:(r + 1) * s_q])) for r in range(R)]
    pages = [(n + 63) // 64 for n in need]
    total = sum(pages) + spare_pages
    cache = wl.fill_kv_cache(total, g, "cpu", outlier_channels=5)
    if poison:
        bad = torch.full((656,), 0x7F, dtype=torch.uint8)
        bad[512:528] = torch.tensor([float("inf")] * 4).view(torch.uint8)
        bad[528:] = torch.full((64,), float("nan"), dtype=torch.bfloat16).view(torch.uint8)
    perm = torch.randperm(total, generator=g).to(torch.int32)
    width = max(1, max(pages))
    bt = torch.full((R, width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        bt[r, :n] = perm[at:at + n]
        at += n
        if poison and need[r] % 64:
            cache[int(bt[r, n - 1]), need[r] % 64:] = bad
    if poison:
        for pg in perm[at:].tolist():
            cache[pg] = bad
    q = (torch.randn((B, H, 576), generator=g) * q_scale).to(torch.bfloat16)
    return q, cache, bt, torch.tensor(lens, dtype=torch.int32)


def check_dense(out, lse, q, cache, bt, lens, sm_scale):
    """Element by element against the float64 oracle.

    out: one bf16 rounding (2^-8 of the value).  A weight is rounded to fp16, times a scale factor rounded to fp16, the
    product rounded to fp16, then to two E4M3 terms of 8 bits in all: 3 * 2^-11 + 2^-9 of itself, with 2^-11 more for
    the float32 exponential, sums and merge, so 2^-8 of the weighted magnitudes; below the range of those 8
    bits the second term has steps of 2^-9 where the tile's largest weight is at least 2^3.75 (of a row whose reference
    has not gone as far below its highest as it may): 2^-13.75 of the tile's largest.  A score error e changes a weight by at most 2 e.
    lse: the score error, and 2^-20 for exponential, sum and logarithm with 2^-22 of its size."""
    ref, rl, weighted, floor, e = dense_oracle.dense_decode(bits(q).reshape(q.shape), cache.cpu().numpy(), bt.cpu().numpy(),
                                                            lens.cpu().numpy(), sm_scale)
    got, gl = out.float().cpu().double().numpy(), lse.cpu().double().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert np.all(got[empty] == 0.0)
    full = ~empty
    if not full.any():
        return
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * e[..., None]) * weighted + 2.0 ** -13.75 * floor
    worst = (np.abs(got - ref) / np.maximum(tol, 1e-300))[full].max()
    ltol = e + 2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(full, rl, 0.0))
    lworst = (np.abs(gl - np.where(full, rl, 0.0)) / ltol)[full].max()
    assert np.isfinite(got[full]).all() and worst <= 1.0, f"out error {worst:.3f} of its bound"
    assert np.isfinite(gl[full]).all() and lworst <= 1.0, f"lse error {lworst:.3f} of its bound"
