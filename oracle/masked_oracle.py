"""Oracle for the decode with capped, biased and masked scores, and for the decode behind shared prefixes.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this module: only the tests may call it.  It shares no
code with the CUDA library.

Results are those of dense_oracle.dense_decode: (out, lse, weighted, floor, score_err), the last three being sizes that
bounds on rounding errors need.
"""
from __future__ import annotations

import numpy as np

from .dense_oracle import TILE, positions_rows, score_error_bound
from .sparse_mla_oracle import D_LATENT, RECORD_BYTES, as_f64_q, decode_record, dequantize_record


def visible(pos, length, start, prefix):
    """Which positions a query of this length sees."""
    seen = pos < length
    if start is not None:
        seen &= (pos >= start) | (pos < (prefix if prefix is not None else 0))
    return seen


def attend(q, k, codes, scales, s, err, tile, steep=None):
    """One query's heads over records k with scores s [H, n], off by err at most, in tiles of these numbers.  The rows
    `steep` keep the reference of their largest weight, so the steps of their small weights follow that one instead of
    the tile's largest."""
    H = q.shape[0]
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    z = e.sum(axis=1, keepdims=True)
    p = e / z
    floor = np.zeros((H, D_LATENT))
    top = np.abs(scales).max(axis=1)
    size = p * np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0))))
    for t in np.unique(tile):
        at = tile == t
        most = size[:, at].max(axis=1)
        if steep is not None:
            most = np.where(steep, size.max(axis=1), most)
        floor += most[:, None] * np.abs(codes[at]).sum(axis=0)
    # a position without weight to speak of adds less than its weight, whatever its score's error
    score_err = np.where(p > 2.0 ** -40, err, 0.0).max(axis=1)
    return p @ k[:, :D_LATENT], (m + np.log(z))[:, 0], p @ np.abs(k[:, :D_LATENT]), floor, score_err


def _empty(B, H):
    return (np.zeros((B, H, D_LATENT)), np.full((B, H), -np.inf), np.zeros((B, H, D_LATENT)), np.zeros((B, H, D_LATENT)),
            np.zeros((B, H)))


def masked_decode(q, kv_cache, block_table, seq_lens, sm_scale, softcap=0.0, slopes=None, starts=None, prefix_lens=None):
    """A capped score is off by the score's error, 2^-20 of itself and the roundings of its factors; a biased one by
    2^-23 of the bias and of the sum more."""
    qf = as_f64_q(q)
    cache = np.asarray(kv_cache, dtype=np.uint8)
    flat = cache.reshape(-1, RECORD_BYTES)
    bt = np.asarray(block_table, dtype=np.int64)
    B, H, _ = qf.shape
    s_q = B // bt.shape[0]
    res = _empty(B, H)
    for b in range(B):
        n = max(0, int(seq_lens[b]))
        rows, pos = positions_rows(bt[b // s_q], n, cache.shape[0])
        seen = visible(pos, n, None if starts is None else int(starts[b]), None if prefix_lens is None else int(prefix_lens[b]))
        rows, pos = rows[seen], pos[seen]
        if rows.size == 0:
            continue
        k = dequantize_record(flat[rows])
        codes, scales, _ = decode_record(flat[rows])
        s = sm_scale * (qf[b] @ k.T)
        err, steep = score_error_bound(qf[b], k, sm_scale), None
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
            err = err + 2.0 ** -20 * np.abs(s)
        if slopes is not None:
            bias = np.asarray(slopes, dtype=np.float64)[:, None] * (pos - (n - 1))[None]
            s = s + bias
            err = err + 2.0 ** -22 * (np.abs(bias) + np.abs(s))
            steep = np.asarray(slopes, dtype=np.float32) * np.log2(np.e) * TILE >= 0.25 - 1e-6
        for to, got in zip(res, attend(qf[b], k, codes, scales, s, err, pos // TILE, steep)):
            to[b] = got
    return res


def shared_decode(q, kv_cache, prefix_table, prefix_lens, block_table, seq_lens, sm_scale, half_keys=False):
    """Requests r attend over the positions of their group's prefix, then over their own.

    With half_keys the keys are rounded to fp16 (2^-11 of each element, or of 2^-28 of the largest of its group of
    32 positions): a score's error is a sum of 576 unrelated roundings a_i u_i, |u_i| <= 1, which exceeds 7 sqrt(sum
    a_i^2) with probability 2 exp(-49 / 2) < 5e-11 and never sum |a_i|; lse's is their mean under the weights, bounded
    alike (to first order; the second adds less than the square of the largest).  Then a sixth size is returned, lse's
    error."""
    qf = as_f64_q(q)
    cache = np.asarray(kv_cache, dtype=np.uint8)
    flat = cache.reshape(-1, RECORD_BYTES)
    pt, bt = np.asarray(prefix_table, dtype=np.int64), np.asarray(block_table, dtype=np.int64)
    B, H, _ = qf.shape
    s_q, each = B // bt.shape[0], bt.shape[0] // pt.shape[0]
    res = _empty(B, H) + ((np.zeros((B, H)),) if half_keys else ())
    for b in range(B):
        r = b // s_q
        a, pa = positions_rows(pt[r // each], int(prefix_lens[r // each]), cache.shape[0])
        c, pc = positions_rows(bt[r], int(seq_lens[b]), cache.shape[0])
        rows = np.concatenate([a, c])
        if rows.size == 0:
            continue
        k = dequantize_record(flat[rows])
        codes, scales, _ = decode_record(flat[rows])
        s = sm_scale * (qf[b] @ k.T)
        tile = np.concatenate([pa // TILE, 10 ** 7 + pc // TILE])
        err = score_error_bound(qf[b], k, sm_scale)
        sigma = np.zeros_like(err)
        if half_keys:
            size = np.abs(k)
            page = np.concatenate([pa // 32, 10 ** 7 + pc // 32])
            each_page, at = np.unique(page, return_inverse=True)
            most = np.array([size[page == t].max() for t in each_page])[at]
            off = abs(sm_scale) * 2.0 ** -11 * np.maximum(size, 2.0 ** -27 * most[:, None])
            sigma = np.sqrt(qf[b] ** 2 @ (off ** 2).T)
            err = err + np.minimum(7 * sigma, np.abs(qf[b]) @ off.T)
        got = attend(qf[b], k, codes, scales, s, err, tile)
        for to, x in zip(res, got):
            to[b] = x
        if half_keys:
            p = np.exp(s - got[1][:, None])
            res[5][b] = 7 * np.sqrt((p ** 2 * sigma ** 2).sum(1)) + got[4] ** 2 + \
                (p * score_error_bound(qf[b], k, sm_scale)).sum(1)
    return res
