"""Oracle for the dense decode (every cached position attends) and for reading records back.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this module:
only the tests may call it.  It shares no code with the CUDA library.

What it computes, in float64: query b, head h of request b // s_q attends over
the positions 0 <= t < seq_lens[b] whose logical page lies in the block-table
row and whose physical page lies in the cache,
    s_t = sm_scale * q.k_t,  lse = ln sum exp(s_t),  out = sum exp(s_t - lse) v_t
(out = 0 and lse = -inf without a position), with k and v of the cache record.

Beside the result it gives sizes that rounding-error bounds need:
    weighted   sum_t exp(s_t - lse) |v_t|
    floor      the sum over tiles of 128 positions of (the tile's largest
               exp(s_t - lse) 2^e_t) times sum_t |code_t|, with e_t the exponent of
               the largest of a position's four scales
    score_err  a bound on the error of a score whose latent part multiplies the
               codes with q as two E4M3 terms and accumulates in float32, see
               score_error_bound.
"""
from __future__ import annotations

import numpy as np

from .sparse_mla_oracle import D_LATENT, PAGE_SIZE, RECORD_BYTES, as_f64_q, decode_record, dequantize_record

TILE = 128


def positions_rows(bt_row, n: int, num_pages: int):
    """Physical rows of positions 0 .. n - 1 (skipping those without a page), and the positions."""
    rows, pos = [], []
    for t in range(max(0, n)):
        lp = t // PAGE_SIZE
        if lp >= len(bt_row):
            break
        page = int(bt_row[lp])
        if 0 <= page < num_pages:
            rows.append(page * PAGE_SIZE + t % PAGE_SIZE)
            pos.append(t)
    return np.array(rows, dtype=np.int64), np.array(pos, dtype=np.int64)


def score_error_bound(q: np.ndarray, k: np.ndarray, sm_scale: float) -> np.ndarray:
    """[H, n] bound on |score error|.

    Accumulating 576 products in float32 is off by at most 2^-20 of the sum of
    their magnitudes (the accumulator adds groups of 16 or 32 products, so about
    40 roundings of 2^-24 each).  q as hi + lo in E4M3, scaled so that the
    largest latent element of a row lies in [2^7, 2^8): hi keeps 4 bits, so an
    element of 8 bits leaves a remainder of 4 bits, which lo holds exactly unless
    it falls below E4M3's step of 2^-9; that needs an element below 2^-8 of the
    largest, and the error is then at most 2^-10 / 2^7 of the largest.
    """
    err = 2.0 ** -20 * (np.abs(q) @ np.abs(k).T)
    ql, kl = np.abs(q[:, :D_LATENT]), np.abs(k[:, :D_LATENT])
    top = ql.max(axis=1, keepdims=True)
    small = (ql < 2.0 ** -8 * top) & (ql > 0)
    err = err + 2.0 ** -17 * (top * small) @ kl.T
    return abs(sm_scale) * err


def dense_decode(q, kv_cache, block_table, seq_lens, sm_scale: float):
    """(out [B, H, 512], lse [B, H], weighted [B, H, 512], floor [B, H, 512], score_err [B, H]) in float64."""
    qf = as_f64_q(q)
    cache = np.asarray(kv_cache, dtype=np.uint8)
    flat = cache.reshape(-1, RECORD_BYTES)
    bt = np.asarray(block_table, dtype=np.int64)
    B, H, _ = qf.shape
    s_q = B // bt.shape[0]
    out = np.zeros((B, H, D_LATENT))
    weighted = np.zeros((B, H, D_LATENT))
    floor = np.zeros((B, H, D_LATENT))
    lse = np.full((B, H), -np.inf)
    score_err = np.zeros((B, H))
    for b in range(B):
        rows, pos = positions_rows(bt[b // s_q], int(seq_lens[b]), cache.shape[0])
        if rows.size == 0:
            continue
        k = dequantize_record(flat[rows])
        s = sm_scale * (qf[b] @ k.T)
        m = s.max(axis=1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(axis=1, keepdims=True)
        lse[b] = (m + np.log(z))[:, 0]
        out[b] = (e / z) @ k[:, :D_LATENT]
        weighted[b] = (e / z) @ np.abs(k[:, :D_LATENT])
        score_err[b] = score_error_bound(qf[b], k, sm_scale).max(axis=1)
        codes, scales, _ = decode_record(flat[rows])
        top = np.abs(scales).max(axis=1)
        size = e / z * np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0))))
        for tile in np.unique(pos // TILE):
            at = pos // TILE == tile
            floor[b] += size[:, at].max(axis=1)[:, None] * np.abs(codes[at]).sum(axis=0)
    return out, lse, weighted, floor, score_err


def dense_errors(q, kv_cache, block_table, seq_lens, sm_scale: float, weight_bits: float, floor: float,
                 least: float):
    """What rounding may do to dense_decode's result: (out, lse, worst, sigma, score_err), worst and sigma as out.

    A position's operand in a 128-dim block is its softmax weight times the block's scale.  It is off by at most
    weight_bits of itself or `floor` of the largest operand that the row has in the block's tile of 128 positions,
    whichever is more, or `least` of the row's largest operand in any block; a block whose codes are all zero has no
    operand.  (A tile more than 2^29 below the row's largest operand in the block has the floor of one 2^29 below.)  The
    result is rounded to bf16 (2^-8 of itself), and a score
    off by e changes a weight by at most 2 e of itself.
    worst: what an element's error cannot exceed when the errors u_t of the positions are unrelated: a sum of a_t u_t
           with |u_t| <= 1 exceeds 7 sqrt(sum a_t^2) with probability 2 exp(-49 / 2) < 5e-11, and never sum a_t.
           Equal weights may share one error: weight_bits of the result.
    sigma: the root of the sum of the squares of the same terms, each at its most.
    """
    qf = as_f64_q(q)
    cache = np.asarray(kv_cache, dtype=np.uint8)
    flat = cache.reshape(-1, RECORD_BYTES)
    bt = np.asarray(block_table, dtype=np.int64)
    B, H, _ = qf.shape
    s_q = B // bt.shape[0]
    out, lse, _, _, score_err = dense_decode(q, kv_cache, block_table, seq_lens, sm_scale)
    worst, sigma = np.zeros_like(out), np.zeros_like(out)
    for b in range(B):
        rows, pos = positions_rows(bt[b // s_q], int(seq_lens[b]), cache.shape[0])
        if rows.size == 0:
            continue
        k = dequantize_record(flat[rows])
        p = np.exp(sm_scale * (qf[b] @ k.T) - lse[b][:, None])
        v = np.abs(k[:, :D_LATENT])
        codes, scales, _ = decode_record(flat[rows])
        codes = np.abs(codes).reshape(-1, 4, D_LATENT // 4)
        size = np.where(codes.any(axis=2), np.abs(scales), 0.0)                     # [n, 4]
        operand = p[:, :, None] * size[None]                                        # [H, n, 4]
        off = np.empty_like(operand)
        for tile in np.unique(pos // TILE):
            at = pos // TILE == tile
            off[:, at] = operand[:, at].max(axis=1, keepdims=True)
        off = floor * np.maximum(off, 2.0 ** -29 * operand.max(axis=1, keepdims=True))
        off += least * operand.max(axis=(1, 2), keepdims=True)
        small = [np.einsum("hnb,nbd->hbd", off ** n, codes ** n).reshape(H, D_LATENT) for n in (1, 2)]
        weighted = p @ v
        spread = np.sqrt(weight_bits ** 2 * (p ** 2 @ v ** 2) + small[1])
        common = (2.0 ** -8 + weight_bits) * np.abs(out[b])
        score = (2 * score_err[b][:, None] + 2.0 ** -18) * weighted
        worst[b] = common + score + np.minimum(7 * spread, weight_bits * weighted + small[0])
        sigma[b] = np.sqrt((2.0 ** -8 * out[b]) ** 2 + score ** 2 + spread ** 2)
    return out, lse, worst, sigma, score_err


def read_records(kv_cache, block_table, positions, requests=None) -> np.ndarray:
    """float64 [T, 576]: the dequantised records; zeros for a token out of range."""
    cache = np.asarray(kv_cache, dtype=np.uint8)
    bt = np.asarray(block_table, dtype=np.int64)
    out = np.zeros((len(positions), D_LATENT + 64))
    for i, t in enumerate(np.asarray(positions, dtype=np.int64)):
        r = int(requests[i]) if requests is not None else i
        if r < 0 or r >= bt.shape[0] or t < 0 or t // PAGE_SIZE >= bt.shape[1]:
            continue
        page = bt[r, t // PAGE_SIZE]
        if 0 <= page < cache.shape[0]:
            out[i] = dequantize_record(cache[page, t % PAGE_SIZE])
    return out
