"""Oracle for the attention weights accumulated per cached position and for eviction by them.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path imports this module: only the tests may call it.  It shares no
code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from .dense_oracle import positions_rows, score_error_bound
from .sparse_mla_oracle import PAGE_SIZE, RECORD_BYTES, as_f64_q, dequantize_record


def attention_weights(q, kv_cache, block_table, seq_lens, lse, sm_scale, weights, decay):
    """(weights [R, n] in float64, a bound on the error of each).

    A term exp(s - lse) is off by the error of its score and by the arithmetic of its exponent in float32 (s and lse
    in units of log2, three roundings of 2^-24 of them, times ln 2; 2^-21 for the exponential itself); the terms of a
    position, all of one sign, are added in at most rows / 2 + 2 roundings of 2^-24 of the sum."""
    qf = as_f64_q(q)
    flat = np.asarray(kv_cache, dtype=np.uint8).reshape(-1, RECORD_BYTES)
    bt, lse = np.asarray(block_table, dtype=np.int64), np.asarray(lse, dtype=np.float64)
    w = np.array(weights, dtype=np.float64)
    err = np.zeros_like(w)
    R, n = w.shape
    s_q, H = qf.shape[0] // R, qf.shape[1]
    most = min(n, bt.shape[1] * PAGE_SIZE)
    for r in range(R):
        lens = [min(most, max(0, int(seq_lens[b]))) for b in range(r * s_q, (r + 1) * s_q)]
        end = max(lens)
        total, bound = np.zeros(end), np.zeros(end)
        for j, m in enumerate(lens):
            b = r * s_q + j
            rows, pos = positions_rows(bt[r], m, len(flat) // PAGE_SIZE)
            if rows.size == 0:
                continue
            k = dequantize_record(flat[rows])
            s = sm_scale * (qf[b] @ k.T)
            p = np.exp(s - lse[b][:, None])
            e = score_error_bound(qf[b], k, sm_scale) + 2.0 ** -21 + 3 * 2.0 ** -24 * (np.abs(s) + np.abs(lse[b])[:, None])
            total[pos] += p.sum(0)
            bound[pos] += (p * np.expm1(e)).sum(0)
        old = decay * w[r, :end] if decay != 0 else np.zeros(end)
        err[r, :end] = bound + (s_q * H / 2 + 2) * 2.0 ** -24 * (total + bound) + 2.0 ** -23 * (np.abs(old) + total)
        w[r, :end] = old + total
    return w, err


def order_key(x):
    """IEEE 754 totalOrder of float32 values as whole numbers."""
    b = np.asarray(x, dtype=np.float32).view(np.int32).astype(np.int64)
    return np.where(b < 0, b ^ 0x7FFFFFFF, b)


def evict(weights, positions, next_positions, seq_lens, keep, kv_cache, block_table, sinks, recent):
    """(weights, positions, cache, new lengths) after the eviction; keep an int or one per request."""
    w, pos = np.array(weights, dtype=np.float32), np.array(positions, dtype=np.int32)
    cache = np.array(kv_cache, dtype=np.uint8)
    flat = cache.reshape(-1, RECORD_BYTES)
    bt = np.asarray(block_table, dtype=np.int64)
    R, cols = w.shape
    new = np.zeros(R, dtype=np.int32)
    row = lambda r, t: bt[r, t // PAGE_SIZE] * PAGE_SIZE + t % PAGE_SIZE
    for r in range(R):
        n = min(max(0, int(seq_lens[r])), cols, bt.shape[1] * PAGE_SIZE)
        at = pos[r, :n].astype(np.int64)
        held = (at < sinks) | (at >= int(next_positions[r]) - recent)
        key = np.where(held, 1 << 40, order_key(w[r, :n]))
        k = max(0, int(keep if np.ndim(keep) == 0 else keep[r]))
        m = min(n, max(k, int(held.sum())))
        kept = np.zeros(n, dtype=bool)
        kept[sorted(range(n), key=lambda t: (-key[t], t))[:m]] = True
        src = [t for t in range(m, n) if kept[t]]
        dst = [t for t in range(m) if not kept[t]]
        for a, b in zip(src, dst):
            if all(0 <= bt[r, t // PAGE_SIZE] < len(cache) for t in (a, b)):
                flat[row(r, b)] = flat[row(r, a)]
            w[r, b], pos[r, b] = w[r, a], pos[r, a]
        w[r, m:n] = 0
        new[r] = m
    return w, pos, cache, new
