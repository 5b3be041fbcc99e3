"""The resident paged cache: append, attention of a step's new rows, received
attention weight, eviction (TEST INFRASTRUCTURE ONLY; see the package
docstring).

Token t of sequence b is pool row table[b, t // page] * page + t % page; an
entry outside the pool is no page and its tokens are absent. Sequence b's new
rows are rows row0[b] .. row0[b+1]-1 of the step, its last ones: row i of n is
at position seq_len[b] - n + i. A row at position p sees t <= p, and with a
window > 0 only t > p - window or t < n_sink.

Plain float64 numpy, one sequence and one row at a time, with the textbook
softmax.
"""
import numpy as np

from .numerics import bf16_to_f64

D_V = 512


def slots(table_row, page, n_slots, n):
    """Slot of tokens 0 .. n-1, -1 where there is no page."""
    out = np.full(n, -1, np.int64)
    for t in range(n):
        if t // page < len(table_row):
            pg = int(table_row[t // page])
            s = pg * page + t % page
            if pg >= 0 and s < n_slots:
                out[t] = s
    return out


def append(pool, table, page, row0, seq_len, rows):
    """Writes the rows in place; returns whether any had no slot."""
    lost = False
    for b in range(len(seq_len)):
        n = int(row0[b + 1]) - int(row0[b])
        sl = slots(table[b], page, len(pool), max(int(seq_len[b]), 0))
        for i in range(n):
            p = int(seq_len[b]) - n + i
            if p < 0 or sl[p] < 0:
                lost = True
            else:
                pool[sl[p]] = rows[int(row0[b]) + i]
    return lost


def visible(p, slot, window, n_sink):
    """Indices of the tokens that a row at position p sees."""
    t = np.arange(len(slot))
    ok = (t <= p) & (slot >= 0)
    if window:
        ok &= (t > p - window) | (t < n_sink)
    return np.flatnonzero(ok)


def attention(q_bits, pool_bits, table, page, row0, seq_len, sm_scale, window=0, n_sink=0):
    """out [T, H, 512], lse [T, H], and for error bounds sum_t p_t |v_t|
    [T, H, 512] and the largest sum_d |q_d k_d| over the visible tokens,
    scaled [T, H]; rows of no sequence stay NaN."""
    T, H, _ = q_bits.shape
    scale = float(np.float32(sm_scale))
    out, absv = np.full((T, H, D_V), np.nan), np.full((T, H, D_V), np.nan)
    lse, mag = np.full((T, H), np.nan), np.full((T, H), np.nan)
    for b in range(len(seq_len)):
        n = int(row0[b + 1]) - int(row0[b])
        if n == 0:
            continue
        sl = slots(table[b], page, len(pool_bits), max(int(seq_len[b]), 0))
        kv = bf16_to_f64(pool_bits[np.maximum(sl, 0)])
        for i in range(n):
            r = int(row0[b]) + i
            see = visible(int(seq_len[b]) - n + i, sl, window, n_sink)
            if len(see) == 0:
                out[r], absv[r], lse[r], mag[r] = 0, 0, -np.inf, 0
                continue
            q, k = bf16_to_f64(q_bits[r]), kv[see]
            s = (q @ k.T) * scale
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            den = p.sum(axis=1, keepdims=True)
            out[r] = (p @ k[:, :D_V]) / den
            absv[r] = (p @ np.abs(k[:, :D_V])) / den
            lse[r] = (m + np.log(den))[:, 0]
            mag[r] = (np.abs(q) @ np.abs(k).T).max(axis=1) * abs(scale)
    return out, lse, absv, mag


def received(q_bits, lse, pool_bits, table, page, row0, seq_len, sm_scale, acc_in, decay, window=0, n_sink=0):
    """decay * acc_in + the weight each token received, [B, ld]; entries at and
    past a sequence's length as in acc_in."""
    scale = float(np.float32(sm_scale))
    acc = np.array(acc_in, np.float64)
    for b in range(len(seq_len)):
        n, length = int(row0[b + 1]) - int(row0[b]), max(int(seq_len[b]), 0)
        acc[b, :length] *= float(np.float32(decay))
        sl = slots(table[b], page, len(pool_bits), length)
        kv = bf16_to_f64(pool_bits[np.maximum(sl, 0)])
        for i in range(n):
            r = int(row0[b]) + i
            see = visible(length - n + i, sl, window, n_sink)
            if len(see):
                s = (bf16_to_f64(q_bits[r]) @ kv[see].T) * scale
                acc[b, see] += np.exp(s - np.asarray(lse[r], np.float64)[:, None]).sum(axis=0)
    return acc


def evict(acc, seq_len, keep, n_sink, n_recent):
    """Kept tokens of each sequence, ascending (list of arrays)."""
    out = []
    for b, n in enumerate(int(x) for x in seq_len):
        n = max(n, 0)
        if n <= keep:
            out.append(np.arange(n))
            continue
        mid = list(range(n_sink, n - n_recent))
        w = np.asarray(acc[b], np.float64)
        # heaviest first: NaN, then descending weight, then the lower index
        mid.sort(key=lambda t: (not np.isnan(w[t]), 0.0 if np.isnan(w[t]) else -w[t], t))
        stay = mid[:keep - n_sink - n_recent] + list(range(n_sink)) + list(range(n - n_recent, n))
        out.append(np.array(sorted(stay)))
    return out
