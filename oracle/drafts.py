"""Drafted tokens over the resident paged cache: attention of trees, which
drafts the target accepts, and the accepted rows' move (TEST INFRASTRUCTURE
ONLY; see the package docstring).

Row i of a sequence's n new rows follows row parent[i] < i (anything else: the
cached tokens, c = seq_len - n of them). Its line is itself and what it follows,
row by row; its position is c + len(line) - 1; it is token c + i of its pages.

Plain float64 numpy, one row at a time.
"""
import numpy as np

from .numerics import bf16_to_f64
from .paged import D_V, slots


def line(parent, i):
    """Row i's line, itself first."""
    out = [i]
    while 0 <= int(parent[out[-1]]) < out[-1]:
        out.append(int(parent[out[-1]]))
    return out


def visible(parent, i, c, slot, window, n_sink):
    """Tokens that row i sees, ascending."""
    ln = line(parent, i)
    p = c + len(ln) - 1
    pos = {t: t for t in range(max(c, 0))}
    pos.update({c + a: c + len(line(parent, a)) - 1 for a in ln})
    return np.array(sorted(t for t, at in pos.items()
                           if 0 <= t < len(slot) and slot[t] >= 0 and (not window or at > p - window or at < n_sink)),
                    np.int64)


def attention(q_bits, pool_bits, table, page, row0, seq_len, parent, sm_scale, window=0, n_sink=0):
    """As paged.attention: out, lse, sum_t p_t |v_t|, largest sum_d |q_d k_d|."""
    T, H, _ = q_bits.shape
    scale = float(np.float32(sm_scale))
    out, absv = np.full((T, H, D_V), np.nan), np.full((T, H, D_V), np.nan)
    lse, mag = np.full((T, H), np.nan), np.full((T, H), np.nan)
    for b in range(len(seq_len)):
        r0, n, length = int(row0[b]), int(row0[b + 1]) - int(row0[b]), int(seq_len[b])
        sl = slots(table[b], page, len(pool_bits), max(length, 0))
        for i in range(n):
            r = r0 + i
            see = visible(parent[r0:r0 + n], i, length - n, sl, window, n_sink)
            if len(see) == 0:
                out[r], absv[r], lse[r], mag[r] = 0, 0, -np.inf, 0
                continue
            q, k = bf16_to_f64(q_bits[r]), bf16_to_f64(pool_bits[sl[see]])
            s = (q @ k.T) * scale
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            den = p.sum(axis=1, keepdims=True)
            out[r] = (p @ k[:, :D_V]) / den
            absv[r] = (p @ np.abs(k[:, :D_V])) / den
            lse[r] = (m + np.log(den))[:, 0]
            mag[r] = (np.abs(q) @ np.abs(k).T).max(axis=1) * abs(scale)
    return out, lse, absv, mag


def weights(logits, temperature):
    """Unnormalised probabilities of one row (the largest is 1). NaN weighs
    nothing, an infinite logit counts as the largest finite float; temperature 0,
    below or NaN: the first largest alone."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    top = x.max()
    if top == -np.inf:
        return np.zeros(len(x))
    if not temperature > 0:
        w = np.zeros(len(x))
        w[int(np.argmax(x))] = 1.0
        return w
    with np.errstate(invalid='ignore', over='ignore'):
        w = np.exp((x - top) / float(np.float32(temperature)))
    return np.where(x == -np.inf, 0.0, w)


def pick(w, u):
    """First token up to which more than u of the weight lies; -1 where nothing weighs."""
    if not w.sum() > 0:
        return -1
    cum = np.cumsum(w)
    return int(min(np.searchsorted(cum, float(u) * cum[-1], side='right'), np.flatnonzero(w)[-1]))


def verify(logits, tokens, row0, u, most, parent=None, draft=None, temperature=None):
    """Per sequence (kept rows, next token): from row 0 on, the first child that
    passes is followed until there is none or `most` rows are kept. `u` in [0,
    1). A decision that lies within 1e-9 of its border is reported: the fourth
    list says how near any came."""
    V, got = logits.shape[1], []
    for b in range(len(row0) - 1):
        r0, n = int(row0[b]), int(row0[b + 1]) - int(row0[b])
        if n == 0:
            got.append(([], -1, 1.0))
            continue
        temp = 1.0 if temperature is None else float(temperature[b])
        at, kept, near = 0, [0], 1.0
        while True:
            w = weights(logits[r0 + at], temp)
            left, moved = w.copy(), False
            if len(kept) < most:
                if parent is None:
                    kids = [at + 1] if at + 1 < n else []
                else:
                    kids = [i for i in range(1, n) if int(parent[r0 + i]) == at and at < i]
                for i in kids:
                    x = int(tokens[r0 + i])
                    mass = left[x] if 0 <= x < V else 0.0
                    if draft is None or not temp > 0:
                        bar = float(u[r0 + i]) * left.sum()
                        ok = mass > 0 and (bar < mass if temp > 0 else True)
                    else:
                        q = np.nan_to_num(np.maximum(np.asarray(draft[r0 + at], np.float64), 0), nan=0.0, posinf=np.inf)
                        bar = float(u[r0 + i]) * (q[x] if 0 <= x < V else 0.0) * left.sum()
                        ok = mass > 0 and bar < mass
                    if temp > 0 and mass > 0 and mass != bar:
                        near = min(near, abs(mass - bar) / max(mass, bar))
                    if ok:
                        at, moved = i, True
                        break
                    if draft is not None and temp > 0:
                        rest = np.maximum(left / left.sum() - q, 0) if left.sum() > 0 else left
                        left = rest if rest.sum() > 0 else left
                    elif temp > 0 and 0 <= x < V:
                        left[x] = 0.0
            if not moved:
                break
            kept.append(at)
        if temp > 0 and left.sum() > 0:
            aim = float(u[r0]) * left.sum()
            near = min(near, np.abs(np.cumsum(left) - aim).min() / left.sum())
        got.append((kept, pick(left, u[r0]), near))
    return [g[0] for g in got], [g[1] for g in got], [g[2] for g in got]


def accept(pool, table, page, row0, seq_len, kept):
    """Moves the kept rows in place; returns the new lengths."""
    out = []
    for b, rows in enumerate(kept):
        n = int(row0[b + 1]) - int(row0[b])
        c = int(seq_len[b]) - n
        sl = slots(table[b], page, len(pool), max(int(seq_len[b]), 0))
        src = [sl[c + a] if c + a >= 0 else -1 for a in rows]
        dst = [sl[c + j] if c + j >= 0 else -1 for j in range(len(rows))]
        new = {d: pool[s].copy() for s, d in zip(src, dst) if s >= 0 and d >= 0}
        for d, v in new.items():
            pool[d] = v
        out.append(c + len(rows))
    return out
