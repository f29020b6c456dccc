"""Plain definitions, in 64 bits or exact integers, of the serving operators
(verification from probabilities, paged decode attention, cache eviction), for
the tests.  They share no code with the library."""
from fractions import Fraction

import numpy as np

ROW_NAN, BAD_TOKEN, RESID_ZERO, P_ZERO = 1, 2, 4, 8
BAD_RAND, BAD_LEN, BAD_PAGE = 128, 256, 512


# ------------------------------------------------- verification from probabilities
def _weights(w):
    """floor(w 2^62) of an fp32 array with 0 <= w < 2, as Python integers."""
    m, e = np.frexp(w.astype(np.float64))
    m24 = np.ldexp(m, 24).astype(np.int64)       # exact: fp32 has 24 bits
    sh = e.astype(np.int64) + 38                 # w 2^62 = m24 2^(e - 24 + 62)
    return [int(a) << int(s) if s >= 0 else int(a) >> int(-s) for a, s in zip(m24, sh)]


def _draw(w, u):
    """First k whose inclusive sum of weights exceeds u * total, exactly."""
    W = _weights(w)
    total = sum(W)
    if total == 0:
        return None
    t = Fraction(float(u)) * total
    run = 0
    for k, x in enumerate(W):
        run += x
        if run > t:
            return k
    raise AssertionError("u outside [0, 1)")


def _bad(x):
    return not (x >= 0 and x < 2)


def verify_one(q, p, d, ua, us):
    """One sequence: q [n+1][V], p [n][V] or None, d [n], ua [n], us; fp32 arrays.
    Returns (tokens, accept_len, status): tokens has accept_len + 1 entries, or
    none on a fault."""
    n, V = len(d), q.shape[1]
    status = 0
    a = n
    for i in range(n):
        if _bad_rand(ua[i]):
            status |= BAD_RAND
        if not 0 <= d[i] < V:
            return [], 0, status | BAD_TOKEN | (BAD_RAND if _bad_rand(us) else 0)
        qd = q[i, d[i]]
        pd = p[i, d[i]] if p is not None else np.float32(1)
        if _bad(qd) or _bad(pd):
            status |= ROW_NAN
        if pd == 0:
            status |= P_ZERO
        if status & (ROW_NAN | BAD_RAND):
            return [], 0, status | (BAD_RAND if _bad_rand(us) else 0)
        if pd != 0 and not Fraction(float(ua[i])) * Fraction(float(pd)) < Fraction(float(qd)):
            a = i
            break
    if _bad_rand(us):
        return [], 0, status | BAD_RAND
    row = q[a].astype(np.float32)
    sub = None
    if a < n:
        if p is not None:
            sub = p[a].astype(np.float32)
        else:
            sub = np.zeros(V, np.float32)
            sub[d[a]] = 1
    rows = [row] if sub is None or p is None else [row, sub]
    if any(not np.all((r >= 0) & (r < 2)) for r in rows):
        return [], 0, status | ROW_NAN
    w = row if sub is None else np.maximum(row - sub, np.float32(0))
    if sub is not None and sum(_weights(w)) == 0:
        status |= RESID_ZERO
        w = row
    if w.astype(np.float64).sum() >= 2:
        return [], 0, status | ROW_NAN
    k = _draw(w, us)
    if k is None:
        return [], 0, status | ROW_NAN
    return [int(x) for x in d[:a]] + [k], a, status


def _bad_rand(u):
    return not (u >= 0 and u < 1)


def verify_probs(q, p, d, ua, us, n=None):
    """The batch: tokens [B][N+1] (-1 after the last), accept_len, status."""
    B, R, _ = q.shape
    N = R - 1
    tokens = np.full((B, R), -1, np.int32)
    alen, status = np.zeros(B, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        k = N if n is None else int(n[b])
        if not 0 <= k <= N:
            status[b] = BAD_LEN | (BAD_RAND if _bad_rand(us[b]) else 0)
            continue
        t, a, s = verify_one(q[b, :k + 1], None if p is None else p[b, :k], d[b, :k], ua[b, :k], us[b])
        tokens[b, :len(t)] = t
        alen[b], status[b] = a, s
    return tokens, alen, status


# ------------------------------------------------------- paged decode attention
def visible_slots(n, window, sinks):
    j = np.arange(n)
    return j[(j >= n - window) | (j < sinks)] if window else j


def paged_attention(q, kv, table, lens, scale, window=0, sinks=0):
    """q [B][Hq][D], kv [2][P][page][Hkv][D], both float64; returns out, lse,
    the weight each slot received [B][Hkv][cap], and per (b, h) the bound
    max_j scale sum_d |q_d k_d| that error bounds are made of."""
    B, Hq, D = q.shape
    page, Hkv = kv.shape[2], kv.shape[3]
    G = Hq // Hkv
    cap = table.shape[1] * page
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    got, size = np.zeros((B, Hkv, cap)), np.zeros((B, Hq))
    for b in range(B):
        j = visible_slots(int(lens[b]), window, sinks)
        if not len(j):
            continue
        k, v = kv[0][table[b, j // page], j % page], kv[1][table[b, j // page], j % page]
        for h in range(Hq):
            s = scale * (k[:, h // G] @ q[b, h])
            size[b, h] = scale * (np.abs(k[:, h // G]) @ np.abs(q[b, h])).max()
            m = s.max()
            if m == -np.inf:
                continue
            e = np.exp(s - m)
            l = e.sum()
            lse[b, h] = m + np.log(l)
            out[b, h] = (e / l) @ v[:, h // G]
            got[b, h // G, j] += e / l
    return out, lse, got, size


# -------------------------------------------------------------------- eviction
def kept_slots(w, n, budget, sinks, recent):
    """The slots kept of one (layer, sequence, head): w its weights."""
    if n <= budget:
        return list(range(n))
    def place(j):
        x = w[j]
        return (1, 0.0, j) if x != x else (0, -float(x), j)
    mid = sorted(range(sinks, n - recent), key=place)[:budget - sinks - recent]
    return list(range(sinks)) + sorted(mid) + list(range(n - recent, n))


def kv_evict(kv, table, lens, w, budget, sinks, recent):
    """kv [L][2][P][page][H][D] (any dtype), w [L][B][H][S]: copies of both
    after the eviction, the kept slots and the new lengths."""
    kv, w = kv.copy(), w.copy()
    L, B, H, _ = w.shape
    page = kv.shape[3]
    kept = np.full((L, B, H, budget), -1, np.int32)
    for b in range(B):
        n = int(lens[b])
        for l in range(L):
            for h in range(H):
                k = np.array(kept_slots(w[l, b, h], n, budget, sinks, recent), np.int64)
                kept[l, b, h, :len(k)] = k
                if n > budget:
                    to = np.arange(budget)
                    rows = kv[l][:, table[b, k // page], k % page, h].copy()
                    kv[l][:, table[b, to // page], to % page, h] = rows
                    w[l, b, h, :budget] = w[l, b, h, k]
                    w[l, b, h, budget:n] = 0
    return kv, w, kept, np.minimum(lens, budget).astype(np.int32)
