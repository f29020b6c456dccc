"""Plain definitions, in 64 bits, of what stands on the target's side of a round
(log probabilities of given tokens, the distillation loss and its gradient,
attention behind a shared prefix), for the tests.  They share no code with the
library."""
import math

import numpy as np

ROW_NAN, BAD_TOKEN, BAD_LEN, BAD_PAGE, BAD_ROW = 1, 2, 256, 512, 1024


def log_softmax(x, T):
    """ln softmax(x / T) of one row, or None where it has none."""
    z = np.asarray(x, np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return None
    z = (z - z.max()) / np.float64(np.float32(T))
    return z - np.log(np.exp(z).sum())


def token_logprobs(x, token, K, T):
    """One row: (logprob, entropy, top tokens, their log probabilities, status);
    token None: not asked for."""
    lp = log_softmax(x, T)
    bad = token is not None and not 0 <= token < len(x)
    if lp is None:
        return math.nan, math.nan, [-1] * K, [math.nan] * K, ROW_NAN | (BAD_TOKEN if bad else 0)
    p = np.exp(lp)
    H = -float(np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0), 0)))
    order = sorted(range(len(x)), key=lambda i: (-float(x[i]), i))[:K]
    order = [i for i in order if x[i] > -np.inf]
    top = order + [-1] * (K - len(order))
    top_lp = [float(lp[i]) for i in order] + [-math.inf] * (K - len(order))
    given = None if token is None else math.nan if bad else float(lp[token])
    return given, H, top, top_lp, BAD_TOKEN if bad else 0


def distill(x, token, value, T, tail):
    """One row: (loss, gradient without weight, status)."""
    x = np.asarray(x, np.float64)
    V = len(x)
    T = np.float64(np.float32(T))
    entries = [(int(t), float(a)) for t, a in zip(token, value) if t != -1]
    status = 0
    if any(t < 0 or t >= V for t, _ in entries):
        status |= BAD_TOKEN
    elif len({t for t, _ in entries}) < len(entries):
        status |= BAD_TOKEN
    if any(math.isnan(a) or a == math.inf for _, a in entries):
        status |= ROW_NAN
    if not entries:
        return 0.0, np.zeros(V), 0
    if not status & ROW_NAN:
        if tail and sum(math.exp(min(a, 50.0)) for _, a in entries) >= 1 + 2.0 ** -8:
            status |= ROW_NAN
        if not tail and all(a == -math.inf for _, a in entries):
            status |= ROW_NAN
    lp = log_softmax(x, T)
    if lp is None:
        status |= ROW_NAN
    if status:
        return math.nan, np.zeros(V), status
    idx = np.array([t for t, _ in entries])
    a = np.array([v for _, v in entries])
    lt = a if tail else a - a.max() - np.log(np.exp(a - a.max()).sum())
    t = np.exp(lt)
    s = np.exp(lp)
    rest = np.ones(V, bool)
    rest[idx] = False
    with np.errstate(divide="ignore", invalid="ignore"):
        loss = float(np.sum(np.where(t > 0, t * (lt - lp[idx]), 0.0)))
        grad = s.copy()
        if tail and rest.any():
            tr = max(0.0, float(-np.expm1(lt.max()) - (t.sum() - t.max())))
            r = lp[rest]
            lsr = r.max() + np.log(np.exp(r - r.max()).sum()) if (r > -np.inf).any() else -np.inf
            if tr > 0:
                loss += tr * (math.log(tr) - lsr)
            if lsr > -np.inf:
                grad[rest] = np.exp(r - lsr) * (math.exp(lsr) - tr)
    grad[idx] = s[idx] - t
    return loss, grad / T, 0


def prefix_attention(q, kv, ptable, plen, table, lens, scale):
    """q [B][Hq][D], kv [2][pages][page][Hkv][D]; (out, lse, status)."""
    B, Hq, D = q.shape
    _, P, page, Hkv, _ = kv.shape
    N, G = len(plen), Hq // Hkv
    W = B // N
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    status = np.zeros(B, np.int64)
    for b in range(B):
        rows = []
        for tab, n in ((ptable[b // W], int(plen[b // W])), (table[b], int(lens[b]))):
            if not 0 <= n <= len(tab) * page:
                status[b] |= BAD_LEN
                continue
            ids = [int(tab[j // page]) for j in range(n)]
            if any(not 0 <= i < P for i in ids):
                status[b] |= BAD_PAGE
                continue
            rows.append(np.array([kv[:, i, j % page] for j, i in enumerate(ids)],
                                 np.float64).reshape(n, 2, Hkv, D))
        if status[b]:
            out[b], lse[b] = np.nan, np.nan
            continue
        rows = np.concatenate(rows)
        if not len(rows):
            continue
        for h in range(Hq):
            s = rows[:, 0, h // G] @ q[b, h].astype(np.float64) * scale
            m = s.max()
            e = np.exp(s - m)
            lse[b, h] = m + math.log(e.sum())
            out[b, h] = e @ rows[:, 1, h // G] / e.sum()
    return out, lse, status
