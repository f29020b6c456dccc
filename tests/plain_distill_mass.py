"""The distillation loss where the teacher's weights and the student's
probabilities do not meet as a list and its rest usually do -- a rest that a mask
leaves nothing of, a list of the whole vocabulary, weights that add up to more
than 1 -- in 64 bits, for the tests.  Shares no code with the library."""
import math

import numpy as np

ROW_NAN, BAD_TOKEN = 1, 2
NO_SHARE, ROUNDING = 2.0 ** -100, 2.0 ** -16


def masses(value, tail):
    """t_k and t_r of a list's values."""
    a = np.asarray(value, np.float64)
    if not tail:
        e = np.exp(a - a.max())
        return e / e.sum(), 0.0
    t = np.exp(a)
    top = int(a.argmax())
    return t, max(0.0, float(-np.expm1(a[top]) - np.delete(t, top).sum()))


def definition(x, token, value, T, tail):
    """One row: (loss, gradient without weight, status)."""
    x = np.asarray(x, np.float64)
    V, T = len(x), np.float64(np.float32(T))
    entries = [(int(t), float(a)) for t, a in zip(token, value) if t != -1]
    if not entries:
        return 0.0, np.zeros(V), 0
    status = 0
    if any(not 0 <= t < V for t, _ in entries) or len({t for t, _ in entries}) < len(entries):
        status |= BAD_TOKEN
    values = np.array([a for _, a in entries])
    if np.isnan(values).any() or (values == np.inf).any():
        status |= ROW_NAN
    elif tail and np.exp(np.minimum(values, 50.0)).sum() >= 1 + 2.0 ** -8 or not tail and (values == -np.inf).all():
        status |= ROW_NAN
    if np.isnan(x).any() or (x == np.inf).any() or (x == -np.inf).all():
        status |= ROW_NAN
    if status:
        return math.nan, np.zeros(V), status
    z = (x - x.max()) / T
    lp = z - np.log(np.exp(z).sum())
    s = np.exp(lp)
    idx = np.array([t for t, _ in entries])
    t, tr = masses(values, tail)
    rest = np.ones(V, bool)
    rest[idx] = False
    lsr = -np.inf  # ln of the rest's share
    if (lp[rest] > -np.inf).any():
        top = lp[rest].max()
        of_rest = np.exp(lp[rest] - top)
        lsr = top + np.log(of_rest.sum())
        of_rest /= of_rest.sum()  # (as ln: lost beside a mask of -3e38)
    if tr < ROUNDING and lsr < math.log(NO_SHARE):
        tr = 0.0
    total = max(1.0, float(t.sum())) if tail else 1.0
    lt = values if tail else values - values.max() - np.log(np.exp(values - values.max()).sum())
    with np.errstate(divide="ignore", invalid="ignore"):
        loss = float(np.sum(np.where(t > 0, t * (lt - lp[idx]), 0.0)))
    if tr > 0:
        loss += tr * (math.log(tr) - lsr)
    grad = np.zeros(V)
    if lsr > -np.inf:
        grad[rest] = of_rest * (np.exp(lsr) * total - tr)
    grad[idx] = s[idx] * total - t
    return loss, grad / T, 0
