"""CPU pins of tests/plain_distill_mass.py: differences of its loss, and the plain
definition where both say the same."""
import math

import numpy as np
import pytest

import plain_distill_mass as mass
import plain_target as plain


def row(V, K, seed, total=None, low=None, noise=1.0):
    """Logits, a list and its values, which add up to `total`; with `low`, all that is
    not listed is that."""
    g = np.random.default_rng(seed)
    x = g.standard_normal(V) * 2
    y = x + noise * g.standard_normal(V)
    token = np.argsort(-y)[:K]
    if low is not None:
        y[np.setdiff1d(np.arange(V), token)] = -np.inf
        x[np.setdiff1d(np.arange(V), token)] = low
    value = y[token] - np.log(np.exp(y).sum())
    if total is not None:
        value += math.log(total) - math.log(np.exp(value).sum())
    return x, token, value


@pytest.mark.parametrize("tail", [True, False])
@pytest.mark.parametrize("T", [1.0, 0.75])
@pytest.mark.parametrize("V,K,total", [(12, 4, None), (12, 4, 1 + 2.0 ** -9), (12, 12, None), (12, 12, 1 + 2.0 ** -9),
                                       (5, 1, 0.4), (9, 3, 1 - 2.0 ** -18)])
def test_gradient_against_differences(V, K, total, T, tail):
    """A step of 1e-4: third derivatives below 1 / T^3, and logs of below 20 in 64 bits."""
    x, token, value = row(V, K, V + K, total)
    _, grad, st = mass.definition(x, token, value, T, tail)
    assert st == 0
    h = 1e-4
    for v in range(V):
        a, b = x.copy(), x.copy()
        a[v] += h
        b[v] -= h
        d = (mass.definition(a, token, value, T, tail)[0] - mass.definition(b, token, value, T, tail)[0]) / (2 * h)
        # (a list of all of V that sums to less than 1 by rounding: t_r counts as 0, up to 2^-16)
        assert abs(d - grad[v]) <= 1e-8 + 20 * 2.0 ** -52 / h, v


def test_as_the_plain_definition_with_a_rest():
    for seed in range(20):
        for tail in (True, False):
            x, token, value = row(30, 6, seed)
            a, b = mass.definition(x, token, value, 1.3, tail), plain.distill(x, token, value, 1.3, tail)
            assert abs(a[0] - b[0]) <= 1e-12 and np.abs(a[1] - b[1]).max() <= 1e-12 and a[2] == b[2] == 0
    for token, value in (([3, 3], [-1.0, -2.0]), ([3, 30], [-1.0, -2.0]), ([3, 4], [math.nan, -1.0]), ([3, 4], [-0.1, -0.2]),
                         ([-1, -1], [0.0, 0.0])):
        a, b = mass.definition(x, token, value, 1.0, True), plain.distill(x, token, value, 1.0, True)
        assert np.array_equal(a[0], b[0], equal_nan=True) and np.array_equal(a[1], b[1]) and a[2] == b[2]


@pytest.mark.parametrize("low", [-math.inf, -3.4028234663852886e38, -80.0])
def test_a_rest_without_a_share(low):
    """What rounding leaves of the teacher's mass is nothing; what is more is not."""
    for total, finite in ((1 - 2.0 ** -18, True), (1.0, True), (1 + 2.0 ** -18, True), (1 - 2.0 ** -14, False)):
        x, token, value = row(20, 5, 1, total, low)
        loss, grad, _ = mass.definition(x, token, value, 1.0, True)
        lp = x[token] - np.log(np.exp(x[token]).sum())
        kl = float(np.sum(np.exp(value) * (value - lp)))
        if finite:
            assert abs(loss - kl) <= 1e-12 and np.abs(grad).sum() < 2
            assert np.abs(np.delete(grad, token)).max() <= 2.0 ** -100
        else:
            assert loss == math.inf if low == -math.inf else loss - kl > 2.0 ** -14 * (80 - 10)
