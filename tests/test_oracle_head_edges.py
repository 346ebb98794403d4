"""Pins of oracle/head.py where rows are out of the ordinary (CPU)."""
import numpy as np

from oracle import head

INF = float("inf")


def test_log_sum_exp_of_infinities():
    """+inf makes it +inf, a NaN anywhere NaN, none but -inf -inf; ordinary
    rows beside them are not touched."""
    z = np.array([[1.0, INF, 2.0], [INF, -INF, INF], [INF, np.nan, 0.0], [-INF, -INF, -INF], [0.0, 0.0, -INF]])
    values, index, lse = head.top_logits(z, 2, 0.5)
    assert lse[0] == INF and lse[1] == INF and np.isnan(lse[2]) and lse[3] == -INF
    assert abs(lse[4] - np.log(2.0)) < 1e-15
    assert list(index[0]) == [1, 2] and list(index[1]) == [0, 2] and list(index[2]) == [1, 0]
    assert values[0, 0] == INF and values[0, 1] == 2.0


def test_mass_far_below_the_largest_logit():
    """Two columns off the list, gap below the one on it: log q_r = -gap / T +
    log(1 + e^(-1 / T)) to what e^-gap leaves, at any gap; the gradient off the list
    shares -w T r, and each row of it sums to 0."""
    T, r, w = 0.5, 0.25, 3.0
    for gap in (2.0, 40.0, 500.0, 20000.0):
        s = np.array([[gap, 0.0, -1.0]])
        val, idx = np.array([[T * np.log(1.0 - r)]]), np.array([[0]])
        loss, grad, stats = head.distill(s, val, idx, np.zeros(1), T, np.array([w]))
        e = np.exp(-1.0 / T)
        log_on = -np.log1p(np.exp(-gap / T) * (1.0 + e))
        log_off = -gap / T + np.log1p(e) + log_on
        want = w * T * T * ((1 - r) * (np.log(1 - r) - log_on) + r * (np.log(r) - log_off))
        assert abs(loss[0] - want) <= 1e-12 * want
        assert abs(stats[0, 2] - log_off) <= 1e-12 * abs(log_off)
        q_off = np.exp(log_off) * np.array([1.0, e]) / (1.0 + e)
        g_off = w * T * (q_off - r * np.array([1.0, e]) / (1.0 + e))
        assert np.all(np.abs(grad[0, 1:] - g_off) <= 1e-12)
        assert abs(grad.sum()) <= 1e-12


def test_stats_do_not_go_by_the_weight():
    rng = np.random.default_rng(2)
    s = rng.normal(0, 2, (3, 20))
    val, idx, lse = head.top_logits(s + rng.normal(0, 1, s.shape), 4)
    a = head.distill(s, val, idx, lse, 1.0, np.array([0.0, 1.0, 0.5]))
    b = head.distill(s, val, idx, lse, 1.0)
    np.testing.assert_array_equal(a[2], b[2])
    assert a[0][0] == 0 and not a[1][0].any() and b[0][0] != 0
