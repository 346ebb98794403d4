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
