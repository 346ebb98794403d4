"""Pins of the oracle's 8-bit product, top logits and distillation (CPU):
hand-worked values, closed forms, and the gradient against differences."""
import numpy as np
import pytest

from oracle import head


def test_quantize_rows_by_hand():
    # scale 2 / 127: 1 lies at 63.5 steps, a tie that goes to the even 64
    c, s, total = head.quantize_rows(np.array([[2.0, -2.0, 1.0, 0.0], [0, 0, 0, 0]], np.float32))
    assert c.tolist() == [[127, -127, 64, 0], [0, 0, 0, 0]]
    assert s[0] == np.float32(2.0) / np.float32(127) and s[1] == 0
    assert total.tolist() == [64, 0]


def test_quantize_rows_clips_and_marks_what_is_not_finite():
    c, s, _ = head.quantize_rows(np.array([[127.0, 64.0, -127.0]], np.float32), clip=0.5)
    assert s[0] == 0.5 and c.tolist() == [[127, 127, -127]]
    for bad in (np.nan, np.inf, -np.inf):
        c, s, _ = head.quantize_rows(np.array([[1.0, bad]], np.float32))
        assert np.isnan(s[0]) and not c.any()


def test_product_by_hand():
    y, acc = head.product(np.array([[1, -2]]), np.array([0.5], np.float32), [[3, 4], [5, -6]], [2.0, 1.0],
                          w_zero=[1, -1], bias=[10.0, 0.0])
    assert acc.tolist() == [[1 * 2 - 2 * 3, 1 * 6 + 2 * 5]]
    assert y.tolist() == [[-4 * 0.5 * 2 + 10, 16 * 0.5]]


def test_top_logits_by_hand():
    v, i, lse = head.top_logits([[1.0, 3.0, 3.0, -np.inf, 0.0, -0.0]], 6)
    assert i.tolist() == [[1, 2, 0, 4, 5, 3]]
    assert v[0, :3].tolist() == [3.0, 3.0, 1.0]
    assert abs(lse[0] - np.log(np.e + 2 * np.e ** 3 + 2)) < 1e-14
    v, i, _ = head.top_logits([[1.0, np.nan, np.inf]], 2)
    assert i.tolist() == [[1, 2]]


def test_distill_of_the_teacher_itself_is_zero():
    rng = np.random.default_rng(0)
    s = rng.normal(0, 2, (3, 40))
    v, i, lse = head.top_logits(s, 7, 1.5)
    loss, grad, _ = head.distill(s, v, i, lse, 1.5)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12
    # renormalised over the whole vocabulary: the same divergence
    v, i, _ = head.top_logits(s, 40, 1.5)
    loss, grad, _ = head.distill(s, v, i, None, 1.5)
    assert np.abs(loss).max() < 1e-12 and np.abs(grad).max() < 1e-12


def test_distill_by_hand():
    # one listed column of two, p = 1/4 on it, the student at q = 1/2
    loss, grad, stats = head.distill([[0.0, 0.0]], [[np.log(0.25)]], [[0]], [0.0])
    assert abs(loss[0] - (0.25 * np.log(0.5) + 0.75 * np.log(1.5))) < 1e-15
    assert np.allclose(grad, [[0.25, -0.25]], atol=1e-15)
    assert np.allclose(stats, [[0.0, np.log(2), -np.log(2)]], atol=1e-15)
    # renormalised, the one column has all of it
    loss, grad, _ = head.distill([[0.0, 0.0]], [[-3.0]], [[0]], None, 2.0, [0.5])
    assert abs(loss[0] - 0.5 * 4 * np.log(2)) < 1e-15
    assert np.allclose(grad, [[-0.5, 0.5]], atol=1e-15)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 2.0])
def test_gradient_against_differences(rest, temperature):
    rng = np.random.default_rng(3)
    n, v, k = 4, 23, 6
    t = rng.normal(0, 2, (n, v))
    s = t + rng.normal(0, 1, (n, v))
    val, idx, lse = head.top_logits(t, k, temperature)
    idx[1, 4:] = -1          # a short list
    idx[2, :] = -1           # an empty one
    idx[3, 1] = idx[3, 0]    # a column twice
    w = rng.uniform(0.5, 2, n)
    args = (val, idx, lse if rest else None, temperature, w)
    _, grad, _ = head.distill(s, *args)
    h = 1e-6
    for i in range(n):
        for j in range(v):
            up, dn = s.copy(), s.copy()
            up[i, j] += h
            dn[i, j] -= h
            d = (head.distill(up, *args)[0][i] - head.distill(dn, *args)[0][i]) / (2 * h)
            # central differences: h^2 of the third derivative, and 1e-16 / h of rounding
            assert abs(d - grad[i, j]) < 2e-8, (i, j)


def test_rows_that_say_nothing():
    s = np.array([[-np.inf, -np.inf], [np.nan, 1.0], [0.0, -np.inf]])
    loss, grad, _ = head.distill(s, [[1.0], [1.0], [1.0]], [[0], [0], [1]], None, 1.0, [1, 0, 1])
    assert loss[0] == np.inf and grad[0].tolist() == [-1.0, 0.0]
    assert loss[1] == 0 and not grad[1].any()          # no weight: not looked at
    assert loss[2] == np.inf and grad[2].tolist() == [1.0, -1.0]


def test_huge_logits_keep_their_differences():
    """Logits at the lowest fp32 value: the distribution is uniform."""
    low = float(np.finfo(np.float32).min)
    loss, grad, stats = head.distill(np.full((1, 4), low), [[0.0]], [[1]])
    assert abs(loss[0] - np.log(4)) < 1e-15
    assert np.allclose(grad, [[0.25, -0.75, 0.25, 0.25]], atol=1e-15)
    assert stats[0, 0] == low and abs(stats[0, 1] - np.log(4)) < 1e-15
