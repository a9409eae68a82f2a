"""Pins of oracle/lm.py's distillation at the ends of the logits' range and for rows of NaN."""
import numpy as np

from oracle import lm


def test_distill_of_a_row_of_one_value_is_uniform_whatever_the_value():
    ids, t = np.array([[3, 4]]), np.zeros((1, 2))
    for v in (0.0, 5.0, float(np.finfo(np.float32).min), float(np.finfo(np.float32).max)):
        loss, _, grad = lm.distill(np.full((1, 10), v), ids, t, 1.0, np.ones(1))
        assert np.isclose(loss[0], np.log(5.0))  # log(1/2) - log(1/10)
        want = np.full(10, 0.1)
        want[[3, 4]] -= 0.5
        assert np.allclose(grad[0], want)


def test_distill_of_a_row_with_nan_is_nan_and_of_minus_infinity_has_no_probability():
    x = np.full((2, 6), -np.inf)
    x[0, 1] = np.nan
    ids, t = np.array([[2, 4]] * 2), np.zeros((2, 2))
    loss, lse, grad = lm.distill(x, ids, t, 1.0, np.ones(2))
    assert np.isnan(loss[0]) and np.isnan(lse[0]) and np.isnan(grad[0]).all()
    assert loss[1] == np.inf and lse[1] == -np.inf
    assert np.array_equal(grad[1], [0, 0, -0.5, 0, -0.5, 0])
