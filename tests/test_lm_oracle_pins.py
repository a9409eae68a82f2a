"""Pins of oracle/lm.py: each definition against something other than itself."""
import numpy as np

from oracle import lm


def test_embed_fwd_is_a_product_with_one_hot_rows():
    rng = np.random.default_rng(0)
    W = rng.standard_normal((7, 3))
    ids = np.array([0, 6, 3, 3, -1, 7, 2])
    one_hot = (ids[:, None] == np.arange(7)).astype(float)
    assert np.allclose(lm.embed_fwd(ids, W, 1.5), 1.5 * one_hot @ W, atol=1e-15)


def test_embed_bwd_is_the_adjoint_and_the_difference_quotient():
    rng = np.random.default_rng(1)
    W, dout = rng.standard_normal((5, 4)), rng.standard_normal((9, 4))
    ids = np.array([0, 4, 4, -1, 2, 2, 2, 9, 0])
    dW = lm.embed_bwd(ids, dout, 5, 0.3)
    # <dout, E W> = <E^T dout, W>
    assert np.isclose((dout * lm.embed_fwd(ids, W, 0.3)).sum(), (dW * W).sum())
    eps = 1e-6
    for v, c in ((0, 1), (2, 3), (3, 0), (4, 2)):
        Wp, Wm = W.copy(), W.copy()
        Wp[v, c] += eps
        Wm[v, c] -= eps
        num = (dout * (lm.embed_fwd(ids, Wp, 0.3) - lm.embed_fwd(ids, Wm, 0.3))).sum() / (2 * eps)
        assert np.isclose(dW[v, c], num, atol=1e-8)
