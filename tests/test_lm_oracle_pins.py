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


def test_distill_with_one_entry_is_cross_entropy():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 11))
    label = np.array([[4], [0], [10]])
    loss, lse, grad = lm.distill(x, label, rng.standard_normal((3, 1)), 1.0, np.ones(3))
    q = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    assert np.allclose(loss, -np.log(q[np.arange(3), label[:, 0]]))
    assert np.allclose(lse, np.log(np.exp(x).sum(1)))
    assert np.allclose(grad, q - (np.arange(11) == label))


def test_distill_against_dense_kl_and_its_minimum():
    rng = np.random.default_rng(3)
    V, tau = 6, 2.5
    t = rng.standard_normal((1, V))
    ids = rng.permutation(V)[None]
    x = rng.standard_normal((1, V))
    p, q = np.zeros(V), np.exp(x[0] / tau) / np.exp(x[0] / tau).sum()
    p[ids[0]] = np.exp(t[0] / tau) / np.exp(t[0] / tau).sum()
    loss, _, _ = lm.distill(x, ids, t, tau)
    assert np.isclose(loss[0], tau ** 2 * (p * np.log(p / q)).sum())
    same = np.zeros((1, V))
    same[0, ids[0]] = t[0] + 3.0  # the teacher's distribution itself
    loss, _, grad = lm.distill(same, ids, t, tau, np.ones(1))
    assert abs(loss[0]) < 1e-14 and np.abs(grad).max() < 1e-15


def test_distill_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 9))
    ids = np.array([[3, 3, 8, -1], [0, 9, 2, 5]])  # an index twice, padding, one past the end
    t = rng.standard_normal((2, 4))
    t[1, 3] = -np.inf
    g = np.array([0.7, -1.3])
    _, _, grad = lm.distill(x, ids, t, 1.7, g)
    eps = 1e-6
    for r in range(2):
        for v in range(9):
            xp, xm = x.copy(), x.copy()
            xp[r, v] += eps
            xm[r, v] -= eps
            num = (g * (lm.distill(xp, ids, t, 1.7)[0] - lm.distill(xm, ids, t, 1.7)[0])).sum()
            assert np.isclose(grad[r, v], num / (2 * eps), atol=1e-8)
    assert np.allclose(grad.sum(1), 0)  # probabilities and targets both sum to 1


def test_distill_empty_and_impossible_rows():
    x = np.array([[0.0, 1.0, -np.inf], [-np.inf, 0.5, 0.25]])
    ids = np.array([[-1, 2], [0, 1]])
    t = np.array([[1.0, -np.inf], [0.0, 0.0]])
    loss, _, grad = lm.distill(x, ids, t, 1.0, np.ones(2))
    assert loss[0] == 0 and not grad[0].any()       # no valid entry
    assert loss[1] == np.inf and grad[1, 0] == -0.5  # a target where the student has 0


def test_logits_process_by_hand():
    x = np.array([[2.0, -2.0, 1.0, 4.0, 4.0], [0.0, 0.0, 0.0, 0.0, 0.0]])
    hist = np.array([[0, 1, 1, -1, 9, 3], [2, 2, 2, 2, 2, 2]])
    out, best = lm.logits_process(x, hist, np.array([5, 0]), np.array([2.0, 2.0]),
                                  np.array([0.25, 1.0]), np.array([0.5, 1.0]),
                                  np.array([[2, 2, 9], [-1, 1, 1]]),
                                  np.array([[10.0, 99.0, 99.0], [99.0, -1.0, 99.0]]))
    #               2/2 - .5 - .25, -2*2 - 1 - .25, 1 + 10
    assert np.array_equal(out, [[0.25, -5.25, 11.0, 4.0, 4.0], [0.0, -1.0, 0.0, 0.0, 0.0]])
    assert best.tolist() == [2, 0]
    out, best = lm.logits_process(x, mask=np.array([[0b11010], [0]]))
    assert np.array_equal(out[0], [-np.inf, -2.0, -np.inf, 4.0, 4.0])
    assert best.tolist() == [3, -1]
    nan = np.array([[np.nan, 1.0, np.nan, 1.0]])
    assert lm.logits_process(nan)[1].tolist() == [1]


def test_w4_weights_by_hand():
    # bytes 0x2f 0x08: codes 15, 2, 8, 0; groups of 2
    q = np.array([[0x2f, 0x08], [0x00, 0xff]], dtype=np.uint8)
    s = np.array([[0.5, 2.0], [1.0, 0.25]])
    assert np.array_equal(lm.w4_weights(q, s, 2), [[3.5, -3.0, 0.0, -16.0], [-8, -8, 1.75, 1.75]])
    z = np.array([[15, 0], [1, 3]], dtype=np.uint8)
    assert np.array_equal(lm.w4_weights(q, s, 2, z), [[0.0, -6.5, 16.0, 0.0], [-1, -1, 3, 3]])
    x = np.array([[1.0, 0.0, 2.0, 0.0]])
    assert np.array_equal(lm.w4_linear(x, q, s, 2, bias=np.array([1.0, 2.0]),
                                       res=np.array([[0.5, 0.0]])), [[5.0, -2.5]])
