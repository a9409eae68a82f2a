"""GPU parity of the distillation loss and its gradient against the fp64 definition.

Tolerances, derived before the first run.  u = 2^-24.  An exponent x - m is
formed from one product with 1/tau (itself rounded: |x| u) and one subtraction,
then scaled by log2 e: its absolute error is at most about 3 u max|x/tau| +
2 u |x - m|, below 8 u X with X = max|x/tau| + 1, and the hardware exponential
adds 2 u relative.  lse inherits that plus its own rounding and a sum of
positive terms (log2 V + V/512 additions deep, each u relative, through the
logarithm absolute): |lse error| <= u (10 X + 32 + V/512).  A loss term p_j
(log p_j - log q_j) has that error and the same for the teacher's side, and
weights that sum to 1: |loss error| <= tau^2 u (30 X' + 64 + V/512) with X' also
over the teacher's values, plus the rounding of p against the size of the gaps,
16 u max|gap| tau^2.  The gradient's q has relative error e_q = u (20 X + 64 +
V/512), p the same with X', so |err| <= |g| tau (q e_q + p e_q) + the io rounding
(2^-8 relative for bf16) of the result.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32_dev, host, to_dev
from oracle import lm
from selective_state_space_naju_amd import binding as nb
from selective_state_space_naju_amd import inputs

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev())


def draw(R, V, k, io, seed, lists="ragged"):
    rng = np.random.default_rng(seed)
    x = 2.5 * rng.standard_normal((R, V), dtype=np.float32)
    x = inputs.bf16_round(x) if io == "bf16" else x
    ids = rng.integers(0, V, (R, k))  # (repeats happen)
    t = (3 * rng.standard_normal((R, k))).astype(np.float32)
    if lists == "ragged":
        gone = rng.random((R, k)) < 0.3
        ids = np.where(gone & (rng.random((R, k)) < 0.5), rng.choice([-1, -5, V, V + 9], (R, k)), ids)
        t = np.where(gone & (rng.random((R, k)) < 0.5), np.float32(-np.inf), t)
        ids[R // 2] = -1  # a row without entries
    elif lists == "same":  # every entry names one token
        ids[:] = V - 1
    g = rng.standard_normal(R).astype(np.float32)
    if R > 3:
        g[1] = 0.0
    return x, ids, t, g


def bounds(x, ids, t, tau, g, io):
    """(loss bound, lse bound, gradient bound) as derived above."""
    V = x.shape[1]
    loss, lse, grad = lm.distill(x, ids, t, tau, g)
    ok = (ids >= 0) & (ids < V) & (t != -np.inf)
    # (logits whose probability is below e^-200 add nothing, whatever their size)
    near = x.astype(np.float64) > x.max(1, keepdims=True).astype(np.float64) - 200 * tau
    X = np.abs(np.where(near & np.isfinite(x), x, 0)).astype(np.float64).max(1) / tau + 1
    Xt = np.abs(np.where(ok & np.isfinite(t), t, 0)).astype(np.float64).max(1, initial=0) / tau + X
    b_lse = U * (10 * X + 32 + V / 512)
    gap = np.abs(lse) + X + Xt + 7
    b_loss = tau * tau * U * (30 * Xt + 64 + V / 512 + 16 * gap)
    e_q = U * (20 * Xt + 64 + V / 512)
    with np.errstate(all="ignore"):
        q = np.exp(np.where(x == -np.inf, -np.inf, x.astype(np.float64) / tau - lse[:, None]))
    size = 2 * q + np.abs(grad) / np.maximum(np.abs(g) * tau, 1e-30)[:, None]  # >= q + p
    io_u = 2.0 ** -8 if io == "bf16" else 2.0 ** -22
    # (bf16 results below its smallest normal number keep an absolute rounding)
    b_grad = (np.abs(g) * tau * e_q)[:, None] * size + io_u * np.abs(grad) + 2.0 ** -133
    return loss, lse, grad, b_loss, b_lse, b_grad


def check(name, got, ref, bound):
    got, ref = np.asarray(got), np.asarray(ref)
    same = np.isfinite(ref)
    assert np.array_equal(np.isfinite(got), same), name
    assert np.array_equal(got[~same], ref[~same], equal_nan=True), name
    bound = np.broadcast_to(bound, ref.shape)
    err = np.abs(got[same] - ref[same]) / bound[same]
    worst = err.max() if err.size else 0.0
    print("  %s: worst error %.3f of the bound" % (name, worst), flush=True)
    assert worst <= 1.0, name


def run_all(x, ids, t, tau, g, io, pad=0):
    """(loss, lse, gradient) by forward and backward, and (loss, gradient) by the joint call."""
    R, V = x.shape
    wide = np.full((R, V + pad), np.nan, dtype=np.float32)
    wide[:, :V] = x
    X = to_dev(wide, io)[:, :V]
    I, T, G = i32(ids), f32_dev(t), f32_dev(g)
    loss, lse = nb.distill_fwd(X, I, T, tau)
    out = torch.full((R, V + pad), 7.0, dtype=X.dtype, device=dev())
    grad = nb.distill_bwd(X, I, T, lse, G, tau, dlogits=out[:, :V])
    loss2, grad2 = nb.distill_fwd_bwd(X, I, T, G, tau)
    torch.cuda.synchronize()
    assert (out[:, V:] == 7.0).all()  # nothing past the vocabulary is written
    return host(loss), host(lse), host(grad), host(loss2), host(grad2)


CASES = [  # rows, vocab, k, io, tau, pad, lists
    (1, 1, 1, "f32", 1.0, 0, "full"),
    (1, 7, 3, "bf16", 2.0, 0, "full"),
    (5, 33, 4, "f32", 1.5, 3, "ragged"),
    (4, 1000, 64, "bf16", 1.0, 1, "ragged"),
    (3, 2047, 5, "f32", 4.0, 0, "ragged"),
    (3, 4096, 65, "bf16", 2.0, 0, "full"),
    (3, 4097, 512, "bf16", 0.5, 7, "ragged"),
    (4, 8193, 17, "f32", 1.0, 0, "same"),
    (2, 10007, 300, "f32", 2.0, 57, "full"),
    (4, 16385, 33, "bf16", 1.0, 0, "ragged"),
    (2, 32769, 1, "bf16", 1.0, 0, "full"),
    (4, 50001, 128, "bf16", 2.0, 0, "ragged"),
    (2, 65537, 40, "f32", 1.0, 1, "full"),
    (4, 65600, 40, "f32", 2.0, 0, "ragged"),
    (2, 131072, 64, "bf16", 1.0, 0, "full"),
    (2, 131073, 64, "bf16", 1.0, 0, "same"),
    (2, 200003, 2, "bf16", 3.0, 0, "full"),
    (700, 300, 9, "bf16", 1.0, 0, "ragged"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "r%d_v%d_k%d_%s_tau%g_pad%d_%s" % c)
def test_distill(case):
    R, V, k, io, tau, pad, lists = case
    print("distill", case, flush=True)
    x, ids, t, g = draw(R, V, k, io, 11, lists)
    loss, lse, grad, b_loss, b_lse, b_grad = bounds(x, ids, t, tau, g, io)
    got = run_all(x, ids, t, tau, g, io, pad)
    check("loss", got[0], loss, b_loss)
    check("lse", got[1], lse, b_lse)
    check("gradient", got[2], grad, b_grad)
    check("loss (joint)", got[3], loss, b_loss)
    check("gradient (joint)", got[4], grad, b_grad)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("V", [40, 5000, 70000])
def test_distill_masked_vocabulary_and_extremes(io, V):
    """-inf and the type's lowest value among the logits, rows of nothing but them, rows of one
    finite logit, large offsets, targets without student probability."""
    rng = np.random.default_rng(12)
    R, k = 8, 6
    low = inputs.bf16_round(np.array([-3.3895e38], np.float32))[0] if io == "bf16" else \
        np.finfo(np.float32).min
    x = 2 * rng.standard_normal((R, V)).astype(np.float32)
    ids = np.stack([rng.permutation(V)[:k] for _ in range(R)])
    t = rng.standard_normal((R, k)).astype(np.float32)
    x[0, rng.random(V) < 0.5] = -np.inf
    x[0, ids[0]] = 1.0
    x[1, rng.random(V) < 0.5] = low
    x[1, ids[1]] = 0.5
    x[2] = -np.inf
    x[3] = -np.inf
    x[3, ids[3, 0]] = 2.0
    t[3, 1:] = -np.inf
    x[4] += 3000.0
    x[5] -= 20000.0
    x[6, ids[6, 2]] = -np.inf
    t[7, 0] = 300.0  # the other probabilities underflow
    x = inputs.bf16_round(x) if io == "bf16" else x
    g = np.linspace(0.5, 1.5, R).astype(np.float32)
    print("distill extremes", io, V, flush=True)
    loss, lse, grad, b_loss, b_lse, b_grad = bounds(x, ids, t, 1.0, g, io)
    assert loss[2] == np.inf and loss[6] == np.inf and np.isfinite(loss[[0, 1, 3, 4, 5, 7]]).all()
    got = run_all(x, ids, t, 1.0, g, io)
    for n, (a, ref, b) in enumerate(((got[0], loss, b_loss), (got[1], lse, b_lse),
                                     (got[2], grad, b_grad), (got[3], loss, b_loss),
                                     (got[4], grad, b_grad))):
        check("output %d" % n, a, ref, b)


def test_distill_nan_stays_in_its_row():
    x = torch.randn(4, 3000, device=dev())
    x[1, 17] = float("nan")
    x[2, 5] = float("inf")
    ids = i32(np.arange(12).reshape(4, 3) + 100)
    t = torch.randn(4, 3, device=dev())
    t[3, 1] = float("nan")
    g = torch.ones(4, device=dev())
    for out in (nb.distill_fwd(x, ids, t)[0], nb.distill_fwd_bwd(x, ids, t, g)[0]):
        assert torch.isnan(out[1:]).all() and torch.isfinite(out[0])
    loss, grad = nb.distill_fwd_bwd(x, ids, t, g)
    assert torch.isfinite(grad[0]).all() and torch.isnan(grad[1]).all()
    g[1:] = 0.0  # rows that do not count
    loss, grad = nb.distill_fwd_bwd(x, ids, t, g)
    assert not grad[1:].any()
    _, lse = nb.distill_fwd(x, ids, t)
    assert not nb.distill_bwd(x, ids, t, lse, g)[1:].any()


def test_distill_a_list_of_nan_reaches_loss_and_gradient():
    x = torch.randn(2, 4000, device=dev())
    ids, one = i32([[5, 77], [9, -1]]), torch.ones(2, device=dev())
    t = torch.tensor([[float("nan")] * 2, [0.5, 0.0]], device=dev())
    loss, grad = nb.distill_fwd_bwd(x, ids, t, one)
    _, lse = nb.distill_fwd(x, ids, t)
    for d in (grad, nb.distill_bwd(x, ids, t, lse, one)):
        assert torch.isnan(d[0, [5, 77]]).all() and torch.isfinite(d[1]).all()
    assert torch.isnan(loss[0]) and torch.isfinite(loss[1])


def test_distill_gradient_against_differences():
    """Central differences of the device's own loss, fp32 logits: the quotient's error is the
    loss error (below 1e-6 here) over 2 eps, plus the third derivative times eps^2 / 6."""
    rng = np.random.default_rng(13)
    x = rng.standard_normal((1, 50)).astype(np.float32)
    ids, t = i32([[3, 20, 49, 3]]), f32_dev([[1.0, 0.0, 2.0, -1.0]])
    one = torch.ones(1, device=dev())
    _, grad = nb.distill_fwd_bwd(f32_dev(x), ids, t, one, 2.0)
    eps = 0.0625
    pairs = np.repeat(x, 100, 0)
    for v in range(50):
        pairs[2 * v, v] += eps
        pairs[2 * v + 1, v] -= eps
    loss, _ = nb.distill_fwd(f32_dev(pairs), ids.expand(100, 4).contiguous(),
                             t.expand(100, 4).contiguous(), 2.0)
    num = (pairs[np.arange(0, 100, 2), range(50)] - pairs[np.arange(1, 100, 2), range(50)])
    quot = (host(loss)[0::2] - host(loss)[1::2]) / num
    # |third derivative of tau^2 log sum exp(x / tau)| <= 1 / tau
    assert np.abs(quot - host(grad)[0]).max() <= 2e-6 / (2 * eps) + eps ** 2 / 12


def test_distill_repeats_bit_for_bit_and_on_another_stream():
    x, ids, t, g = draw(40, 9001, 100, "bf16", 14)
    X, I, T, G = to_dev(x, "bf16"), i32(ids), f32_dev(t), f32_dev(g)
    loss, grad = nb.distill_fwd_bwd(X, I, T, G, 2.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        loss2, grad2 = nb.distill_fwd_bwd(X, I, T, G, 2.0)
    s.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2)


def test_distill_no_entries_at_all_and_empty_batches():
    x = torch.randn(3, 100, device=dev())
    none, no_t = i32(np.zeros((3, 0))), torch.empty(3, 0, device=dev())
    loss, grad = nb.distill_fwd_bwd(x, none, no_t, torch.ones(3, device=dev()))
    assert not loss.any() and not grad.any()
    e = torch.empty(0, 100, device=dev())
    loss, grad = nb.distill_fwd_bwd(e, i32(np.zeros((0, 4))), torch.empty(0, 4, device=dev()),
                                    torch.empty(0, device=dev()))
    assert loss.shape == (0,) and grad.shape == (0, 100)


def test_distill_refusals():
    x = torch.randn(2, 10, device=dev())
    ids, t = i32([[1, 2], [3, 4]]), torch.randn(2, 2, device=dev())
    with pytest.raises(TypeError):
        nb.distill_fwd(x, ids.long(), t)
    with pytest.raises(TypeError):
        nb.distill_fwd(x, ids, t.bfloat16())
    with pytest.raises(TypeError):
        nb.distill_fwd(x.half(), ids, t)
    with pytest.raises(ValueError):
        nb.distill_fwd(torch.randn(10, 2, device=dev()).T, ids, t)
    with pytest.raises(ValueError):
        nb.distill_fwd(x[:1].expand(2, 10), ids, t)
    with pytest.raises(ValueError):
        nb.distill_fwd_bwd(x, ids, t, torch.ones(3, device=dev()))
    with pytest.raises(nb.NajuError):
        nb.distill_fwd(x, ids, t, temperature=0.0)
