"""Distillation where logits or teacher values lie at the ends of their type's range: a
vocabulary masked with the lowest value (all but a few tokens, or all of them), the largest value,
values far from zero.  Forward, backward and the joint call against the fp64 definition.

Tolerances, derived before the first run.  u = 2^-24.  A maximum m is taken off before a difference
is scaled, so an exponent (s - m) / tau has one rounding of the difference, two of 1/tau times
log2 e and one of the product: at most 4 u |s - m| / tau, whatever m is.  With G the largest such
exponent that matters (those beyond 104 leave less than the smallest fp32 number), the hardware
exponential's 2 u and a sum log2 V + V/512 additions deep, q is off by e_q = u (20 G + 64 + V/512)
relative, and a loss by tau^2 u (30 G + 64 + V/512 + 16 (G + log V)).  distill_bwd takes q from lse
where |lse| <= 16384, whose own rounding adds 4 u |lse|.  lse itself is m / tau + log(sum), rounded
as an fp32 number: u (3 |lse| + 64 + V/512), infinite where it leaves the type.  Gradients that
underflow may be flushed: 2^-125 |g| tau absolute.
"""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, to_dev
from oracle import lm
from selective_state_space_naju_amd import binding as nb
from selective_state_space_naju_amd import inputs
from test_gpu_distill import check, run_all

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def bounds(x, ids, t, tau, g, io):
    V = x.shape[1]
    loss, lse, grad = lm.distill(x, ids, t, tau, g)
    with np.errstate(all="ignore"):
        gap = (x.max(1, keepdims=True).astype(np.float64) - x) / tau
        t_gap = (t.max(1, keepdims=True).astype(np.float64) - t) / tau
    q = np.exp(-gap)
    q /= q.sum(1, keepdims=True)
    G = np.where(gap < 104, gap, 0).max(1)
    listed = np.take_along_axis(gap, ids, 1)
    G = np.maximum(G, np.where(t_gap < 104, np.maximum(t_gap, listed), 0).max(1))
    deep = 64 + V / 512
    b_loss = tau * tau * U * (30 * G + deep + 16 * (G + np.log(V) + 7))
    b_lse = U * (3 * np.abs(lse) + deep)
    e_q = U * (20 * G + deep + 4 * np.where(np.abs(lse) <= 16384, np.abs(lse), 0))
    size = 2 * q + np.abs(grad) / (np.abs(g) * tau)[:, None]
    io_u = 2.0 ** -8 if io == "bf16" else 2.0 ** -22
    b_grad = (np.abs(g) * tau * e_q)[:, None] * size + io_u * np.abs(grad)
    return loss, lse, grad, b_loss, b_lse, b_grad + 2.0 ** -125 * (1 + np.abs(g) * tau)[:, None]


# one vocabulary for each form of the joint kernel, and one past its registers
SIZES = [("f32", 40), ("f32", 1500), ("f32", 3000), ("f32", 8000), ("f32", 16000), ("f32", 20001),
         ("f32", 60000), ("f32", 70001), ("bf16", 7), ("bf16", 40), ("bf16", 4000),
         ("bf16", 8000), ("bf16", 16000), ("bf16", 32000), ("bf16", 50001), ("bf16", 131072),
         ("bf16", 140001)]


@pytest.mark.parametrize("tau", [0.5, 1.0, 4.0])
@pytest.mark.parametrize("io,V", SIZES)
def test_distill_at_the_ends_of_the_range(io, V, tau):
    print("distill range", io, V, tau, flush=True)
    rng = np.random.default_rng(15)
    R, k = 9, 4
    top = np.float32(3.3895314e38) if io == "bf16" else np.finfo(np.float32).max
    x = 2 * rng.standard_normal((R, V)).astype(np.float32)
    ids = np.stack([rng.permutation(V)[:k] for _ in range(R)])
    t = rng.standard_normal((R, k)).astype(np.float32)
    for r in (0, 1):  # all but the listed tokens are masked with the lowest value
        kept = x[r, ids[r]]
        x[r] = -top
        x[r, ids[r]] = kept
    x[2] = -top                         # every token
    t[3, 1:] = np.finfo(np.float32).min  # a teacher's masked entries
    t[4] = np.finfo(np.float32).min
    x[5, ids[5, 0]] = top               # one token takes it all
    t[5, 1:] = -np.inf
    x[6] = top
    x[7] = -top
    x[7, ids[7]] = top                  # the widest difference
    x[8] *= np.float32(1e9)
    x[8, ids[8, 0]] = 2 * np.abs(x[8]).max()
    t[8, 1:] = -np.inf
    x = inputs.bf16_round(x) if io == "bf16" else x
    g = np.linspace(0.5, 1.5, R).astype(np.float32)
    loss, lse, grad, b_loss, b_lse, b_grad = bounds(x, ids, t, tau, g, io)
    assert np.isfinite(loss).all()
    with np.errstate(over="ignore"):
        lse = lse.astype(np.float32)
    got = run_all(x, ids, t, tau, g, io, pad=3)
    for name, a, ref, b in (("loss", got[0], loss, b_loss), ("lse", got[1], lse, b_lse),
                            ("gradient", got[2], grad, b_grad),
                            ("loss (joint)", got[3], loss, b_loss),
                            ("gradient (joint)", got[4], grad, b_grad)):
        check(name, a, ref, b)


@pytest.mark.parametrize("io,V", [("bf16", 40), ("bf16", 70001), ("f32", 20000)])
def test_distill_rows_of_weight_zero_whatever_they_hold(io, V):
    """Padding: zeros, from logits and an lse of any kind, and nothing in the rows beside them."""
    x = torch.randn(7, V, device=dev())
    for r, v in enumerate((-np.inf, np.nan, -3.4e38, 3e4, np.inf)):
        x[r] = v
    x = to_dev(x.cpu().numpy(), io)
    ids = torch.zeros(7, 2, dtype=torch.int32, device=dev())
    ids[:, 1] = V - 1
    t = torch.zeros(7, 2, device=dev())
    g = torch.tensor([0.0] * 6 + [1.0], device=dev())
    lse = nb.distill_fwd(x, ids, t)[1]
    lse[5] = 1e30
    grad, joint = nb.distill_bwd(x, ids, t, lse, g), nb.distill_fwd_bwd(x, ids, t, g)[1]
    for d in (grad, joint):
        assert not d[:6].any() and d[6].any() and torch.isfinite(d).all()
