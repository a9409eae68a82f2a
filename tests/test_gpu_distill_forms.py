"""Distillation in the forms that sizes choose and that test_gpu_distill's cases do not reach: the
joint call's 4 accesses a thread at 128 threads and its 16 and 32 in fp32, the gradient of 8
accesses a thread (512 workgroups and more), and gradients written into rows of any stride and
alignment.  The bounds are test_gpu_distill's."""
import pytest
import torch

from gpu_helpers import dev, f32_dev, host, to_dev
from selective_state_space_naju_amd import binding as nb
from test_gpu_distill import bounds, check, draw, i32, run_all

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


CASES = [  # rows, vocab, k, io, tau, pad, lists
    (3, 1500, 100, "f32", 1.0, 0, "ragged"),
    (3, 3001, 128, "bf16", 2.0, 3, "ragged"),
    (3, 2048, 128, "f32", 1.0, 0, "full"),
    (3, 2048, 129, "f32", 1.0, 0, "full"),
    (3, 20001, 60, "f32", 1.5, 0, "ragged"),
    (3, 40001, 60, "f32", 1.0, 2, "ragged"),
    (180, 33001, 20, "f32", 2.0, 1, "ragged"),
    (180, 70001, 20, "bf16", 1.0, 1, "ragged"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "r%d_v%d_k%d_%s_tau%g_pad%d_%s" % c)
def test_distill_form(case):
    R, V, k, io, tau, pad, lists = case
    print("distill form", case, flush=True)
    x, ids, t, g = draw(R, V, k, io, 17, lists)
    loss, lse, grad, b_loss, b_lse, b_grad = bounds(x, ids, t, tau, g, io)
    got = run_all(x, ids, t, tau, g, io, pad)
    for name, a, ref, b in (("loss", got[0], loss, b_loss), ("lse", got[1], lse, b_lse),
                            ("gradient", got[2], grad, b_grad),
                            ("loss (joint)", got[3], loss, b_loss),
                            ("gradient (joint)", got[4], grad, b_grad)):
        check(name, a, ref, b)


@pytest.mark.parametrize("io,V", [("f32", 5), ("bf16", 9), ("f32", 500), ("f32", 2047),
                                  ("bf16", 1024), ("bf16", 4095), ("f32", 8190),
                                  ("bf16", 16384), ("bf16", 32768), ("f32", 32767),
                                  ("bf16", 65536), ("f32", 65536), ("bf16", 131071),
                                  ("bf16", 131072), ("bf16", 140003)])
@pytest.mark.parametrize("shift,pad", [(0, 0), (1, 0), (0, 1), (3, 5), (7, 9)])
def test_distill_joint_call_into_rows_of_any_stride(io, V, shift, pad):
    """The accesses are laid out from the gradient's rows: their start and their stride move, the
    logits' rows stay aligned, so the two disagree by every number of elements."""
    print("distill stride", io, V, shift, pad, flush=True)
    R, k, tau = 5, 7, 1.5
    x, ids, t, g = draw(R, V, k, io, 18, "full")
    loss, _, grad, b_loss, _, b_grad = bounds(x, ids, t, tau, g, io)
    X, I, T, G = to_dev(x, io), i32(ids), f32_dev(t), f32_dev(g)
    memory = torch.full((R * (V + pad) + shift + 16,), 7.0, dtype=X.dtype, device=dev())
    out = torch.as_strided(memory, (R, V), (V + pad, 1), shift)
    got_loss, same = nb.distill_fwd_bwd(X, I, T, G, tau, dlogits=out)
    assert same is out
    check("loss", host(got_loss), loss, b_loss)
    check("gradient", host(out), grad, b_grad)
    rest = torch.ones_like(memory, dtype=torch.bool)
    torch.as_strided(rest, (R, V), (V + pad, 1), shift).fill_(False)
    assert (memory[rest] == 7.0).all()  # nothing between the rows is written
