"""Norms and linear attention where element and byte offsets pass 2^31 and 2^32: the far end of a
large tensor gives what the same tokens give alone."""
import pytest
import torch

from gpu_helpers import dev
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


@pytest.mark.parametrize("d", [1024, 4100])
def test_norms_far_rows(d):
    R, n = 4300000 * 1024 // d, 37  # 4.4e9 channels
    print("norms", R, d, flush=True)

    def tensor():
        t = torch.zeros(R, d, dtype=torch.bfloat16, device=dev())
        t[-n:] = torch.randn(n, d, device=dev())
        return t
    x, y = tensor(), tensor()
    w = torch.randn(d, device=dev())
    x_new, xn = nb.res_norm_fwd(x, y, w_post=w, w_pre=w)
    few = [t[-n:].clone() for t in (x, y)]
    f_new, fn = nb.res_norm_fwd(*few, w_post=w, w_pre=w)
    assert torch.equal(x_new[-n:], f_new) and torch.equal(xn[-n:], fn)
    assert not x_new[:n].any() and not xn[:n].any()
    g = nb.res_norm_bwd(x, y, x_new, y, w_post=w, w_pre=w)
    f = nb.res_norm_bwd(*few, f_new, few[1], w_post=w, w_pre=w)
    for k in ("dx", "dy"):
        assert torch.equal(g[k][-n:], f[k]), k
    for k in ("dw_pre", "dw_post"):
        # zeros add nothing, so 37 terms in two orders: 37 roundings of 2^-24 each
        size = f[k].abs().max()
        assert ((g[k] - f[k]).abs() <= 2 * 37 * 2.0 ** -24 * 40 * size).all(), k


def test_linear_attention_far_tokens():
    """300000 tokens of 128 heads: only the last 100 are not zero.  Both calls hold fp32 sums and
    round each output once, so they differ by a step of bf16 at most, and by fp32's roundings of a
    hundred terms."""
    L, n, H, Hk, d = 300000, 100, 128, 64, 128  # 4.9e9 elements of q and o
    print("linear attention", L, H, d, flush=True)

    def tensor(heads):
        t = torch.zeros(1, L, heads, d, dtype=torch.bfloat16, device=dev())
        t[:, -n:] = torch.randn(n, heads, d, device=dev())
        return t
    q, k, v, do = tensor(H), tensor(Hk), tensor(Hk), tensor(H)
    a = torch.linspace(-0.5, 0.0, H, device=dev())
    few = [t[:, -n:].clone() for t in (q, k, v)]
    own = do[:, -n:].clone()

    def near(x, y, name):
        x, y = x.float(), y.float()
        assert ((x - y).abs() <= 2.0 ** -7 * y.abs() + 1e-5 * y.abs().max()).all(), name
    o, s = nb.linattn_fwd(q, k, v, a)
    fo, fs = nb.linattn_fwd(*few, a)
    near(o[:, -n:], fo, "o")
    near(s, fs, "state")
    assert not o[:, :-n].any()
    del o
    g = nb.linattn_bwd(q, k, v, a, do)
    f = nb.linattn_bwd(*few, a, own)
    for name in ("dq", "dk", "dv"):
        near(g[name][:, -n:], f[name], name)
    assert not g["dq"][:, :-n].any()


def test_single_tokens_of_many_rows():
    B, H, d = 8200, 16, 128  # 2.1e9 elements of the state, and more rows than a launch takes
    print("step", B, H, d, flush=True)
    state = torch.zeros(B, H, d, d, device=dev())
    state[-3:] = torch.randn(3, H, d, d, device=dev())
    q, k, v = (torch.randn(B, H, d, dtype=torch.bfloat16, device=dev()) for _ in range(3))
    a = torch.linspace(-0.5, 0.0, H, device=dev())
    alone = state[-3:].clone()
    o = nb.linattn_step(q, k, v, a, state)
    fo = nb.linattn_step(q[-3:].clone(), k[-3:].clone(), v[-3:].clone(), a, alone)
    assert torch.equal(o[-3:], fo) and torch.equal(state[-3:], alone)
    first = torch.zeros(3, H, d, d, device=dev())
    fo = nb.linattn_step(q[:3].clone(), k[:3].clone(), v[:3].clone(), a, first)
    assert torch.equal(o[:3], fo) and torch.equal(state[:3], first)


@pytest.mark.parametrize("dv", [8, 136, 256])
def test_most_heads(dv):
    """2^20 heads in all, in one, two or three parts of the columns each: the last rows give what
    they give alone (one chunk, so whatever its cut the sums are the same)."""
    B, L, H, dk, n = 1 << 16, 2, 16, 8, 3
    print("heads", B * H, dv, flush=True)
    q, k = (torch.randn(B, L, H, dk, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    v, do = (torch.randn(B, L, H, dv, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    a = torch.linspace(-0.5, 0.0, H, device=dev())
    o, s = nb.linattn_fwd(q, k, v, a)
    g = nb.linattn_bwd(q, k, v, a, do)
    few = [t[-n:].clone() for t in (q, k, v)]
    fo, fs = nb.linattn_fwd(*few, a)
    f = nb.linattn_bwd(*few, a, do[-n:].clone())
    assert torch.equal(o[-n:], fo) and torch.equal(s[-n:], fs)
    for name in f:
        assert torch.equal(g[name][-n:], f[name]), name
    with pytest.raises(nb.NajuError, match="too large"):
        nb.linattn_fwd(q[:, :, :1].expand(B, L, 17, dk).contiguous(), k[:, :, :1].contiguous(),
                       v[:, :, :1].contiguous(), torch.zeros(17, device=dev()))
