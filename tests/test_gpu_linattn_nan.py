"""How far a NaN or an infinity reaches in linear attention: other rows, heads that do not read it
and tokens more than a chunk away on the side that the sum does not come from keep their bits."""
import pytest
import torch

from gpu_helpers import dev
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu
B, L, H, HK, D, AT, ROW, HEAD = 2, 300, 4, 2, 24, 150, 1, 1  # (head of k and v; q's 2 and 3)


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def inputs(dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    t = {k: torch.randn(B, L, h, D, generator=g, device=dev()).to(dt)
         for k, h in (("q", H), ("k", HK), ("v", HK), ("do", H))}
    t["a"] = torch.linspace(-0.3, -0.01, H, device=dev())
    return t


def run(t):
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"])
    return dict(nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"]), o=o, state=s)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
def test_reach(where, value, dt):
    t = inputs(dt)
    clean = run(t)
    shared = where in ("k", "v")
    t[where][ROW, AT, HEAD if shared else 2, 5] = value
    got = run(t)
    readers = [2, 3] if shared else [2]
    for name, c in clean.items():
        x = got[name]
        assert torch.equal(x[0], c[0]), name  # the other row
        if name in ("state", "dstate"):
            heads, axis = readers, 0
        else:
            heads, axis = (readers, 1) if name in ("o", "dq") else ([HEAD], 1)
        others = [h for h in range(c.shape[1 + axis]) if h not in heads]
        for h in others:
            assert torch.equal(x[1].select(axis, h), c[1].select(axis, h)), (name, h)
    for name in ("o", "dq"):
        assert torch.equal(got[name][1, :AT - 63], clean[name][1, :AT - 63]), name
    for name in ("dk", "dv"):
        assert torch.equal(got[name][1, AT + 64:], clean[name][1, AT + 64:]), name
    # and where it has to arrive
    if where == "do":
        assert torch.equal(got["o"], clean["o"]) and not got["dv"][1, AT, HEAD].isfinite().all()
    else:
        assert not got["o"][1, AT, 2].isfinite().all()
        if where != "q":
            assert not got["o"][1, AT:, 2:].isfinite().all(-1).any()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_what_lies_behind_a_rows_length_is_not_read(dt):
    t = inputs(dt)
    n = torch.tensor([200, 77], dtype=torch.int32, device=dev())

    def both():
        o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], lengths=n)
        return dict(nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"], lengths=n), o=o, s=s)
    clean = both()
    for k in ("q", "k", "v", "do"):
        t[k][0, 200:] = float("nan")
        t[k][1, 77:] = float("inf")
    for name, x in both().items():
        assert torch.equal(x, clean[name]), name
