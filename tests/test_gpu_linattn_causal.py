"""A NaN or an infinity in a token of linear attention reaches the outputs of that token and of those
after it (their keys' and values' gradients: of those before it), as the formula says: all others keep
their bits, and of its own and the later ones those that the fp64 formula makes neither NaN nor
infinite stay finite."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from oracle import layer
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def inputs(B, L, H, Hk, dk, dv, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(L + dk)
    t = {k: torch.randn(B, L, h, d, generator=g, device=dev()).to(dt)
         for k, h, d in (("q", H, dk), ("k", Hk, dk), ("v", Hk, dv), ("do", H, dv))}
    t["a"] = torch.linspace(-0.3, -0.01, H, device=dev())
    t["s"] = torch.randn(B, H, dk, dv, generator=g, device=dev())
    t["n"] = torch.tensor([L, L - L // 3][:B], dtype=torch.int32, device=dev())
    return t


def run(t, lengths):
    n = t["n"] if lengths else None
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["s"], n)
    return dict(nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"], t["s"], None, n), o=o,
                state=s)


SHAPES = [(2, 300, 4, 2, 24, 40), (1, 130, 2, 2, 128, 128), (2, 70, 2, 1, 16, 136),
          (1, 90, 1, 1, 256, 72), (1, 2000, 1, 1, 64, 64)]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_other_tokens_keep_their_bits(shape, value, dt):
    t = inputs(*shape, dt)
    L = shape[1]
    for lengths in (False, True):
        clean = run(t, lengths)
        last = int(t["n"][0]) if lengths else L
        for where in ("q", "k", "v", "do"):
            for at in sorted({0, 17, last // 2, last - 1}):
                bad = dict(t)
                bad[where] = t[where].clone()
                bad[where][0, at, 0, 3] = value
                got = run(bad, lengths)
                what = (where, at, lengths)
                # outputs and the gradients of queries: nothing before the token
                for name in ("o", "dq"):
                    assert torch.equal(got[name][0, :at], clean[name][0, :at]), (name, what)
                # of keys and values: nothing behind it
                for name in ("dk", "dv"):
                    assert torch.equal(got[name][0, at + 1:], clean[name][0, at + 1:]), (name, what)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("where", ["q", "k", "v", "do"])
def test_bad_outputs_are_the_formulas(where, dt):
    """Element by element: not finite where the formula is not, and nowhere else; what is finite is
    what it was without the bad value (there it does not depend on it)."""
    B, L, H, dk, dv, at = 1, 150, 2, 24, 40, 77
    t = inputs(B, L, H, H, dk, dv, dt)
    clean = run(t, False)
    for value in (float("nan"), float("inf")):
        bad = dict(t)
        bad[where] = t[where].clone()
        bad[where][0, at, 1, 5] = value
        got = run(bad, False)
        c = {k: x.double().cpu().numpy() for k, x in bad.items()}
        with np.errstate(all="ignore"):
            o, s = layer.linattn_fwd(c["q"], c["k"], c["v"], c["a"], c["s"], None, dk ** -0.5)
            want = dict(layer.linattn_bwd(c["q"], c["k"], c["v"], c["a"], c["do"], c["s"], None,
                                          None, dk ** -0.5), o=o, state=s)
        for name, x in got.items():
            finite = torch.from_numpy(np.isfinite(want[name])).to(dev())
            assert torch.equal(x.isfinite(), finite), (name, where, value)
            assert torch.equal(x[finite], clean[name][finite]), (name, where, value)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_many_bad_values(dt):
    """Values and keys of every second token from one on are NaN in some columns: columns and tokens
    that none of them reach keep their bits."""
    B, L, H, dk, dv = 1, 200, 1, 64, 64
    t = inputs(B, L, H, H, dk, dv, dt)
    clean = run(t, False)
    bad = dict(t)
    bad["v"] = t["v"].clone()
    bad["v"][0, 35::2, 0, 7:20:3] = float("nan")
    bad["v"][0, 131, 0, 50] = float("inf")
    o = run(bad, False)["o"][0, :, 0]
    want = clean["o"][0, :, 0].clone()
    want[35:, 7:20:3] = float("nan")
    assert torch.equal(o.isfinite()[:131], want.isfinite()[:131])
    assert not o[131:, 50].isfinite().any()
    keep = want.isfinite()
    keep[131:, 50] = False
    assert torch.equal(o[keep], want[keep])


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [100, 3000])
def test_states_in_place(L, dt):
    """The walk that is done again starts from the state that the first one started from."""
    t = inputs(1, L, 2, 1, 32, 72, dt)
    t["v"][0, L // 2, 0, 9] = float("nan")
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["s"])
    o2, s2 = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["s"], state_out=t["s"])
    assert s2 is t["s"]
    assert torch.equal(o.isnan(), o2.isnan()) and torch.equal(o.nan_to_num(), o2.nan_to_num())
    assert torch.equal(s.isnan(), s2.isnan()) and torch.equal(s.nan_to_num(), s2.nan_to_num())
    assert s[..., 9].isnan().all() and s[..., :9].isfinite().all()
    assert o[0, :L // 2].isfinite().all() and o[0, L // 2:, :, 9].isnan().all()


def test_replays():
    """A captured call whose inputs become bad and good again."""
    t = inputs(1, 500, 2, 1, 32, 40, torch.bfloat16)
    good = t["v"].clone()
    run(t, False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(t, False)
    for bad in (False, True, False, True):
        t["v"].copy_(good)
        if bad:
            t["v"][0, 333, 0, 1] = float("inf")
        want = run(t, False)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k].isfinite(), want[k].isfinite()), (k, bad)
            ok = want[k].isfinite()
            assert torch.equal(out[k][ok], want[k][ok]), (k, bad)
