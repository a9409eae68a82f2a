"""Linear attention with a decay for each head: chunked forward and gradients, and single tokens,
against the fp64 recurrence."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32_dev, host, to_dev
from oracle import layer
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def rounded(rng, shape, io, std=1.0):
    x = torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32))
    return (x.bfloat16() if io == "bf16" else x).double().numpy()


def draw(B, L, H, Hk, dk, dv, io, seed=0, state=True, lengths=None, decays=None):
    rng = np.random.default_rng(seed)
    c = dict(q=rounded(rng, (B, L, H, dk), io), k=rounded(rng, (B, L, Hk, dk), io, dk ** -0.5),
             v=rounded(rng, (B, L, Hk, dv), io), do=rounded(rng, (B, L, H, dv), io))
    a = -np.exp2(-1.0 - 9.0 * rng.random(H)) if decays is None else np.asarray(decays)
    c["a"] = a.astype(np.float32).astype(np.float64)
    c["state"] = rounded(rng, (B, H, dk, dv), "f32") if state else None
    c["ds"] = rounded(rng, (B, H, dk, dv), "f32") if state else None
    c["n"] = None if lengths is None else np.asarray(lengths, dtype=np.int32)
    c["scale"] = dk ** -0.5
    return c


def on_dev(c, io):
    t = {k: to_dev(c[k], io) for k in ("q", "k", "v", "do")}
    t["a"] = f32_dev(c["a"])
    for k in ("state", "ds"):
        t[k] = None if c[k] is None else f32_dev(c[k])
    t["n"] = None if c["n"] is None else torch.from_numpy(c["n"]).to(dev())
    return t


def close(name, got, want, terms, io, L, d):
    """|got - want| against one rounding of the output, and the products' own error, measured
    against `terms`, the result with every factor's magnitude in its place: parts of 16 bits in
    bf16 products (2^-16 with a factor of two for two such factors), and fp32 sums over a head's
    elements, a chunk's tokens and the chunks before it."""
    got = host(got)
    assert got.shape == want.shape
    own = (2.0 ** -15 if io[0] == "bf16" else 0) + (64 + d ** 0.5 + (L / 32) ** 0.5) * 2.0 ** -24
    bound = HALF[io[1]] * np.abs(want) + own * terms + 1e-30
    err = np.abs(got - want)
    worst = float((err / bound).max()) if err.size else 0.0
    rel = float(np.linalg.norm(err) / max(np.linalg.norm(want), 1e-30))
    print("  %-7s worst %.3f of the bound, relative error %.1e" % (name, worst, rel), flush=True)
    assert worst <= 1.0, name
    # all over, the rounding of outputs is what is seen
    assert rel <= HALF[io[1]] + own * np.linalg.norm(terms) / max(np.linalg.norm(want), 1e-30)


def check_fwd(B, L, H, Hk, dk, dv, io, **kw):
    c = draw(B, L, H, Hk, dk, dv, io, **kw)
    t = on_dev(c, io)
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"], t["n"])
    args = (c["q"], c["k"], c["v"], c["a"], c["state"], c["n"], c["scale"])
    wo, ws = layer.linattn_fwd(*args)
    to, ts = layer.linattn_fwd(*[x if i > 2 and i != 4 or x is None else np.abs(x)
                                 for i, x in enumerate(args)])
    close("o", o, wo, to, (io, io), L, dk)
    # the state's sum takes the decayed values in three parts: fp32's precision
    close("state", s, ws, ts, ("f32", "f32"), L, dk)
    return c, t, o, s


def check_bwd(B, L, H, Hk, dk, dv, io, **kw):
    c = draw(B, L, H, Hk, dk, dv, io, **kw)
    t = on_dev(c, io)
    g = nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"], t["state"], t["ds"], t["n"])
    args = (c["q"], c["k"], c["v"], c["a"], c["do"], c["state"], c["ds"], c["n"], c["scale"])
    want = layer.linattn_bwd(*args)
    terms = layer.linattn_bwd(*[x if i in (3, 7, 8) or x is None else np.abs(x)
                                for i, x in enumerate(args)])
    for k in ("dq", "dk", "dv"):
        close(k, g[k], want[k], terms[k], (io, io), L, max(dk, dv))
    close("dstate", g["dstate"], want["dstate"], terms["dstate"], ("f32", "f32"), L, dk)
    return g


SHAPES = [(1, 1, 1, 1, 8, 8), (2, 3, 2, 1, 16, 24), (1, 31, 3, 3, 32, 32), (2, 64, 2, 2, 40, 72),
          (1, 65, 4, 2, 64, 64), (3, 129, 2, 2, 128, 128), (1, 200, 1, 1, 72, 136),
          (1, 97, 2, 1, 136, 8), (1, 130, 1, 1, 256, 256), (2, 70, 6, 2, 24, 200),
          (1, 1500, 2, 2, 32, 48)]


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, io):
    check_fwd(*shape, io, seed=sum(shape))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(shape, io):
    check_bwd(*shape, io, seed=sum(shape) + 1)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("L", [100, 1300])
def test_ragged_rows(L, io):
    """Lengths of zero, one, whole chunks and past the end; what lies behind them is NaN and must
    not be read, and outputs are zero there."""
    n = [0, 1, 63, 64, 65, L - 1, L, L + 5, -3]
    B = len(n)
    c = draw(B, L, 2, 1, 24, 40, io, seed=L, lengths=n)
    t = on_dev(c, io)
    for b in range(B):
        for k in ("q", "k", "v", "do"):
            t[k][b, max(0, n[b]):] = float("nan")
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"], t["n"])
    g = nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"], t["state"], t["ds"], t["n"])
    u = on_dev(c, io)
    o2, s2 = nb.linattn_fwd(u["q"], u["k"], u["v"], u["a"], u["state"], u["n"])
    g2 = nb.linattn_bwd(u["q"], u["k"], u["v"], u["a"], u["do"], u["state"], u["ds"], u["n"])
    assert torch.equal(o, o2) and torch.equal(s, s2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    for b in range(B):
        for x in (o, g["dq"], g["dk"], g["dv"]):
            assert (x[b, min(max(0, n[b]), L):] == 0).all()
    assert torch.equal(s[0], u["state"][0]) and torch.equal(g["dstate"][0], u["ds"][0])
    check_fwd(B, L, 2, 1, 24, 40, io, seed=L, lengths=n)
    check_bwd(B, L, 2, 1, 24, 40, io, seed=L, lengths=n)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decays(io):
    """No decay at all, no memory at all, and those between."""
    decays = [0.0, -1e-5, -0.05, -3.0, -200.0, -np.inf]
    check_fwd(1, 300, 6, 6, 32, 32, io, seed=3, decays=decays)
    check_bwd(1, 300, 6, 3, 32, 32, io, seed=4, decays=decays)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_without_states(io):
    check_fwd(2, 90, 2, 2, 32, 16, io, seed=5, state=False)
    check_bwd(2, 90, 2, 2, 32, 16, io, seed=6, state=False)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_segments(io):
    """One head over a sequence long enough to be cut into many segments, ragged too."""
    nbytes = nb.lib().naju_linattn_fwd_workspace_bytes(2, 5000, 1, 1, 16, 32)
    assert nbytes >= 2 * 9 * 16 * 32 * 4  # (nine segments or more)
    check_fwd(2, 5000, 1, 1, 16, 32, io, seed=7, lengths=[5000, 2600], decays=[-0.002])
    check_bwd(2, 5000, 1, 1, 16, 32, io, seed=8, lengths=[3001, 5000], decays=[-0.002])


def test_parts_of_a_joint_projection():
    """q, k and v as parts of one tensor, and through padded rows."""
    B, L, H, d = 2, 150, 3, 32
    joint = torch.randn(B, L, 3 * H * d + 16, device=dev()).bfloat16()
    q, k, v = (joint[:, :, 8 + i * H * d:8 + (i + 1) * H * d].unflatten(2, (H, d))
               for i in range(3))
    a = torch.tensor([-0.1, -0.5, -0.01], device=dev())
    do = torch.randn(B, L, H, d, device=dev()).bfloat16()
    o, s = nb.linattn_fwd(q, k, v, a)
    o2, s2 = nb.linattn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), a)
    assert torch.equal(o, o2) and torch.equal(s, s2)
    g = nb.linattn_bwd(q, k, v, a, do)
    g2 = nb.linattn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), a, do)
    for x in g:
        assert torch.equal(g[x], g2[x]), x


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 8, 8), (3, 4, 2, 40, 72), (2, 3, 3, 128, 128),
                                          (5, 2, 1, 256, 256), (2, 2, 2, 24, 200), (300, 2, 2, 16, 32)])
def test_single_tokens(B, H, Hk, dk, dv, io):
    c = draw(B, 1, H, Hk, dk, dv, io, seed=B + dk, decays=[0.0, -0.3, -np.inf, -2.0][:H])
    t = on_dev(c, io)
    q, k, v = (t[x][:, 0].contiguous() for x in ("q", "k", "v"))
    kept = t["state"].clone()
    new = torch.empty_like(kept)
    o = nb.linattn_step(q, k, v, t["a"], t["state"], state_out=new)
    assert torch.equal(t["state"], kept)
    args = (c["q"], c["k"], c["v"], c["a"], c["state"], None, c["scale"])
    wo, ws = layer.linattn_fwd(*args)
    to, ts = layer.linattn_fwd(*[np.abs(x) if i in (0, 1, 2, 4) else x
                                 for i, x in enumerate(args)])
    close("o", o, wo[:, 0], to[:, 0], ("f32", io), 1, dk)
    close("state", new, ws, ts, ("f32", "f32"), 1, dk)
    o2 = nb.linattn_step(q, k, v, t["a"], t["state"])
    assert torch.equal(o, o2) and torch.equal(t["state"], new)


def test_steps_continue_a_prompt():
    """A prompt in chunks, then tokens one at a time, give what the whole
    sequence gives: both keep fp32 states and round each output once."""
    B, L, H, d = 2, 140, 2, 64
    c = draw(B, L, H, H, d, d, "bf16", seed=12, state=False)
    t = on_dev(c, "bf16")
    whole, end = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"])
    cut = 133
    _, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"],
                          lengths=torch.full((B,), cut, dtype=torch.int32, device=dev()))
    for i in range(cut, L):
        o = nb.linattn_step(*(t[k][:, i].contiguous() for k in ("q", "k", "v")), t["a"], s)
        d_ = (o.float() - whole[:, i].float()).abs()
        # (two roundings of nearly equal values: a step of bf16 apart at most)
        assert (d_ <= 2.0 ** -7 * whole[:, i].float().abs() + 1e-4).all()
    assert torch.allclose(s, end, rtol=1e-4, atol=1e-5)


def test_states_in_place():
    c = draw(2, 1300, 1, 1, 16, 16, "bf16", seed=13)
    t = on_dev(c, "bf16")
    o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"])
    o2, s2 = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"], state_out=t["state"])
    assert s2 is t["state"] and torch.equal(s, s2) and torch.equal(o, o2)


def test_empty():
    a = torch.zeros(2, device=dev())
    s = torch.randn(3, 2, 16, 8, device=dev())
    q, v = torch.zeros(3, 0, 2, 16, device=dev()), torch.zeros(3, 0, 2, 8, device=dev())
    o, s2 = nb.linattn_fwd(q, q, v, a, s)
    assert o.shape == (3, 0, 2, 8) and torch.equal(s, s2)
    g = nb.linattn_bwd(q, q, v, a, v, s, s)
    assert torch.equal(g["dstate"], s) and g["dk"].shape == q.shape
    o, s2 = nb.linattn_fwd(q[:0], q[:0], v[:0], a)
    assert s2.shape == (0, 2, 16, 8)


def test_repeats_give_equal_bits():
    c = draw(2, 1500, 2, 1, 40, 56, "bf16", seed=14)
    t = on_dev(c, "bf16")
    f = lambda: [*nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"])] + list(  # noqa: E731
        nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], t["do"], t["state"], t["ds"]).values())
    first = f()
    for _ in range(3):
        for x, y in zip(f(), first):
            assert torch.equal(x, y)


def test_graph_replays():
    c = draw(1, 1400, 2, 1, 32, 32, "bf16", seed=15)
    t = on_dev(c, "bf16")

    def step():
        o, s = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"])
        g = nb.linattn_bwd(t["q"], t["k"], t["v"], t["a"], o, t["state"], s)
        new = torch.empty_like(s)
        last = nb.linattn_step(*(t[k][:, -1].contiguous() for k in ("q", "k", "v")), t["a"], s,
                               state_out=new)
        return [o, s, new, last] + list(g.values())
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(4):
        t["v"].copy_(torch.randn_like(t["v"]))
        want = step()
        for x in out:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), n


def test_another_stream():
    c = draw(2, 1400, 1, 1, 32, 32, "bf16", seed=16)
    t = on_dev(c, "bf16")
    want = nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for st in streams:
        with torch.cuda.stream(st):
            got.append(nb.linattn_fwd(t["q"], t["k"], t["v"], t["a"], t["state"]))
    torch.cuda.synchronize()
    for o, s in got:
        assert torch.equal(o, want[0]) and torch.equal(s, want[1])
