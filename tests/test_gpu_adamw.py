"""The AdamW step over many tensors, states in 32 and 8 bits, against the fp64 definition."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from oracle import layer
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn
SIZES = [1, 2, 3, 5, 255, 256, 257, 1000, 1023, 4095, 4096, 4097, 8192, 12345, 70001]


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


def draw(sizes, bits, g_dt=torch.float32, seed=0):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    rand = lambda n, s: torch.randn(n, generator=g, device=dev()) * s  # noqa: E731
    t = dict(p=[rand(n, 0.1) for n in sizes], g=[rand(n, 1e-2).to(g_dt) for n in sizes],
             m=[rand(n, 1e-2) for n in sizes], v=[rand(n, 1e-2).square() for n in sizes])
    if bits == 8:
        blocks = [-(-n // 256) for n in sizes]
        t["m"] = [(rand(n, 100.0)).clamp(-448, 448).to(E4M3) for n in sizes]
        t["v"] = [(rand(n, 100.0)).abs().clamp(max=448).to(E4M3) for n in sizes]
        t["m_scale"] = [rand(b, 1e-4).abs() for b in blocks]
        t["v_scale"] = [rand(b, 1e-4).abs() for b in blocks]
    return t


def values(codes, scale):
    n = codes.numel()
    return host(codes).ravel() * np.repeat(host(scale), 256)[:n]


def call(t, step=7, lr=1e-2, **kw):
    scales = {k: t[k] for k in ("m_scale", "v_scale") if k in t}
    nb.adamw_step(t["p"], t["g"], t["m"], t["v"], step, lr, **scales, **kw)


def clone(t):
    return {k: [x.clone() for x in v] for k, v in t.items()}


def want_of(t, i, step=7, lr=1e-2, gs=1.0, **kw):
    m, v = t["m"][i], t["v"][i]
    if "m_scale" in t:
        m, v = values(m, t["m_scale"][i]), values(v, t["v_scale"][i]) ** 2
    else:
        m, v = host(m).ravel(), host(v).ravel()
    return layer.adamw(host(t["p"][i]).ravel(), host(t["g"][i]).ravel(), m, v, step, lr,
                       grad_scale=gs, **kw)


def check(got, before, i, lr=1e-2, **kw):
    """p, m and v are sums of terms, each after at most 16 fp32 operations (2^-20 of the terms'
    sizes); a code of 8 bits is at most half a step of 2^-3 from its value, 2^-4 relative and
    2^-10 of a scale below the smallest normal one."""
    p, m, v = want_of(before, i, lr=lr, **kw)
    b1, b2 = kw.get("beta1", 0.9), kw.get("beta2", 0.999)
    gs = kw.get("gs", 1.0)
    g = np.abs(host(before["g"][i]).ravel() * gs)
    e = 2.0 ** -20
    p0 = np.abs(host(before["p"][i]).ravel())
    # (m cancels where its old value and the gradient have opposite signs)
    terms = (b1 * (np.abs(m) + g) + (1 - b1) * g) / max(1e-30, 1 - b1 ** kw.get("step", 7))
    vh = np.sqrt(v / (1 - b2 ** kw.get("step", 7))) + kw.get("eps", 1e-8)
    bound = e * (p0 + np.abs(p) + lr * terms / vh)
    err = np.abs(host(got["p"][i]).ravel() - p)
    assert (err <= bound).all(), (i, float((err / bound).max()))
    if "m_scale" in got:
        for k, x in (("m", m), ("v", np.sqrt(v))):
            n = len(x)
            blocks = np.pad(np.abs(x), (0, -n % 256)).reshape(-1, 256).max(1)
            sc = host(got[k + "_scale"][i])
            assert np.allclose(sc, blocks / 448, rtol=1e-5, atol=0), (k, i)
            err = np.abs(values(got[k][i], got[k + "_scale"][i]) - x)
            unit = np.repeat(blocks / 448, 256)[:n]
            assert (err <= 2.0 ** -4 * np.abs(x) * (1 + 1e-5) + 2.0 ** -10 * unit +
                    e * (np.abs(x) + (g if k == "m" else 0))).all(), (k, i)
    else:
        assert (np.abs(host(got["m"][i]).ravel() - m) <= e * (np.abs(m) + g)).all()
        assert (np.abs(host(got["v"][i]).ravel() - v) <= e * v).all()


@pytest.mark.parametrize("g_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
def test_sizes(bits, g_dt):
    t = draw(SIZES, bits, g_dt, seed=bits)
    before = clone(t)
    call(t)
    for i in range(len(SIZES)):
        check(t, before, i)
        assert torch.equal(t["g"][i], before["g"][i])


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(bits):
    """Over a hundred tensors, empty ones among them; shapes of any number of dimensions."""
    sizes = [(7 * i) % 600 for i in range(101)]
    t = draw(sizes, bits, seed=3)
    t["p"][50] = t["p"][50].view(-1, 2)
    t["g"][50] = t["g"][50].view(-1, 2)
    t["m"][50], t["v"][50] = t["m"][50].view(-1, 2), t["v"][50].view(-1, 2)
    before = clone(t)
    call(t)
    for i in range(101):
        if sizes[i]:
            check(t, before, i)


@pytest.mark.parametrize("step", [1, 2, 100, 1000000])
def test_steps_and_options(step):
    t = draw([300, 5000], 32, seed=step)
    kw = dict(beta1=0.8, beta2=0.95, eps=1e-6, weight_decay=0.3)
    coef = torch.full((1,), 0.25, device=dev())
    copies = [torch.zeros(n, device=dev()).bfloat16() for n in (300, 5000)]
    before = clone(t)
    call(t, step=step, lr=3e-3, grad_scale=coef, copies=copies, **kw)
    for i in range(2):
        check(t, before, i, lr=3e-3, step=step, gs=0.25, **kw)
        assert torch.equal(copies[i], t["p"][i].bfloat16())


def test_zero_betas_and_zero_rate():
    t = draw([600], 32)
    before = clone(t)
    call(t, beta1=0.0, beta2=0.0, eps=1e-8, weight_decay=0.0)
    g = host(before["g"][0])
    assert np.allclose(host(t["p"][0]), host(before["p"][0]) - 1e-2 * g / (np.abs(g) + 1e-8),
                       atol=1e-6)
    t = draw([600], 32)
    before = clone(t)
    call(t, lr=0.0)
    assert torch.equal(t["p"][0], before["p"][0])
    assert not torch.equal(t["m"][0], before["m"][0])


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_zeros(bits):
    """All states zero: the step is lr g / (|g| + eps), whatever the gradient's size."""
    t = draw([777], bits)
    for k in t:
        if k not in "pg":
            t[k] = [torch.zeros_like(x) for x in t[k]]
    t["g"][0][:5] = 0.0
    before = clone(t)
    call(t, step=1, weight_decay=0.0, eps=1e-12)
    g = host(before["g"][0])
    assert np.allclose(host(t["p"][0]), host(before["p"][0]) - 1e-2 * np.sign(g), atol=1e-6)


@pytest.mark.parametrize("bits", [32, 8])
def test_out_of_place(bits):
    t = draw(SIZES, bits, seed=5)
    before = clone(t)
    out = {k: [torch.full_like(x, 3.0) if x.dtype != E4M3 else torch.zeros_like(x) for x in v]
           for k, v in t.items() if k != "g"}
    call(t, out=out)
    for k in t:
        for a, b in zip(t[k], before[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
    call(t)
    for k in out:
        for a, b in zip(t[k], out[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


@pytest.mark.parametrize("bits", [32, 8])
def test_views_at_any_element(bits):
    """Tensors that start and end anywhere inside a buffer; what lies around them stays."""
    n, at = 1111, 3
    t = draw([n + 10], bits, seed=8)
    before = clone(t)
    inner = {k: [x[at:at + n] if "scale" not in k else x[:-(-n // 256)] for x in v]
             for k, v in t.items()}
    fresh = clone(inner)
    call(inner)
    call(fresh)
    for k in ("p", "m", "v"):
        a, b, c = (x[k][0].view(torch.uint8) for x in (t, before, fresh))
        e = a.numel() // (n + 10)
        assert torch.equal(a[at * e:(at + n) * e], c), k
        assert torch.equal(a[:at * e], b[:at * e]) and torch.equal(a[(at + n) * e:],
                                                                   b[(at + n) * e:]), k


def test_codes_are_the_nearest_values():
    """With beta1 = 0 and beta2 = 0 the states are the gradient itself: its codes are the nearest
    of the 8-bit type's values, ties to an even code."""
    vals = layer.e4m3_values()
    x = np.concatenate([vals, (vals[1:] + vals[:-1]) / 2, vals[1:] * 1.03])
    x = x[x <= 448][:255]
    g = np.zeros(512, dtype=np.float32)
    g[:len(x)] = x
    g[255], g[256 + 255] = 448.0, -448.0  # the scales are 1
    g[256:256 + len(x)] = -x
    t = draw([512], 8)
    t["g"] = [torch.from_numpy(g).to(dev())]
    call(t, beta1=0.0, beta2=0.0)
    assert (host(t["m_scale"][0]) == 1.0).all() and (host(t["v_scale"][0]) == 1.0).all()
    dist = np.abs(np.abs(g)[:, None] - vals[None, :])
    near = dist.argmin(1)
    tie = np.isclose(np.sort(dist, 1)[:, 0], np.sort(dist, 1)[:, 1], rtol=0, atol=1e-9)
    near = np.where(tie & (near % 2 == 1), near + 1, near)
    assert np.array_equal(np.abs(host(t["m"][0])), vals[near])
    assert np.array_equal(host(t["v"][0]), vals[near])
    assert (np.sign(host(t["m"][0])) * np.sign(g) >= 0).all()


def test_bad_gradients():
    for bits in (32, 8):
        t = draw([700], bits, seed=9)
        t["g"][0][10] = float("nan")
        t["g"][0][300] = float("inf")
        call(t)
        p = host(t["p"][0])
        assert np.isnan(p[10])
        rest = np.delete(p, [10, 300])
        assert np.isfinite(rest).all()
        m = host(t["m"][0]) if bits == 32 else values(t["m"][0], t["m_scale"][0])
        assert np.isnan(m[10]) and np.isfinite(np.delete(m[:256], 10)).all()
        assert not np.isfinite(m[300])
        if bits == 8:
            assert np.isnan(m[256:512]).all() and np.isfinite(m[512:]).all()


def test_step_and_rate_on_the_device_and_replays():
    """A captured step reads its number and rate at every replay."""
    t = draw([3000, 17], 32, seed=4)
    twin = clone(t)
    step = torch.ones(1, dtype=torch.int32, device=dev())
    lr = torch.full((1,), 1e-2, device=dev())
    call(clone(t), step=step, lr=lr)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(t, step=step, lr=lr)
        step += 1
    for n in range(1, 5):
        lr.fill_(1e-2 / n)
        for a, b in zip(t["g"], twin["g"]):
            a.copy_(torch.randn_like(a) * 1e-2)
            b.copy_(a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        before = clone(twin)
        call(twin, step=n, lr=1e-2 / n)
        for i in range(2):
            check(t, before, i, step=n, lr=float(np.float32(1e-2 / n)))
            for k in ("p", "m", "v"):
                twin[k][i].copy_(t[k][i])


def test_one_large_tensor():
    """Offsets past 2^32 bytes."""
    n = (1 << 30) + 4097 + 3
    p = torch.zeros(n, device=dev())
    g = torch.ones(n, device=dev()).bfloat16()
    m, v = (torch.zeros(n, dtype=torch.uint8, device=dev()).view(E4M3) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device=dev()) for _ in range(2))
    nb.adamw_step([p], [g], [m], [v], 1, 0.5, weight_decay=0.0, m_scale=[ms], v_scale=[vs])
    assert float(p[-1]) == pytest.approx(-0.5, rel=1e-6)
    assert float(p.min()) == float(p.max())
    assert float(ms.min()) == float(ms.max()) > 0
    assert float(m[-3:].float().min()) == 448.0
