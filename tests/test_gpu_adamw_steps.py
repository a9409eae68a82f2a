"""The AdamW step's 8-bit states over many steps, against the fp64 update with states that are not
rounded: what storing them does to the steps after."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


class Run:
    """One tensor of n elements with 8-bit states, and the fp64 moments beside it; lr 1 and no
    weight decay, so that p moves by the step itself."""

    def __init__(self, n, **kw):
        self.n, self.t, self.kw = n, 0, kw
        self.p = torch.zeros(n, device=dev())
        self.m, self.v = (torch.zeros(n, device=dev()).to(E4M3) for _ in range(2))
        self.ms, self.vs = (torch.zeros(-(-n // 256), device=dev()) for _ in range(2))
        self.M, self.V = (torch.zeros(n, dtype=torch.float64, device=dev()) for _ in range(2))

    def step(self, g):
        """The change of p, and what exact states give."""
        self.t += 1
        before = self.p.clone()
        nb.adamw_step([self.p], [g], [self.m], [self.v], self.t, 1.0, weight_decay=0.0,
                      m_scale=[self.ms], v_scale=[self.vs], **self.kw)
        self.M.mul_(0.9).add_(g.double(), alpha=0.1)
        self.V.mul_(0.999).addcmul_(g.double(), g.double(), value=0.001)
        want = self.M / (1 - 0.9 ** self.t) / ((self.V / (1 - 0.999 ** self.t)).sqrt() + 1e-8)
        return before - self.p, want

    def code(self, k):
        return getattr(self, k).view(torch.uint8) & 127

    def root(self):
        """The stored root of v."""
        return self.v.float() * self.vs.repeat_interleave(256)[:self.n]


def mixed_blocks(n, seed):
    """Half of each block with gradients of size 1 at every step, half with ones of 1e-5 to 6e-5 in
    one step of twenty: rows of a table that most batches do not look up, beside those they do."""
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    rand = lambda f: f(n, generator=g, device=dev())  # noqa: E731
    quiet = torch.arange(n, device=dev()) % 256 >= 128
    size = 1e-5 + 5e-5 * rand(torch.rand)

    def draw():
        x = rand(torch.randn)
        return torch.where(quiet, size * x.sign() * (rand(torch.rand) < 0.05), x)
    return quiet, draw


def test_small_roots_beside_large_ones():
    """Exact states move an element by at most 0.1 / sqrt(0.001 (1 - 0.81 / 0.999)) = 7.3 lr
    (Cauchy's inequality for the two sums).  A stored first moment is at most twice its value (the
    smallest code in place of half of it), which the 0.9 of it that the next step keeps can add up
    to 0.1 / (1 - 0.9 * 17 / 16) = 2.3 times; a stored root is at least 2 / 3 of its own (a code in
    place of one and a half): 7.3 * 2 * 2.3 * 1.5 = 50.  A root lost altogether moves it by
    hundreds."""
    n = 256 * 8 + 77
    run = Run(n)
    quiet, draw = mixed_blocks(n, 1)
    most = exact = 0.0
    for _ in range(400):
        got, want = run.step(draw())
        most, exact = max(most, float(got.abs().max())), max(exact, float(want.abs().max()))
    print("  largest step %.2f lr, of exact states %.2f" % (most, exact), flush=True)
    assert exact <= 7.3 and most <= 50.0
    # where the first moment is kept, so is the root
    assert not ((run.code("m") != 0) & (run.code("v") == 0)).any()
    assert ((run.code("m") != 0) & quiet).any()


def test_roots_that_are_kept_are_the_smallest_code():
    """A root below half the smallest code is stored as that code (2^-9 of the scale) beside a first
    moment that is not 0, and as 0 beside one that is."""
    n = 512
    m, v = torch.zeros(n, device=dev()), torch.zeros(n, device=dev())
    m[::256], v[::256] = 0.448, 448.0  # units of 0.001 and of 1
    m[1], v[1] = 2.0 ** -9 * 0.001, 0.0
    m[2], v[2] = -0.3, 0.0
    m[3], v[3] = 0.0, 0.0
    g = torch.zeros(n, device=dev())
    ms, vs = torch.full((2,), 0.001, device=dev()), torch.ones(2, device=dev())
    codes = [(m / 0.001).to(E4M3), v.to(E4M3)]
    g[1:4] = 1e-9
    nb.adamw_step([torch.zeros(n, device=dev())], [g], [codes[0]], [codes[1]], 7, 1e-3,
                  m_scale=[ms], v_scale=[vs])
    got = host(codes[1])
    assert got[0] == 448 and got[1] == got[2] == 2.0 ** -9 and (got[3:256] == 0).all()
    # the scale 0 of a block without gradients and states holds zeros
    z = [torch.zeros(n, device=dev()).to(E4M3) for _ in range(2)]
    zs = [torch.zeros(2, device=dev()) for _ in range(2)]
    nb.adamw_step([torch.zeros(n, device=dev())], [torch.zeros(n, device=dev())], z[:1], z[1:], 7,
                  1e-3, m_scale=zs[:1], v_scale=zs[1:])
    for x in z + zs:
        assert not np.any(host(x))


# --------------------------------------------------------------------- stochastic rounding
def neighbours(x):
    """The 8-bit type's values around 0 <= x <= 448, and how far x is from the lower one to the
    upper one."""
    vals = torch.arange(127, dtype=torch.uint8).view(E4M3).double().to(x.device)
    i = (torch.searchsorted(vals, x.double(), right=True) - 1).clamp(0, 125)
    return vals[i], vals[i + 1], (x.double() - vals[i]) / (vals[i + 1] - vals[i])


def spread_step(g, step, stochastic=True, **kw):
    """The codes' values of m and the root of v of one step from zeros with beta1 = beta2 = 0: those
    of g and of its magnitude."""
    n = g.numel()
    m, v = (torch.zeros(n, device=dev()).to(E4M3) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device=dev()) for _ in range(2))
    nb.adamw_step([torch.zeros(n, device=dev())], [g], [m], [v], step, 0.0, 0.0, 0.0,
                  m_scale=[ms], v_scale=[vs], stochastic=stochastic, **kw)
    assert (ms == 1).all() and (vs == 1).all()
    return m, v


def test_stochastic_codes_are_neighbours_and_right_in_the_mean():
    """Values across the type's range, those of codes among them, over 3000 steps: always one of the
    two codes around the value (a code's own value: itself), the upper one in the share of steps
    that the value's place between them asks for, within six standard deviations of independent
    draws (16384 shares: 3e-5 that one of them lies outside).  v is squared and rooted in fp32, so
    its value is held to be near a code by 2^-22 of itself."""
    n, steps = 8192, 3000
    gen = torch.Generator(device=dev())
    gen.manual_seed(2)
    g = torch.exp2(torch.rand(n, generator=gen, device=dev()) * 20 - 11.3)
    vals = torch.arange(127, dtype=torch.uint8).view(E4M3).float().to(dev())
    g[1::64] = vals[torch.arange(n // 64, device=dev()) % 127]
    g[2::64] = torch.rand(n // 64, generator=gen, device=dev()) * 2.0 ** -8
    g = g.clamp(max=448)
    g[::256] = 448.0
    g[3::7] *= -1
    lo, hi, f = neighbours(g.abs())
    ups = [torch.zeros(n, dtype=torch.float64, device=dev()) for _ in range(2)]
    lifted = torch.zeros(n, dtype=torch.float64, device=dev())
    for s in range(1, steps + 1):
        m, v = spread_step(g, s)
        kept = (m.float() != 0)
        for k, x in enumerate((m, v)):
            x = x.double()
            assert (x * g >= 0).all() or k == 1
            up = x.abs() == hi
            assert (up | (x.abs() == lo)).all(), (k, s)
            if k == 1:  # (a root is kept beside a first moment: counted apart)
                alone = (lo > 0) | ~kept
                ups[k] += up & alone
                lifted += ~alone
                assert up[~alone].all()
            else:
                ups[k] += up
    for k in range(2):
        count = steps - (lifted if k == 1 else 0)
        off = (ups[k] - count * f).abs()
        if k == 1:
            off -= count * 2.0 ** -22 * hi / (hi - lo)
        z = off / (steps * f * (1 - f)).sqrt().clamp(min=1.0)
        print("  %s: largest deviation %.2f" % ("mv"[k], float(z.max())), flush=True)
        assert float(z.max()) < 6.0


def test_stochastic_roots_follow_their_gradients():
    """10000 steps; from step 1000 on the gradients of half of each block are a tenth.  A root moves
    by a code (a share u of itself, 1/16 to 1/8) with the probability that makes 0.05 % of itself a
    step, |g^2 / v - 1| times that (1 in the mean): 0.0005 u a step in the square, drawn back by
    0.001 of the distance a step, which leaves 0.0005 u / 0.002 = u / 4, a standard deviation of 12
    to 18 % (in the logarithm).  Eight of ten lie within 1.28 deviations, 0.79 to 1.26, and three
    deviations of the quantiles of 1024 elements are 0.03 more; the median is right within 5 %.
    Rounded to nearest the fallen half's median is over 5."""
    n = 256 * 8
    run = Run(n, stochastic=True)
    gen = torch.Generator(device=dev())
    gen.manual_seed(3)
    size = torch.exp(torch.randn(n, generator=gen, device=dev()))
    fallen = torch.arange(n, device=dev()) % 2 == 1
    small = torch.where(fallen, 0.1, 1.0)
    most = 0.0
    for t in range(10000):
        g = torch.randn(n, generator=gen, device=dev()) * size
        got, want = run.step(g if t < 1000 else g * small)
        if t % 100 == 0:
            most = max(most, float(got.abs().max()))
    ratio = run.root().double() / run.V.sqrt()
    for name, r in (("fallen", ratio[fallen]), ("others", ratio[~fallen])):
        q = [float(torch.quantile(r, x)) for x in (0.1, 0.5, 0.9)]
        print("  %s: stored over exact root %.3f, %.3f, %.3f" % (name, *q), flush=True)
        assert abs(q[1] - 1) < 0.05 and q[0] > 0.76 and q[2] < 1.29
    print("  largest step %.2f lr" % most, flush=True)
    assert most <= 50.0


def test_stochastic_small_roots_beside_large_ones():
    """As with rounding to nearest (the bound is that test's; here a first moment may be rounded up
    to a code in place of any part of it, but not step after step: its mean is right)."""
    n = 256 * 8 + 77
    run = Run(n, stochastic=True)
    _, draw = mixed_blocks(n, 4)
    most = 0.0
    for _ in range(400):
        most = max(most, float(run.step(draw())[0].abs().max()))
        assert not ((run.code("m") != 0) & (run.code("v") == 0)).any()
    print("  largest step %.2f lr" % most, flush=True)
    assert most <= 50.0


def test_stochastic_first_moments_end():
    """Without gradients a first moment falls to 0: its smallest code is kept with 0.9 a step, so
    after 300 steps behind the last code's 150 none of 2048 is left (0.9^150 = 1e-7)."""
    n = 2048
    run = Run(n, stochastic=True)
    for t in range(20):
        run.step(torch.randn(n, device=dev()))
    z = torch.zeros(n, device=dev())
    for t in range(20 + 450):
        z[::256] = 1.0 if t % 2 else -1.0  # (the block's scale stays)
        run.step(z)
    left = run.code("m").view(-1, 256)[:, 1:]
    assert not left.any()
    assert (run.root().view(-1, 256)[:, 1:] > 0).all()


def state_bytes(t):
    return [x.view(torch.uint8) for k in sorted(t) for x in t[k]]


@pytest.mark.parametrize("g_dt", [torch.float32, torch.bfloat16])
def test_stochastic_calls_repeat(g_dt):
    """Equal calls give equal bits, in place, out of place, with the step's number on the device, at
    any place in memory and in lists of any length; p does not depend on the rounding; another step
    rounds otherwise."""
    sizes = [1, 255, 257, 4097, 9001]
    gen = torch.Generator(device=dev())
    gen.manual_seed(5)
    rand = lambda n, s: torch.randn(n, generator=gen, device=dev()) * s  # noqa: E731
    t = dict(p=[rand(n, 0.1) for n in sizes], m=[rand(n, 100.0).clamp(-448, 448).to(E4M3)
                                                 for n in sizes],
             v=[rand(n, 100.0).abs().clamp(max=448).to(E4M3) for n in sizes],
             m_scale=[rand(-(-n // 256), 1e-4).abs() for n in sizes],
             v_scale=[rand(-(-n // 256), 1e-4).abs() for n in sizes])
    g = [rand(n, 1e-2).to(g_dt) for n in sizes]
    clone = lambda t: {k: [x.clone() for x in v] for k, v in t.items()}  # noqa: E731

    def call(t, step=7, g=g, **kw):
        nb.adamw_step(t["p"], g, t["m"], t["v"], step, 1e-2, m_scale=t["m_scale"],
                      v_scale=t["v_scale"], **{"stochastic": True, **kw})
        return t
    want = call(clone(t))
    same = lambda a: all(torch.equal(x, y) for x, y in zip(state_bytes(a),  # noqa: E731
                                                          state_bytes(want)))
    assert same(call(clone(t)))
    assert same(call(clone(t), step=torch.full((1,), 7, dtype=torch.int32, device=dev())))
    out = {k: [torch.zeros_like(x) for x in v] for k, v in t.items()}
    before = clone(t)
    call(t, out=out)
    assert same(out)
    assert all(torch.equal(x, y) for x, y in zip(state_bytes(t), state_bytes(before)))
    alone = clone(t)
    for i in range(len(sizes)):
        call({k: [v[i]] for k, v in alone.items()}, g=[g[i]])
    assert same(alone)
    def elsewhere(x):  # three bytes further than where memory blocks begin
        room = torch.zeros(x.numel() + 16, dtype=torch.uint8, device=dev())
        return room[3:3 + x.numel()].view(E4M3).copy_(x)
    moved = {k: [elsewhere(x) if k in ("m", "v") else x.clone() for x in v] for k, v in t.items()}
    assert same(call(moved))
    near, other = call(clone(t), stochastic=False), call(clone(t), step=8)
    assert all(torch.equal(x, y) for x, y in zip(near["p"], want["p"]))
    for k in ("m", "v"):
        assert not torch.equal(other[k][4].view(torch.uint8), want[k][4].view(torch.uint8)), k
        assert not torch.equal(near[k][4].view(torch.uint8), want[k][4].view(torch.uint8)), k


def test_stochastic_replays():
    """A captured step draws its numbers from the step that it reads."""
    n = 3000
    a, b = Run(n, stochastic=True), Run(n, stochastic=True)
    step = torch.zeros(1, dtype=torch.int32, device=dev())
    g = torch.zeros(n, device=dev())

    def call(r, at):
        nb.adamw_step([r.p], [g], [r.m], [r.v], at, 1e-2, m_scale=[r.ms], v_scale=[r.vs],
                      stochastic=True)
    call(Run(n), 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        call(a, step)
    for t in range(1, 6):
        g.copy_(torch.randn(n, device=dev()))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        call(b, t)
        for k in ("m", "v"):
            assert torch.equal(a.code(k), b.code(k)), (k, t)
        assert torch.equal(a.ms, b.ms) and torch.equal(a.vs, b.vs)


def test_stochastic_bad_gradients():
    """A NaN stays with its element; an infinity takes its block's states."""
    n = 700
    g = torch.randn(n, device=dev()) * 1e-2
    g[10], g[300] = float("nan"), float("inf")
    run = Run(n, stochastic=True)
    run.step(g)
    m = run.m.float() * run.ms.repeat_interleave(256)[:n]
    root = run.root()
    for x in (m, root):
        assert x[10].isnan() and not x[300].isfinite()
        assert not x[256:512].isfinite().any() and x[512:].isfinite().all()
        assert x[:256].isnan().sum() == 1
    assert run.p[10].isnan() and run.p[512:].isfinite().all()
