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
