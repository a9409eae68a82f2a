"""The 4-bit linear layer in every form that sizes choose: waves that split the inputs (d_out below
24576) and waves that do not, 1-4, 5-8, 9-16, 17-32 and 33-64 rows, inputs that fit the staging
memory at once and inputs that take several stages and end inside a block of 128.  The bound is
test_gpu_w4's; of wide layers the first, the last and some other outputs are compared."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev
from selective_state_space_naju_amd import binding as nb
from test_gpu_w4 import call, check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


CASES = [  # rows, d_in, d_out, group, zeros, bias and residual
    # waves side by side, one stage
    (5, 386, 24600, 64, True, True),
    (8, 200, 24576, 32, False, False),
    (9, 514, 24601, 128, True, False),
    (16, 258, 24600, 64, False, True),
    # several stages
    (3, 15010, 24600, 128, False, True),
    (8, 7510, 24577, 64, True, False),
    (16, 4010, 24600, 32, True, True),
    (16, 2050, 33000, 64, False, False),
    (32, 4130, 24600, 128, True, False),
    (32, 1030, 66000, 32, False, True),
    (64, 2110, 24590, 32, True, False),
    (64, 700, 33001, 64, False, True),
    # waves that split the inputs, several stages
    (3, 30002, 100, 32, True, True),
    (8, 12010, 70, 64, False, False),
    (16, 9002, 33, 128, True, False),
    (32, 5010, 100, 64, False, True),
    (64, 2502, 47, 32, True, False),
    (16, 3002, 20000, 32, True, True),
    # one output less than the rule's border
    (4, 260, 24575, 64, True, False),
    (64, 260, 24575, 64, False, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "r%d_k%d_n%d_g%d_z%d_e%d" % c)
def test_w4_form(case):
    R, K, N, G, zeros, extra = case
    print("w4 form", case, flush=True)
    x, q, s, z, bias, res = draw(R, K, N, G, 42, zeros, extra)
    y = call(x, q, s, G, z, bias, res)
    rng = np.random.default_rng(43)
    some = np.unique(np.concatenate([np.arange(min(N, 130)), np.arange(max(0, N - 130), N),
                                     rng.integers(0, N, 200)]))
    at = torch.from_numpy(some).to(dev())
    check(y[:, at], x, q[some], s[some], G, None if z is None else z[some],
          None if bias is None else bias[some], None if res is None else res[:, some])
