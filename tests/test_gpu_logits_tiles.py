"""Logits processing at the borders of its tiles: 4096 tokens of a row a workgroup while there are
few of them, 16384 where rows times the row's tiles of that size reach 64.  The bounds are
test_gpu_logits's."""
import pytest
import torch

from selective_state_space_naju_amd import binding as nb
from test_gpu_logits import call, check, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


CASES = [  # rows, vocab, history, biases, io, grammar, pad
    (2, 4095, 300, 20, "f32", True, 0),
    (2, 4096, 300, 20, "bf16", True, 1),
    (2, 4097, 300, 20, "f32", True, 0),
    (3, 8193, 9000, 100, "bf16", False, 0),
    (2, 16384, 900, 4000, "f32", True, 3),
    (2, 16385, 900, 40, "bf16", True, 0),
    (31, 16385, 60, 5, "f32", True, 0),     # 62 large tiles would do: small ones
    (64, 16383, 60, 5, "bf16", True, 0),
    (64, 16384, 20000, 5, "f32", False, 0),  # a list as long as the tile
    (32, 16385, 60, 5, "f32", True, 1),     # 64: large ones, the second holds one token
    (22, 32769, 60, 50, "bf16", True, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "r%d_v%d_h%d_n%d_%s_g%d_pad%d" % c)
def test_logits_tiles(case):
    R, V, H, n, io, grammar, pad = case
    print("logits tiles", case, flush=True)
    a = draw(R, V, H, n, io, 25, grammar)
    check(a, *call(a, io, pad))
