"""Quantisation of weights whose extremes lie further apart than the largest number.

The step is (max - min) / 15 rounded to bf16; dividing before subtracting costs one rounding more,
2^-24.  Weights within half a step of their code, and a step of slack for z's and the scale's own
rounding, as for ordinary weights."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, host, to_dev
from oracle import lm
from selective_state_space_naju_amd import binding as nb
from selective_state_space_naju_amd import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_w4_quantize_of_extremes_beyond_the_largest_difference(io):
    K, N, G = 128, 33, 64
    rng = np.random.default_rng(41)
    W = (rng.uniform(-1, 1, (K, N)) * 3.3e38).astype(np.float32)
    W[0], W[1] = -3.3e38, 3.3e38
    W[64], W[65] = 3.3e38, -3.3e38
    W = inputs.bf16_round(W) if io == "bf16" else W
    q, s, z = nb.w4_quantize(to_dev(W, io), G, zeros=True)
    sd = host(s)
    for g in range(K // G):
        w = W[g * G:(g + 1) * G].astype(np.float64)
        step = (w.max(0) - w.min(0)) / 15
        assert np.allclose(sd[:, g], step, rtol=2.0 ** -8, atol=0)
    back = lm.w4_weights(q.cpu().numpy(), sd, G, z.cpu().numpy())
    slack = 1.0 + 15 * 2.0 ** -8
    assert np.all(np.abs(back.T - W) <= slack * np.repeat(sd.T, G, 0))
