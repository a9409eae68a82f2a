"""Rows that hold NaN, and nothing above -inf beside it: NaN reaches everything the row gives, in
the forward, the backward and the joint call; rows of -inf alone keep their meaning, and no row
disturbs another."""
import numpy as np
import pytest
import torch

from gpu_helpers import dev, f32_dev, to_dev
from oracle import lm
from selective_state_space_naju_amd import binding as nb
from test_gpu_distill import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


@pytest.mark.parametrize("io,V", [("f32", 3), ("bf16", 6), ("f32", 40), ("bf16", 3000),
                                  ("f32", 20001), ("bf16", 50001), ("f32", 70000),
                                  ("bf16", 140000)])
def test_distill_rows_of_nan(io, V):
    print("distill nan", io, V, flush=True)
    rng = np.random.default_rng(16)
    R, k = 8, 3
    x = rng.standard_normal((R, V)).astype(np.float32)
    ids = np.stack([rng.permutation(V)[:k] for _ in range(R)])
    t = rng.standard_normal((R, k)).astype(np.float32)
    x[0] = np.nan
    x[2] = -np.inf                # NaN at a listed token, -inf everywhere else
    x[2, ids[2, 0]] = np.nan
    x[4] = np.nan                 # a listed token at -inf, NaN everywhere else
    x[4, ids[4, 0]] = -np.inf
    x[5] = -np.inf                # NaN at one token (not listed, if there are others)
    x[5, [v for v in range(V) if v not in ids[5]][:1] or 0] = np.nan
    x[6] = -np.inf
    nan_rows, others = [0, 2, 4, 5], [1, 3, 7]
    X, I, T, G = to_dev(x, io), i32(ids), f32_dev(t), torch.ones(R, device=dev())
    loss, lse = nb.distill_fwd(X, I, T)
    loss2, grad2 = nb.distill_fwd_bwd(X, I, T, G)
    grad = nb.distill_bwd(X, I, T, lse, G)
    for out in (loss, lse, loss2, grad, grad2):
        assert torch.isnan(out[nan_rows]).all()
        assert torch.isfinite(out[others]).all()
    # no probability anywhere: lse -inf, and the listed tokens draw against nothing
    ref_loss, ref_lse, ref_grad = lm.distill(x, ids, t, 1.0, np.ones(R))
    assert np.isnan(ref_grad[nan_rows]).all() and np.isnan(ref_loss[nan_rows]).all()
    assert lse[6] == -np.inf and loss[6] == np.inf and loss2[6] == np.inf
    want = torch.from_numpy(ref_grad[6]).to(dev())
    for g in (grad, grad2):
        assert torch.allclose(g[6].double(), want, rtol=2 ** -8, atol=0)
