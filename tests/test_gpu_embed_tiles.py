"""The embedding gradient at the borders of its sort: one workgroup up to 4096 tokens, tiles of 1024
up to 16384 tokens, tiles of 4096 beyond.  The bound is test_gpu_embed's."""
import numpy as np
import pytest
import torch

from gpu_helpers import f32_dev, host, to_dev
from selective_state_space_naju_amd import binding as nb
from selective_state_space_naju_amd import inputs
from test_gpu_embed import draw_ids, ids_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


CASES = [  # tokens, vocab, d, io, ids
    (1023, 5000, 10, "f32", "zipf"),
    (1025, 5000, 10, "bf16", "padded"),
    (4095, 1048575, 3, "f32", "padded"),
    (4096, 1048576, 3, "f32", "zipf"),
    (5120, 600, 17, "bf16", "zipf"),
    (5121, 600, 17, "f32", "padded"),
    (16383, 300000, 5, "f32", "zipf"),
    (16384, 511, 300, "bf16", "padded"),
    (20480, 3000, 7, "f32", "zipf"),
    (20481, 3000, 7, "bf16", "padded"),
]


@pytest.mark.parametrize("accumulate", [False, True], ids=["write", "add"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "t%d_v%d_d%d_%s_%s" % c)
def test_embed_bwd_tiles(case, accumulate):
    T, V, d, io, kind = case
    print("embed tiles", case, accumulate, flush=True)
    rng = np.random.default_rng(6)
    dout = rng.standard_normal((T, d), dtype=np.float32)
    dout = inputs.bf16_round(dout) if io == "bf16" else dout
    ids = draw_ids(rng, T, V, kind)
    before = rng.standard_normal((V, d), dtype=np.float32) if accumulate else None
    dW = f32_dev(before) if accumulate else None
    got = host(nb.embed_bwd(ids_dev(ids), to_dev(dout, io), V, 0.75, dW=dW))
    ok = (ids >= 0) & (ids < V)
    ref, size = np.zeros((V, d)), np.zeros((V, d))
    np.add.at(ref, ids[ok], 0.75 * dout[ok].astype(np.float64))
    np.add.at(size, ids[ok], 0.75 * np.abs(dout[ok]).astype(np.float64))
    n = np.bincount(ids[ok], minlength=V)[:, None]
    if accumulate:
        ref += before
        size += np.abs(before) * (n > 0)
    assert np.all(np.abs(got - ref) <= (n + 1) * 2.0 ** -23 * size)
    untouched = n[:, 0] == 0
    want = before[untouched].astype(np.float64) if accumulate else 0
    assert np.all(got[untouched] == want)
