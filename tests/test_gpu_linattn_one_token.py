"""Linear attention over one token a row that is cut from longer tensors: whatever the distance of
the rows, it gives what the token gives alone."""
import pytest
import torch

from gpu_helpers import dev
from selective_state_space_naju_amd import binding as nb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    nb.lib()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,H,Hk,d", [(3, 1000, 16, 16, 128), (2, 700, 12, 3, 136),
                                        (2, 30000, 4, 2, 16)])
def test_last_token_of_a_longer_tensor(B, T, H, Hk, d, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    # q, k and v as parts of one tensor; rows lie T (H + 2 Hk) d elements apart
    joint = torch.randn(B, T, (H + 2 * Hk), d, generator=g, device=dev()).to(dt)
    parts = [joint[:, -1:, a:b] for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk))]
    assert parts[0].stride(0) > 1 << 20
    a = torch.linspace(-0.5, 0.0, H, device=dev())
    s, ds = (torch.randn(B, H, d, d, generator=g, device=dev()) for _ in range(2))
    do = torch.randn(B, 1, H, d, generator=g, device=dev()).to(dt)
    n = torch.tensor([1, 0, 5][:B], dtype=torch.int32, device=dev())
    alone = [t.clone(memory_format=torch.contiguous_format) for t in parts]
    for lengths in (None, n):
        print("B %d T %d H %d d %d %s" % (B, T, H, d, dt), flush=True)
        o, new = nb.linattn_fwd(*parts, a, s, lengths)
        wo, wnew = nb.linattn_fwd(*alone, a, s, lengths)
        assert torch.equal(o, wo) and torch.equal(new, wnew)
        got = nb.linattn_bwd(*parts, a, do, s, ds, lengths)
        want = nb.linattn_bwd(*alone, a, do, s, ds, lengths)
        for k in want:
            assert torch.equal(got[k], want[k]), k
