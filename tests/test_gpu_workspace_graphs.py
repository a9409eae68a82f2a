"""Workspaces first needed under graph capture: each graph clears its own, and none is kept for
calls outside it."""
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


def scan_inputs(seed, L=301, Di=72, N=16):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev())
    h, a, b = (normal(2, L, Di).bfloat16() for _ in range(3))
    return h, a, b, normal(2, L, N).bfloat16(), normal(2, L, N).bfloat16(), normal(Di)


def test_graphs_captured_without_a_warm_up():
    x, y = scan_inputs(1), scan_inputs(2)
    want_x, want_y = nb.scan_fwd(*x, check_errors=True), nb.scan_fwd(*y, check_errors=True)
    side = torch.cuda.Stream()
    kept = len(nb._ws_cache)
    gx, gy = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gx, stream=side):
        got_x = nb.scan_fwd(*x)
    with torch.cuda.graph(gy, stream=side):
        got_y = nb.scan_fwd(*y)
    assert len(nb._ws_cache) == kept
    for graph, got, want in ((gy, got_y, want_y), (gx, got_x, want_x), (gy, got_y, want_y)):
        graph.replay()
        torch.cuda.synchronize()
        # (the look-back may fold a state in another order: bf16 results to their rounding)
        assert torch.allclose(got[0].float(), want[0].float(), rtol=2 ** -7, atol=1e-2)
        assert torch.allclose(got[1], want[1], rtol=1e-3, atol=1e-3)
    with torch.cuda.stream(side):  # an eager call on the stream of the captures
        again = nb.scan_fwd(*x, check_errors=True)
    side.synchronize()
    assert torch.allclose(again[0].float(), want_x[0].float(), rtol=2 ** -7, atol=1e-2)
    assert len(nb._ws_cache) == kept + 1
