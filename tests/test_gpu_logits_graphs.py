"""The logits' records between the tiles of a row, under graph capture: graphs captured without a
call before them, replayed in any order and beside eager calls; and what is kept between calls."""
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


def draw(R, V, seed):
    g = torch.Generator(device=dev())
    g.manual_seed(seed)
    x = torch.randn(R, V, generator=g, device=dev())
    hist = torch.randint(0, V, (R, 50), generator=g, device=dev(), dtype=torch.int32)
    return x, hist, torch.full((R,), 1.3, device=dev())


def call(a):
    return nb.logits_process(a[0], a[1], None, a[2])


def test_graphs_captured_without_a_warm_up_replay_in_any_order():
    """Rows of several tiles.  A graph before them leaves ones all over the graphs' memory when it
    is replayed, so records that a graph does not clear itself show."""
    R, V = 5, 70001
    a, b = draw(R, V, 1), draw(R, V, 2)
    want_a, want_b = call(a), call(b)
    torch.cuda.synchronize()
    side, pool = torch.cuda.Stream(), torch.cuda.graph_pool_handle()
    ones, ga, gb = (torch.cuda.CUDAGraph() for _ in range(3))
    with torch.cuda.graph(ones, pool=pool, stream=side):
        full = [torch.empty(1 << 20, dtype=torch.uint8, device=dev()).fill_(255)
                for _ in range(4)]
        del full
    with torch.cuda.graph(ga, pool=pool, stream=side):
        got_a = call(a)
    with torch.cuda.graph(gb, pool=pool, stream=side):
        got_b = call(b)
    for order in ((gb,), (ga,), (gb, ga), (ga, gb, gb)):
        ones.replay()
        torch.cuda.synchronize()
        for graph in order:
            graph.replay()
            torch.cuda.synchronize()
            got, want = (got_a, want_a) if graph is ga else (got_b, want_b)
            assert torch.equal(got[1], want[1]) and torch.equal(got[0], want[0])
        with torch.cuda.stream(side):  # eager calls on the stream of the capture
            again = call(a)
        side.synchronize()
        assert torch.equal(again[1], want_a[1])


def test_rows_that_vary_keep_one_buffer():
    x, hist, rep = draw(200, 20000, 3)
    call((x, hist, rep))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for R in range(1, 200, 7):
        call((x[:R], hist[:R], rep[:R]))
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


def test_rows_that_grow_past_the_buffer():
    x, hist, rep = draw(1500, 20000, 4)
    want = None
    for R in (3, 1500, 700, 3):
        out, best = call((x[:R], hist[:R], rep[:R]))
        want = call((x, hist, rep)) if want is None else want
        assert torch.equal(out, want[0][:R]) and torch.equal(best, want[1][:R])
