"""The embedding gradient's scratch: nothing of it is kept from call to call, and calls from
several host threads on one stream do not share it."""
import threading

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


def test_batches_of_varying_length_keep_no_memory():
    V, d = 400, 64
    ids = torch.randint(0, V, (6000,), device=dev(), dtype=torch.int32)
    dout = torch.randn(6000, d, device=dev())
    nb.embed_bwd(ids[:5000].contiguous(), dout[:5000], V)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in range(5000, 5040):
        nb.embed_bwd(ids[:T].contiguous(), dout[:T], V)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before


def test_a_callers_workspace_is_used():
    V, d, T = 300, 40, 5000
    ids = torch.randint(-1, V, (T,), device=dev(), dtype=torch.int32)
    dout = torch.randn(T, d, device=dev())
    ws = nb.Workspace(nb.lib().naju_embed_bwd_workspace_bytes(T, V, d), dev())
    ws.tensor.fill_(255)
    assert torch.equal(nb.embed_bwd(ids, dout, V, ws=ws), nb.embed_bwd(ids, dout, V))
    small = nb.Workspace(256, dev())
    with pytest.raises(nb.NajuError, match="needs"):
        nb.embed_bwd(ids, dout, V, ws=small)


def test_two_host_threads_on_one_stream():
    """Equal sizes, other ids: a thread's launches may fall between another's."""
    V, d, T = 900, 32, 20000
    g = torch.Generator(device=dev())
    work = []
    for n in range(2):
        g.manual_seed(n)
        ids = torch.randint(0, V, (T,), generator=g, device=dev(), dtype=torch.int32)
        dout = torch.randn(T, d, generator=g, device=dev())
        work.append((ids, dout, nb.embed_bwd(ids, dout, V)))
    torch.cuda.synchronize()
    bad, go = [], threading.Barrier(2)

    def run(n):
        ids, dout, want = work[n]
        go.wait()
        got = [nb.embed_bwd(ids, dout, V) for _ in range(40)]
        if not all(torch.equal(g, want) for g in got):
            bad.append(n)
    threads = [threading.Thread(target=run, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad
