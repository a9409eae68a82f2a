"""The operators around the mixer layer where element and byte offsets pass 2^31 and 2^32: the far
end of a large tensor gives, bit for bit, what the same rows give alone.  And the same calls
captured in a HIP graph and replayed."""
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


def tokens(shape, vocab):
    return torch.randint(0, vocab, shape, device=dev(), dtype=torch.int32)


def test_distill_far_rows():
    R, V, k = 33000, 131071, 3  # 4.3e9 logits
    print("distill", R, V, flush=True)
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=dev())
    x[-2:] = torch.randn(2, V, device=dev()) * 2
    ids, t = tokens((R, k), V), torch.randn(R, k, device=dev())
    g = torch.ones(R, device=dev())
    loss, grad = nb.distill_fwd_bwd(x, ids, t, g, 2.0)
    own = (x[-2:].clone(), ids[-2:].clone(), t[-2:].clone())
    l2, lse = nb.distill_fwd(*own, 2.0)
    far = nb.distill_bwd(x, ids, t, torch.cat((torch.zeros(R - 2, device=dev()), lse)), g, 2.0)
    few = nb.distill_bwd(*own, lse, g[-2:].clone(), 2.0)
    assert torch.equal(far[-2:], few)
    # the joint call forms q over the row's sum, the other from lse: both round to bf16
    assert torch.allclose(grad[-2:].float(), few.float(), rtol=2 ** -7, atol=1e-9)
    assert torch.allclose(loss[-2:], l2, rtol=1e-6, atol=1e-6)


def test_logits_far_rows():
    R, V = 17000, 131072  # 2.2e9 results of 4 bytes
    print("logits", R, V, flush=True)
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=dev())
    x[-3:] = torch.randn(3, V, device=dev())
    hist, f = tokens((R, 9), V), torch.full((R,), 0.5, device=dev())
    out, best = nb.logits_process(x, hist, frequency=f)
    own, ob = nb.logits_process(x[-3:].clone(), hist[-3:].clone(), frequency=f[-3:].clone())
    assert torch.equal(out[-3:], own) and torch.equal(best[-3:], ob)


def test_embed_far_rows():
    V, d, T = 4200000, 1024, 300  # 4.3e9 elements
    print("embed", V, d, flush=True)
    W = torch.zeros(V, d, dtype=torch.bfloat16, device=dev())
    W[-50:] = torch.randn(50, d, device=dev())
    ids = V - 1 - tokens((T,), 50)
    out = nb.embed_fwd(ids, W, 3.0)
    assert torch.equal(out, nb.embed_fwd(ids - (V - 50), W[-50:].clone(), 3.0))
    del W
    dW = nb.embed_bwd(ids, out, V, 0.5)
    assert torch.equal(dW[-50:], nb.embed_bwd(ids - (V - 50), out, 50, 0.5))
    assert not dW[:-50].any()


def test_embed_grad_of_few_tokens_over_a_vocabulary_past_the_small_sort():
    V, d = 1048577, 4
    ids = torch.tensor([V - 1, 0, V - 1, V, 524288, -1, 0], dtype=torch.int32, device=dev())
    dW = nb.embed_bwd(ids, torch.ones(7, d, device=dev()), V)
    want = torch.zeros(V, d, device=dev())
    want[0], want[V - 1], want[524288] = 2, 2, 1
    assert torch.equal(dW, want)


def test_w4_far_outputs():
    K, N, R = 4096, 2100000, 2  # 4.3e9 bytes of codes
    print("w4", K, N, flush=True)
    q = torch.zeros(N, K // 2, dtype=torch.uint8, device=dev())
    q[-100:] = torch.randint(0, 256, (100, K // 2), device=dev(), dtype=torch.uint8)
    s = torch.full((N, K // 128), 0.01, dtype=torch.bfloat16, device=dev())
    x = torch.randn(R, K, device=dev()).bfloat16()
    y = nb.w4_linear(x, q, s, 128)
    # (few outputs split the inputs over waves: the fp32 sums differ in order)
    few = nb.w4_linear(x, q[-100:].clone(), s[-100:].clone(), 128)
    assert torch.allclose(y[:, -100:].float(), few.float(), rtol=2 ** -7, atol=1e-3)


def test_operators_in_a_replayed_graph():
    V, d, T, k = 5003, 96, 700, 8
    ids = tokens((T,), V)
    W = torch.randn(V, d, device=dev()).bfloat16()
    logits = torch.randn(T, V, device=dev()).bfloat16()
    t_ids, t = tokens((T, k), V), torch.randn(T, k, device=dev())
    g = torch.rand(T, device=dev())
    hist = tokens((T, 40), V)
    rep = torch.full((T,), 1.2, device=dev())
    q, s, z = nb.w4_quantize(torch.randn(d, V, device=dev()), 32, zeros=True)

    def run():
        x = nb.embed_fwd(ids, W, 2.0)
        dW = nb.embed_bwd(ids, x, V)
        loss, dl = nb.distill_fwd_bwd(logits, t_ids, t, g)
        out, best = nb.logits_process(logits, hist, None, rep)
        y = nb.w4_linear(x, q, s, 32, z)
        return x, dW, loss, dl, out, best, y
    eager = run()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            captured = run()
    for _ in range(3):
        for c in captured:
            c.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("x", "dW", "loss", "dl", "out", "best", "y"), captured, eager):
            assert torch.equal(a, b), name
        again = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, eager))
