"""The language-model example end to end: distillation lowers the loss, a decode step with 4-bit
weights gives what the whole-sequence forward gives with the weights they stand for, and generation
keeps to the grammar."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import dev, host
from oracle import lm
from selective_state_space_naju_amd import binding as nb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def model():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")
    import language_model
    m = language_model.Model(vocab=203, d_model=64, d_inner=128)
    print("train", flush=True)
    m.losses = language_model.train(m, 30, batch=4, length=96)
    m.quantise()
    return m


def test_distillation_lowers_the_loss(model):
    print("  loss %.3f -> %.3f" % (model.losses[0], model.losses[-1]), flush=True)
    assert np.isfinite(model.losses).all()
    assert model.losses[-1] < 0.8 * model.losses[0]


def test_decode_steps_match_the_sequence_forward(model):
    """Prompt through decode steps against the sequence path with dequantised weights: both round
    to bf16 at the same points, in another order, and the sequence path's weights once more
    (2^-9 relative each); a few percent of the logits' size over two layers."""
    import language_model
    ids = torch.arange(40, dtype=torch.int32, device=dev()).view(2, 20) * 5 % 203
    state = model.start(2)
    for t in range(20):
        got = model.decode(ids[:, t].contiguous(), state)

    def back(pair):
        q, s = pair
        w = lm.w4_weights(q.cpu().numpy(), host(s), language_model.GROUP)
        return torch.from_numpy(w.T.copy()).to(dev()).bfloat16()
    twin = language_model.Model(vocab=203, d_model=64, d_inner=128)
    twin.E, twin.E_bf16 = model.E, model.E_bf16
    twin.bf16 = [{k: (back(w[k]) if k in language_model.QUANTISED else v) for k, v in p.items()}
                 for p, w in zip(model.bf16, model.w4)]
    x, _ = twin.forward(ids)
    y, _ = language_model.norm(x[:, -1])
    want = host(y) @ lm.w4_weights(model.w4_head[0].cpu().numpy(), host(model.w4_head[1]),
                                   language_model.GROUP).T
    err = np.linalg.norm(host(got) - want) / np.linalg.norm(want)
    print("  decode against sequence: relative error %.2e" % err, flush=True)
    assert err < 0.05


def test_generation_keeps_to_the_grammar(model):
    words = np.zeros((2, 7), dtype=np.uint32)
    allowed = [{3, 77, 150, 202}, set(range(10, 60))]
    for b, tokens in enumerate(allowed):
        for v in tokens:
            words[b, v // 32] |= np.uint32(1 << (v % 32))
    mask = torch.from_numpy(words.view(np.int32)).to(dev())
    prompt = torch.tensor([[1, 2, 3], [4, 5, 6]], dtype=torch.int32, device=dev())
    out = model.generate(prompt, 12, repetition=1.3, mask=mask)
    again = model.generate(prompt, 12, repetition=1.3, mask=mask)
    assert torch.equal(out, again)
    for b in range(2):
        assert set(out[b].tolist()) <= allowed[b]
    nothing = model.generate(prompt, 2, mask=torch.zeros_like(mask))
    assert (nothing == -1).all()  # and the padding token decodes without a fault


def test_tied_gradient_adds_the_looked_up_rows(model):
    ids = torch.tensor([5, 5, 9, -1], dtype=torch.int32, device=dev())
    d = torch.randn(4, 64, device=dev())
    base = torch.randn(203, 64, device=dev())
    got = nb.embed_bwd(ids, d, 203, 2.0, dW=base.clone())
    want = base.clone()
    want[5] += 2 * (d[0] + d[1])
    want[9] += 2 * d[2]
    assert torch.allclose(got, want, rtol=1e-6, atol=1e-5)
