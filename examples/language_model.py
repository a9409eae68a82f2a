"""A small language model of Naju mixer layers: trained by distillation, served with 4-bit weights.

    python examples/language_model.py [--steps N] [--tokens N]

Training step (bf16 weights, fp32 gradients):
    embedding -> [norm -> mixer layer + residual] x layers -> norm -> logits with the
    embedding's transpose -> distillation from a teacher's top logits, and the reverse of it all.
    The embedding and the output layer share one table: its gradient is the output layer's
    product, with the looked-up rows' gradient added to it.
Serving (one token per call for every sequence): embedding of the last tokens, projections with
    4-bit weights around the block's decode step, 4-bit output layer, penalties and a grammar mask
    on the logits, the best allowed token.

The teacher is a fixed table: for each token, the k most likely next ones and their logits.  Norms,
the training step's output layer, the updates, and the decode step's convolution that the gates are
projected from are plain torch; everything else goes through the library.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from selective_state_space_naju_amd import binding as nb  # noqa: E402

MIXER = ("W_u", "W_z", "conv_w", "W_a", "a_bias", "W_b", "b_bias", "W_B", "W_C", "D", "W_out")
QUANTISED = ("W_u", "W_z", "W_a", "W_b", "W_B", "W_C", "W_out")
GROUP = 32


def norm(x):
    """x over its root mean square, and that factor."""
    r = torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
    return (x.float() * r).bfloat16(), r


def norm_bwd(dy, y, r):
    y = y.float()
    return r * (dy - y * (dy * y).mean(-1, keepdim=True))


class Model:
    """Parameters as fp32 master copies; `bf16` holds what the kernels read."""

    def __init__(self, vocab, d_model=96, d_inner=192, d_state=16, layers=2, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std

        self.vocab, self.d_model, self.d_inner, self.d_state = vocab, d_model, d_inner, d_state
        self.scale = math.sqrt(d_model)
        self.E = normal(vocab, d_model, std=d_model ** -0.5)
        s_in, s_h = d_model ** -0.5, (0.355 * d_inner) ** -0.5
        self.layers = [dict(
            W_u=normal(d_model, d_inner, std=s_in), W_z=normal(d_model, d_inner, std=s_in),
            conv_w=normal(d_inner, 4, std=0.5), W_a=normal(d_inner, d_inner, std=s_h),
            a_bias=torch.full((d_inner,), 5.0, device=device),
            W_b=normal(d_inner, d_inner, std=s_h),
            b_bias=torch.full((d_inner,), -2.0, device=device),
            W_B=normal(d_inner, d_state, std=s_h), W_C=normal(d_inner, d_state, std=s_h),
            D=normal(d_inner, std=1.0), W_out=normal(d_inner, d_model, std=d_inner ** -0.5),
        ) for _ in range(layers)]
        self.refresh()

    def refresh(self):
        self.E_bf16 = self.E.bfloat16()
        self.bf16 = [{k: (v.bfloat16() if k in QUANTISED else v) for k, v in p.items()}
                     for p in self.layers]

    # ------------------------------------------------------------------- training
    def forward(self, ids):
        """The final hidden states [batch, length, d_model] and what the backward needs."""
        x = nb.embed_fwd(ids, self.E_bf16, self.scale)
        saved = []
        for p in self.bf16:
            xn, r = norm(x)
            saved.append((xn, r))
            x = nb.mixer_fwd(xn, *[p[k] for k in MIXER], res=x)
        return x, saved

    def logits(self, x):
        y, r = norm(x)
        return y, r, y.reshape(-1, self.d_model) @ self.E_bf16.t().contiguous()

    def step(self, ids, t_ids, t_logits, weight, lr, temperature=1.0):
        """One training step; returns the mean loss (a tensor, not synchronised)."""
        x, saved = self.forward(ids)
        y, r, logits = self.logits(x)
        loss, dlogits = nb.distill_fwd_bwd(logits, t_ids, t_logits, weight, temperature)
        y2 = y.reshape(-1, self.d_model)
        dE = (dlogits.t().contiguous() @ y2).float()
        dx = norm_bwd((dlogits @ self.E_bf16).float().view_as(y), y, r)
        grads = []
        for p, (xn, rn) in zip(reversed(self.bf16), reversed(saved)):
            g = nb.mixer_bwd(xn, *[p[k] for k in MIXER], dx.bfloat16())
            dx = dx + norm_bwd(g["dxn"], xn, rn)
            grads.append(g)
        # the looked-up rows' gradient joins the output layer's
        nb.embed_bwd(ids, dx.bfloat16(), self.vocab, self.scale, dW=dE)
        self.E -= lr * dE / dE.norm().clamp(min=1e-6)
        for p, g in zip(self.layers, reversed(grads)):
            for k in MIXER:
                d = g["d" + k]
                p[k] -= lr * d / d.norm().clamp(min=1e-6) * (0.1 if k in ("a_bias", "b_bias") else 1)
        self.refresh()
        return (loss * weight).sum()

    # -------------------------------------------------------------------- serving
    def quantise(self):
        """4-bit weights of every projection, and of the output layer ([d_model, vocab])."""
        self.w4 = [{k: nb.w4_quantize(p[k], GROUP)[:2] for k in QUANTISED} for p in self.bf16]
        self.w4_head = nb.w4_quantize(self.E_bf16.t().contiguous(), GROUP)[:2]

    def start(self, batch):
        """The state of `batch` sequences: per layer the scan state and the conv window."""
        dev = self.E.device
        return [(torch.zeros(batch, self.d_inner, self.d_state, device=dev),
                 torch.zeros(batch, 3, self.d_inner, dtype=torch.bfloat16, device=dev))
                for _ in self.layers]

    def decode(self, tokens, state):
        """Logits [batch, vocab] after the given tokens [batch] (int32); the state moves on."""
        x = nb.embed_fwd(tokens, self.E_bf16, self.scale)
        for p, w, (scan, window) in zip(self.bf16, self.w4, state):
            def lin(v, k, bias=None, res=None):
                return nb.w4_linear(v, *w[k], GROUP, None, bias, res)
            xn, _ = norm(x)
            u, z = lin(xn, "W_u"), lin(xn, "W_z")
            taps = torch.cat((window, u.unsqueeze(1)), dim=1).float()
            h = torch.nn.functional.silu((taps * p["conv_w"].t()).sum(1)).bfloat16()
            a, b = lin(h, "W_a", p["a_bias"]), lin(h, "W_b", p["b_bias"])
            y = nb.block_step(u, z, p["conv_w"], window, a, b, lin(h, "W_B"), lin(h, "W_C"),
                              p["D"], scan)
            x = lin(y, "W_out", None, x)
        return nb.w4_linear(norm(x)[0], *self.w4_head, GROUP)

    def generate(self, prompt, n, repetition=1.1, mask=None):
        """n tokens after the prompt [batch, length]: the best allowed one each time."""
        batch, length = prompt.shape
        dev = prompt.device
        history = torch.full((batch, length + n), -1, dtype=torch.int32, device=dev)
        history[:, :length] = prompt
        lengths = torch.full((batch,), length, dtype=torch.int32, device=dev)
        penalty = torch.full((batch,), repetition, device=dev)
        state = self.start(batch)
        for t in range(length):
            logits = self.decode(prompt[:, t].contiguous(), state)
        for i in range(n):
            _, best = nb.logits_process(logits, history, lengths, penalty, mask=mask)
            history[:, length + i] = best
            lengths += 1
            if i + 1 < n:
                logits = self.decode(best, state)
        return history[:, length:]


def teacher(vocab, k, seed, device):
    """For each token, k different next ones and their logits, descending."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    first = torch.randint(0, vocab, (vocab, 1), generator=g, device=device)
    ids = (first + 17 * torch.arange(k, device=device)) % vocab
    t = torch.randn((vocab, k), generator=g, device=device).abs() * 2
    return ids.to(torch.int32), t.sort(dim=1, descending=True).values


def train(model, steps, batch=8, length=128, k=16, lr=0.3, seed=1):
    dev = model.E.device
    t_ids, t_logits = teacher(model.vocab, k, seed, dev)
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    losses = []
    for _ in range(steps):
        ids = torch.randint(0, model.vocab, (batch, length), generator=g, device=dev,
                            dtype=torch.int32)
        ids[0, length // 2:] = -1  # a sequence that ends early
        flat = ids.reshape(-1).long()
        weight = (flat >= 0).float()
        weight /= weight.sum()
        at = flat.clamp(min=0)
        losses.append(model.step(ids, t_ids[at].contiguous(), t_logits[at].contiguous(), weight,
                                 lr))
    return torch.stack(losses).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=16)
    a = ap.parse_args()
    model = Model(vocab=1003)
    losses = train(model, a.steps)
    print("distillation loss: %.3f -> %.3f over %d steps" % (losses[0], losses[-1], a.steps))
    model.quantise()
    prompt = torch.arange(12, dtype=torch.int32, device=model.E.device).view(2, 6)
    print("tokens:", model.generate(prompt, a.tokens).tolist())


if __name__ == "__main__":
    main()
