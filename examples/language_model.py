"""A small language model of Naju mixer layers: trained by distillation, served with 4-bit weights.

    python examples/language_model.py [--steps N] [--tokens N] [--heads N]

Training step (bf16 weights, fp32 gradients):
    embedding -> norm -> [mixer layer -> x + scale * out, norm] x layers -> logits with the
    embedding's transpose -> distillation from a teacher's top logits, and the reverse of it all;
    then AdamW over all parameters, which writes the weights' bf16 copies too.  With --heads a
    linear-attention layer follows each mixer layer.
    The embedding and the output layer share one table: its gradient is the output layer's
    product, with the looked-up rows' gradient added to it.
Serving (one token per call for every sequence): embedding of the last tokens, projections with
    4-bit weights around the block's decode step and the linear attention's, 4-bit output layer,
    penalties and a grammar mask on the logits, the best allowed token.

The teacher is a fixed table: for each token, the k most likely next ones and their logits.  The
training step's output layer and attention projections, and the decode step's convolution that the
gates are projected from are plain torch; everything else goes through the library.
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
ATTENTION = ("W_qkv", "W_o")
QUANTISED = ("W_u", "W_z", "W_a", "W_b", "W_B", "W_C", "W_out") + ATTENTION
GROUP = 32


def norm(x, w=None):
    """x over its root mean square, times w, and x itself."""
    if w is None:
        w = torch.ones(x.shape[-1], device=x.device)
    x = x.contiguous()
    return nb.res_norm_fwd(x, w_pre=w)[1], x


class Model:
    """Parameters as fp32 master copies; `bf16` holds what the kernels read: the matrices' copies,
    and the vectors themselves.  heads: of a linear-attention layer behind each mixer layer (0:
    none)."""

    def __init__(self, vocab, d_model=96, d_inner=192, d_state=16, layers=2, seed=0,
                 device="cuda", heads=0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=g, device=device) * std

        self.vocab, self.d_model, self.d_inner, self.d_state = vocab, d_model, d_inner, d_state
        self.heads = heads
        self.scale = math.sqrt(d_model)
        self.E = normal(vocab, d_model, std=d_model ** -0.5)
        s_in, s_h = d_model ** -0.5, (0.355 * d_inner) ** -0.5
        self.layers = []
        for _ in range(layers):
            self.layers.append(dict(
                W_u=normal(d_model, d_inner, std=s_in), W_z=normal(d_model, d_inner, std=s_in),
                conv_w=normal(d_inner, 4, std=0.5), W_a=normal(d_inner, d_inner, std=s_h),
                a_bias=torch.full((d_inner,), 5.0, device=device),
                W_b=normal(d_inner, d_inner, std=s_h),
                b_bias=torch.full((d_inner,), -2.0, device=device),
                W_B=normal(d_inner, d_state, std=s_h), W_C=normal(d_inner, d_state, std=s_h),
                D=normal(d_inner, std=1.0), W_out=normal(d_inner, d_model, std=d_inner ** -0.5)))
            if heads:
                self.layers.append(dict(W_qkv=normal(d_model, 3 * d_model, std=s_in),
                                        W_o=normal(d_model, d_model, std=s_in)))
        for p in self.layers:  # the norm before the layer, and the scale of what it adds
            p["w_pre"] = torch.ones(d_model, device=device)
            p["scale"] = torch.ones(d_model, device=device)
        self.last_norm = torch.ones(d_model, device=device)  # (fixed: the output layer follows)
        if heads:  # from a memory of one token to one of 2^heads
            self.log_decay = torch.log1p(-torch.exp2(-1.0 - torch.arange(heads, device=device)))
        self.refresh()
        self.steps = 0

    def refresh(self):
        self.E_bf16 = self.E.bfloat16()
        self.bf16 = [{k: (v.bfloat16() if k in QUANTISED else v) for k, v in p.items()}
                     for p in self.layers]

    def w_pre(self, i):
        """The norm's weight that follows layer i - 1: the next layer's, or the last one."""
        return self.bf16[i]["w_pre"] if i < len(self.bf16) else self.last_norm

    # ------------------------------------------------------------------- training
    def qkv(self, p, xn):
        B, L, _ = xn.shape
        heads = (xn.reshape(-1, self.d_model) @ p["W_qkv"]).view(B, L, 3, self.heads, -1)
        return heads[:, :, 0], heads[:, :, 1], heads[:, :, 2]

    def layer(self, p, xn, lengths):
        if "W_qkv" not in p:
            return nb.mixer_fwd(xn, *[p[k] for k in MIXER])
        o, _ = nb.linattn_fwd(*self.qkv(p, xn), self.log_decay, lengths=lengths)
        return (o.reshape(-1, self.d_model) @ p["W_o"]).view(xn.shape)

    def layer_bwd(self, p, xn, lengths, dy):
        """Gradients of a layer's parameters, and of its input."""
        if "W_qkv" not in p:
            return nb.mixer_bwd(xn, *[p[k] for k in MIXER], dy)
        q, k, v = self.qkv(p, xn)
        o, _ = nb.linattn_fwd(q, k, v, self.log_decay, lengths=lengths)
        dy, x2 = dy.reshape(-1, self.d_model), xn.reshape(-1, self.d_model)
        do = (dy @ p["W_o"].t().contiguous()).view(o.shape)
        g = nb.linattn_bwd(q, k, v, self.log_decay, do, lengths=lengths)
        dqkv = torch.stack((g["dq"], g["dk"], g["dv"]), 2).view(-1, 3 * self.d_model)
        return dict(dW_o=(o.reshape(-1, self.d_model).t().contiguous() @ dy).float(),
                    dW_qkv=(x2.t().contiguous() @ dqkv).float(),
                    dxn=(dqkv @ p["W_qkv"].t().contiguous()).float().view(xn.shape))

    def forward(self, ids):
        """The final hidden states [batch, length, d_model] and what the backward needs: each
        layer's input and output, the sums, the last norm."""
        lengths = (ids >= 0).sum(1, dtype=torch.int32) if self.heads else None
        x = nb.embed_fwd(ids, self.E_bf16, self.scale)
        x, xn = nb.res_norm_fwd(x, w_pre=self.w_pre(0))
        saved = [(x, None, None)]
        for i, p in enumerate(self.bf16):
            y = self.layer(p, xn, lengths)
            x, after = nb.res_norm_fwd(x, y, scale=p["scale"], w_pre=self.w_pre(i + 1))
            saved.append((x, xn, y))
            xn = after
        return x, (saved, xn, lengths)

    def gradients(self, ids, t_ids, t_logits, weight, temperature=1.0):
        """The mean loss (not synchronised), and the gradients: of the table, and each layer's."""
        _, (saved, xn, lengths) = self.forward(ids)
        y2 = xn.reshape(-1, self.d_model)
        logits = y2 @ self.E_bf16.t().contiguous()
        loss, dlogits = nb.distill_fwd_bwd(logits, t_ids, t_logits, weight, temperature)
        dE = (dlogits.t().contiguous() @ y2).float()
        dxn, dx = (dlogits @ self.E_bf16).float().view_as(xn), None
        grads = [None] * len(self.bf16)
        dw_pre = None
        for i in range(len(self.bf16) - 1, -1, -1):
            p, (x, xn, y) = self.bf16[i], saved[i + 1]
            n = nb.res_norm_bwd(dxn, dx, x, y, scale=p["scale"], w_pre=self.w_pre(i + 1))
            if i + 1 < len(grads):
                grads[i + 1]["dw_pre"] = n["dw_pre"]
            grads[i] = self.layer_bwd(p, xn, lengths, n["dy"])
            grads[i]["dscale"] = n["dscale"]
            dxn, dx = grads[i]["dxn"], n["dx"]
        n = nb.res_norm_bwd(dxn, dx, saved[0][0], w_pre=self.w_pre(0))
        grads[0]["dw_pre"] = n["dw_pre"]
        # the looked-up rows' gradient joins the output layer's
        nb.embed_bwd(ids, n["dx"].bfloat16(), self.vocab, self.scale, dW=dE)
        return (loss * weight).sum(), dE, grads

    def step(self, ids, t_ids, t_logits, weight, lr, temperature=1.0):
        """One training step; returns the mean loss (a tensor, not synchronised)."""
        loss, dE, grads = self.gradients(ids, t_ids, t_logits, weight, temperature)
        matrices, vectors = [(self.E, dE, self.E_bf16)], []
        for p, q, g in zip(self.layers, self.bf16, grads):
            for k in p:
                if k in QUANTISED:
                    matrices.append((p[k], g["d" + k], q[k]))
                else:
                    vectors.append((p[k], g["d" + k]))
        self.steps += 1
        if self.steps == 1:
            self.moments = [[[torch.zeros_like(t[0]) for t in group] for _ in range(2)]
                            for group in (matrices, vectors)]
        p, g, copies = map(list, zip(*matrices))
        nb.adamw_step(p, g, *self.moments[0], self.steps, lr, copies=copies)
        p, g = map(list, zip(*vectors))
        nb.adamw_step(p, g, *self.moments[1], self.steps, lr, weight_decay=0.0)
        return loss

    # -------------------------------------------------------------------- serving
    def quantise(self):
        """4-bit weights of every projection, and of the output layer ([d_model, vocab])."""
        self.w4 = [{k: nb.w4_quantize(p[k], GROUP)[:2] for k in QUANTISED if k in p}
                   for p in self.bf16]
        self.w4_head = nb.w4_quantize(self.E_bf16.t().contiguous(), GROUP)[:2]

    def start(self, batch):
        """The state of `batch` sequences: per mixer layer the scan state and the conv window, per
        attention layer its heads' states."""
        dev = self.E.device
        d = self.d_model // self.heads if self.heads else 0
        return [torch.zeros(batch, self.heads, d, d, device=dev) if "W_qkv" in p else
                (torch.zeros(batch, self.d_inner, self.d_state, device=dev),
                 torch.zeros(batch, 3, self.d_inner, dtype=torch.bfloat16, device=dev))
                for p in self.layers]

    def layer_step(self, p, w, xn, state):
        def lin(v, k, bias=None):
            return nb.w4_linear(v, *w[k], GROUP, None, bias)
        if "W_qkv" in p:
            q, k, v = lin(xn, "W_qkv").view(len(xn), 3, self.heads, -1).transpose(0, 1).contiguous()
            o = nb.linattn_step(q, k, v, self.log_decay, state)
            return lin(o.view(len(xn), -1), "W_o")
        scan, window = state
        u, z = lin(xn, "W_u"), lin(xn, "W_z")
        taps = torch.cat((window, u.unsqueeze(1)), dim=1).float()
        h = torch.nn.functional.silu((taps * p["conv_w"].t()).sum(1)).bfloat16()
        a, b = lin(h, "W_a", p["a_bias"]), lin(h, "W_b", p["b_bias"])
        y = nb.block_step(u, z, p["conv_w"], window, a, b, lin(h, "W_B"), lin(h, "W_C"),
                          p["D"], scan)
        return lin(y, "W_out")

    def decode(self, tokens, state):
        """Logits [batch, vocab] after the given tokens [batch] (int32); the state moves on."""
        x = nb.embed_fwd(tokens, self.E_bf16, self.scale)
        x, xn = nb.res_norm_fwd(x, w_pre=self.w_pre(0))
        for i, (p, w, s) in enumerate(zip(self.bf16, self.w4, state)):
            y = self.layer_step(p, w, xn, s)
            x, xn = nb.res_norm_fwd(x, y, scale=p["scale"], w_pre=self.w_pre(i + 1))
        return nb.w4_linear(xn, *self.w4_head, GROUP)

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


def train(model, steps, batch=8, length=128, k=16, lr=0.01, seed=1):
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
    ap.add_argument("--heads", type=int, default=4)
    a = ap.parse_args()
    model = Model(vocab=1003, heads=a.heads)
    losses = train(model, a.steps)
    print("distillation loss: %.3f -> %.3f over %d steps" % (losses[0], losses[-1], a.steps))
    model.quantise()
    prompt = torch.arange(12, dtype=torch.int32, device=model.E.device).view(2, 6)
    print("tokens:", model.generate(prompt, a.tokens).tolist())


if __name__ == "__main__":
    main()
