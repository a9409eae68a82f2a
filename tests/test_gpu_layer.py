"""The operators around a token mixer together, as a layer's training step and a server use them:
norm -> linear attention -> norm with gate and residual, the gradients back through all three, the
AdamW step; prompts and then single tokens; the same inside captured graphs and on another stream."""
import os
import sys

import numpy as np
import pytest
import torch

from gpu_helpers import TOL, dev, host, rel_err
from oracle import layer as ol
from selective_state_space_naju_amd import binding as nb

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm device")


# ------------------------------------------------------------------ a layer's training step
NAMES = ("W_q", "W_k", "W_v", "W_z", "W_o", "scale", "w_post", "w_in", "w_out")


def make(d, H, Hk, dh, seed):
    rng = np.random.default_rng(seed)
    p = {"W_q": rng.standard_normal((d, H * dh)) * d ** -0.5,
         "W_k": rng.standard_normal((d, Hk * dh)) * d ** -0.5,
         "W_v": rng.standard_normal((d, Hk * dh)) * d ** -0.5,
         "W_z": rng.standard_normal((d, d)) * d ** -0.5,
         "W_o": rng.standard_normal((H * dh, d)) * (H * dh) ** -0.5}
    for k in ("scale", "w_post", "w_in", "w_out"):
        p[k] = 1 + 0.2 * rng.standard_normal(d)
    return {k: v.astype(np.float32) for k, v in p.items()}


def plain_layer(x, p, log_decay, state, lengths, H, Hk, dh):
    """The layer in torch's own operations (64 bits, on the CPU, differentiable)."""
    def rms(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    B, L, d = x.shape
    xn = rms(x) * p["w_in"]
    q = (xn @ p["W_q"]).view(B, L, H, dh)
    k = (xn @ p["W_k"]).view(B, L, Hk, dh).repeat_interleave(H // Hk, 2)
    v = (xn @ p["W_v"]).view(B, L, Hk, dh).repeat_interleave(H // Hk, 2)
    rows, last = [], []
    for b in range(B):
        S, o = state[b], []
        for t in range(L):
            if t < lengths[b]:
                S = log_decay.exp()[:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
                o.append(dh ** -0.5 * (S * q[b, t][:, :, None]).sum(1).reshape(-1))
            else:
                o.append(torch.zeros(H * dh, dtype=x.dtype))
        rows.append(torch.stack(o))
        last.append(S)
    y = torch.stack(rows) @ p["W_o"]
    z = xn @ p["W_z"]
    x1 = x + p["scale"] * rms(y) * p["w_post"] * torch.nn.functional.silu(z)
    return x1, rms(x1) * p["w_out"], torch.stack(last)


def gpu_layer(x, p, log_decay, state, lengths, H, Hk, dh):
    B, L, d = x.shape
    _, xn = nb.res_norm_fwd(x, w_pre=p["w_in"], eps=EPS)
    x2 = xn.view(-1, d)
    q, k, v = ((x2 @ p[w]).view(B, L, h, dh) for w, h in (("W_q", H), ("W_k", Hk), ("W_v", Hk)))
    o, last = nb.linattn_fwd(q, k, v, log_decay, state, lengths)
    y = (o.view(-1, H * dh) @ p["W_o"]).view(B, L, d)
    z = (x2 @ p["W_z"]).view(B, L, d)
    x1, out = nb.res_norm_fwd(x, y, z, scale=p["scale"], w_post=p["w_post"], w_pre=p["w_out"],
                              eps=EPS)
    return x1, out, last, (xn, q, k, v, o, y, z)


def gpu_layer_bwd(x, p, log_decay, state, lengths, x1, saved, dout, dx1, dlast):
    xn, q, k, v, o, y, z = saved
    d = x.shape[-1]
    n = nb.res_norm_bwd(dout, dx1, x1, y, z, scale=p["scale"], w_post=p["w_post"],
                        w_pre=p["w_out"], eps=EPS)
    g = {"scale": n["dscale"], "w_post": n["dw_post"], "w_out": n["dw_pre"]}
    dy, dz, x2 = n["dy"].view(-1, d), n["dz"].view(-1, d), xn.view(-1, d)
    do = (dy @ p["W_o"].t()).view(o.shape)
    g["W_o"] = o.view(dy.shape[0], -1).t() @ dy
    a = nb.linattn_bwd(q, k, v, log_decay, do, state, dlast, lengths)
    dxn = dz @ p["W_z"].t()
    g["W_z"] = x2.t() @ dz
    for w, t in (("W_q", a["dq"]), ("W_k", a["dk"]), ("W_v", a["dv"])):
        t = t.view(dy.shape[0], -1)
        dxn += t @ p[w].t()
        g[w] = x2.t() @ t
    n = nb.res_norm_bwd(dxn.view(x.shape), n["dx"], x, w_pre=p["w_in"], eps=EPS)
    g["w_in"] = n["dw_pre"]
    return {k: t.contiguous() for k, t in g.items()}, n["dx"], a["dstate"]


@pytest.mark.parametrize("B,L,d,H,Hk,dh", [(3, 37, 64, 4, 2, 16), (2, 70, 100, 3, 3, 24),
                                           (1, 1, 64, 2, 1, 8)])
def test_a_layers_training_steps(B, L, d, H, Hk, dh):
    """All in fp32: eight products or sums after one another, of at most 140 terms each, every
    term rounded to 2^-24: 8 * 140 * 2^-24 = 7e-5 of the largest value.  The update is held to the
    formula at the gradients it was given, within the 8 roundings of 2^-24 that it makes."""
    rng = np.random.default_rng(L)
    x = rng.standard_normal((B, L, d)).astype(np.float32)
    state = (0.3 * rng.standard_normal((B, H, dh, dh))).astype(np.float32)
    log_decay = -np.exp2(-1.0 - np.arange(H)).astype(np.float32)
    lengths = np.array([L, max(L - 20, 0), 0][:B], dtype=np.int32)
    w_out, w_x1 = (rng.standard_normal((B, L, d)).astype(np.float32) for _ in range(2))
    w_last = rng.standard_normal(state.shape).astype(np.float32)
    p = {k: torch.from_numpy(v).to(dev()) for k, v in make(d, H, Hk, dh, 1).items()}
    gx, gs, gl, glen, g_out, g_x1, g_last = (
        torch.from_numpy(t).to(dev()) for t in (x, state, log_decay, lengths, w_out, w_x1, w_last))
    m, v = ([torch.zeros_like(p[k]) for k in NAMES] for _ in range(2))
    for step in (1, 2, 3):
        print("step %d" % step, flush=True)
        rx, rs, rl = (torch.from_numpy(t).double() for t in (x, state, log_decay))
        rp = {k: t.cpu().double().requires_grad_() for k, t in p.items()}
        rx.requires_grad_()
        rs.requires_grad_()
        want = plain_layer(rx, rp, rl, rs, lengths, H, Hk, dh)
        loss = sum((a * torch.from_numpy(b).double()).sum()
                   for a, b in zip(want, (w_x1, w_out, w_last)))
        loss.backward()
        x1, out, last, saved = gpu_layer(gx, p, gl, gs, glen, H, Hk, dh)
        g, dx, dstate = gpu_layer_bwd(gx, p, gl, gs, glen, x1, saved, g_out, g_x1, g_last)
        for name, got, ref in (("x1", x1, want[0]), ("out", out, want[1]), ("last", last, want[2]),
                               ("dx", dx, rx.grad), ("dstate", dstate, rs.grad)) + tuple(
                                   ("d" + k, g[k], rp[k].grad) for k in NAMES):
            err = rel_err(host(got), ref.detach().numpy())
            assert err < TOL["f32"], (step, name, err)
        before = [(host(p[k]), host(g[k]), host(m[i]), host(v[i])) for i, k in enumerate(NAMES)]
        nb.adamw_step([p[k] for k in NAMES], [g[k] for k in NAMES], m, v, step, 0.01)
        for i, k in enumerate(NAMES):
            wp, wm, wv = ol.adamw(*before[i], step, 0.01)[:3]
            assert rel_err(host(p[k]), wp) < 2.0 ** -21, (step, k)
            assert rel_err(host(m[i]), wm) < 2.0 ** -21, (step, k)
            assert rel_err(host(v[i]), wv) < 2.0 ** -21, (step, k)


def test_a_layers_gradient_against_differences():
    """The 64-bit layer's differences along random directions, against the GPU's gradients: the
    difference of step 1e-5 is right to 1e-9 or so, the gradients to 7e-5 of their size (above),
    which a random direction does not add up to more than (sqrt of the number of elements)."""
    B, L, d, H, Hk, dh = 2, 21, 64, 4, 1, 16
    rng = np.random.default_rng(5)
    x = rng.standard_normal((B, L, d)).astype(np.float32)
    state = (0.3 * rng.standard_normal((B, H, dh, dh))).astype(np.float32)
    log_decay = -np.exp2(-1.0 - np.arange(H)).astype(np.float32)
    lengths = np.array([L, 9], dtype=np.int32)
    weight = rng.standard_normal((B, L, d)).astype(np.float32)
    raw = make(d, H, Hk, dh, 2)
    p = {k: torch.from_numpy(v).to(dev()) for k, v in raw.items()}
    gx, gs, gl, glen, g_out = (torch.from_numpy(t).to(dev())
                               for t in (x, state, log_decay, lengths, weight))
    x1, _, _, saved = gpu_layer(gx, p, gl, gs, glen, H, Hk, dh)
    g, dx, dstate = gpu_layer_bwd(gx, p, gl, gs, glen, x1, saved, g_out, None, None)

    def loss(x, state, p):
        out = plain_layer(x, p, torch.from_numpy(log_decay).double(), state, lengths, H, Hk, dh)[1]
        return float((out * torch.from_numpy(weight).double()).sum())
    base = {"x": torch.from_numpy(x).double(), "state": torch.from_numpy(state).double()}
    base.update({k: torch.from_numpy(v).double() for k, v in raw.items()})
    grads = dict(g, x=dx, state=dstate)
    for name in base:
        direction = torch.from_numpy(rng.standard_normal(tuple(base[name].shape)))
        ends = []
        for s in (1e-5, -1e-5):
            at = dict(base)
            at[name] = base[name] + s * direction
            ends.append(loss(at["x"], at["state"], {k: at[k] for k in raw}))
        got = (grads[name].cpu().double() * direction).sum().item()
        size = float((grads[name].cpu().double() ** 2).sum().sqrt())
        assert abs(got - (ends[0] - ends[1]) / 2e-5) < 1e-4 * size, name


# ------------------------------------------------------------------ prompts, then single tokens
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("L,steps", [(5, 3), (130, 6)])
def test_prompts_then_single_tokens(io, L, steps):
    """Ragged prompts (one empty) through the chunked kernel, then tokens one at a time, against
    the definition over each row's whole sequence: norms and attention in between rounded to the
    io type on both paths."""
    dt = torch.float32 if io == "f32" else torch.bfloat16
    B, H, Hk, dh = 4, 4, 2, 16
    d = H * dh
    rng = np.random.default_rng(L)
    lengths = np.array([L, L // 2, 0, 1], dtype=np.int32)
    log_decay = -np.exp2(-1.0 - np.arange(H)).astype(np.float32)
    seqs = torch.from_numpy(rng.standard_normal((B, L + steps, d)).astype(np.float32)).to(dev())
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(d)).astype(np.float32)).to(dev())
    gl, glen = torch.from_numpy(log_decay).to(dev()), torch.from_numpy(lengths).to(dev())

    def heads(xn):  # keys from one half of the channels, values from the other
        kv = xn.view(*xn.shape[:-1], 2, Hk, dh)
        return (xn.view(*xn.shape[:-1], H, dh), kv.select(-3, 0).contiguous(),
                kv.select(-3, 1).contiguous())
    _, xn = nb.res_norm_fwd(seqs, w_pre=w, eps=EPS, dtype=dt)
    prompt = xn[:, :L].contiguous()
    o, state = nb.linattn_fwd(*heads(prompt), gl, lengths=glen)
    rows = torch.arange(B, device=dev())
    singles = []
    for t in range(steps):
        x_t = seqs[rows, glen.long() + t].contiguous()
        _, xn_t = nb.res_norm_fwd(x_t, w_pre=w, eps=EPS, dtype=dt)
        y_t = nb.linattn_step(*heads(xn_t), gl, state)
        singles.append(nb.res_norm_fwd(x_t, y_t.view(B, d), w_post=w, eps=EPS)[0])
    for b in range(B):
        n = int(lengths[b])
        assert not o[b, n:].any()
        q, k, v = (host(t) for t in heads(xn[b:b + 1, :n + steps].contiguous()))
        want, _ = ol.linattn_fwd(q, k, v, log_decay.astype(np.float64), scale=dh ** -0.5)[:2]
        assert rel_err(host(o[b, :n]), want[0, :n]) < TOL[io]
        y = torch.from_numpy(want[0, n:].reshape(steps, d))
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.cpu().double()
        ref = seqs[b, n:n + steps].cpu().double() + y
        got = torch.stack([s[b] for s in singles])
        assert rel_err(host(got), ref.numpy()) < TOL[io], b


# ------------------------------------------------------------------ graphs and streams
class Trainer:
    """norm -> attention of the normed tokens with themselves -> norm -> gradients -> AdamW on the
    tokens and the weights; everything a call needs is its own."""

    def __init__(self, seed, bits=32):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.B, self.L, self.H, self.dh = 2, 193, 4, 16
        d = self.H * self.dh
        self.x = torch.randn(self.B, self.L, d, generator=g, device=dev())
        self.w = [torch.ones(d, device=dev()) for _ in range(3)]
        self.goal = torch.randn(self.B, self.L, d, generator=g, device=dev())
        self.log_decay = torch.log1p(-torch.exp2(-1.0 - torch.arange(self.H, device=dev())))
        self.params = [self.x] + self.w
        self.step = torch.zeros(1, dtype=torch.int32, device=dev())
        self.lr = torch.full((1,), 0.05, device=dev())
        st = torch.float32 if bits == 32 else torch.float8_e4m3fn
        self.m, self.v = ([torch.zeros(p.shape, device=dev()).to(st) for p in self.params]
                          for _ in range(2))
        self.scales = {}
        if bits == 8:
            self.scales = {k: [torch.zeros(-(-p.numel() // 256), device=dev())
                               for p in self.params] for k in ("m_scale", "v_scale")}

    def run(self):
        x, (w0, w1, w2) = self.x, self.w
        _, xn = nb.res_norm_fwd(x, w_pre=w0, eps=EPS)
        h = xn.view(self.B, self.L, self.H, self.dh)
        o, _ = nb.linattn_fwd(h, h, h, self.log_decay)
        y = o.view(x.shape)
        x1, out = nb.res_norm_fwd(x, y, xn, w_post=w1, w_pre=w2, eps=EPS)
        n = nb.res_norm_bwd(out - self.goal, None, x1, y, xn, w_post=w1, w_pre=w2, eps=EPS)
        a = nb.linattn_bwd(h, h, h, self.log_decay, n["dy"].view(h.shape))
        dxn = n["dz"] + (a["dq"] + a["dk"] + a["dv"]).view(x.shape)
        f = nb.res_norm_bwd(dxn, n["dx"], x, w_pre=w0, eps=EPS)
        self.step += 1
        nb.adamw_step(self.params, [f["dx"], f["dw_pre"], n["dw_post"], n["dw_pre"]], self.m,
                      self.v, self.step, self.lr, **self.scales)

    def values(self):
        return [t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
                for t in self.params + self.m + self.v + sum(self.scales.values(), [])]

    def same(self, other):
        return all(torch.equal(a, b) for a, b in zip(self.values(), other.values()))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_replay_as_eager_ones(bits):
    """Two captured training steps, replayed in turn with eager steps of a third trainer and
    synchronisations between: bit for bit what eager steps give."""
    captured = [Trainer(1, bits), Trainer(2, bits)]
    eager = [Trainer(1, bits), Trainer(2, bits)]
    other, alone = Trainer(3, bits), Trainer(3, bits)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in captured:
            t.run()
    torch.cuda.current_stream().wait_stream(side)
    for t in eager:
        t.run()
    graphs = []
    for t in captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            t.run()
        graphs.append(graph)
    for replay in range(4):
        print("replay %d" % replay, flush=True)
        for c, e, graph in zip(captured, eager, graphs):
            graph.replay()
            other.run()
            e.run()
            torch.cuda.synchronize()
            assert c.same(e), replay
    for _ in range(8):
        alone.run()
    assert other.same(alone)
    assert int(captured[0].step) == 5


def test_steps_on_two_streams_at_once():
    trainers, alone = [Trainer(7), Trainer(8)], [Trainer(7), Trainer(8)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for t, s in zip(trainers, streams):
            with torch.cuda.stream(s):
                t.run()
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    for t, a in zip(trainers, alone):
        for _ in range(5):
            a.run()
        assert t.same(a)


# ------------------------------------------------------------------ the example's model
@pytest.fixture(scope="module")
def model():
    import language_model
    m = language_model.Model(vocab=203, d_model=64, d_inner=128, heads=4)
    print("train", flush=True)
    m.losses = language_model.train(m, 4, batch=3, length=70)
    m.quantise()
    return m


def test_example_with_attention_layers_runs(model):
    assert np.isfinite(model.losses).all()
    prompt = torch.tensor([[1, 2, 3], [4, 5, 6]], dtype=torch.int32, device=dev())
    out = model.generate(prompt, 5)
    assert torch.equal(out, model.generate(prompt, 5))
    assert int(out.min()) >= 0 and int(out.max()) < 203


def test_example_copies_are_the_rounded_parameters(model):
    """What the update wrote for the kernels is what rounding its parameters gives."""
    import language_model
    assert torch.equal(model.E_bf16, model.E.bfloat16())
    for p, q in zip(model.layers, model.bf16):
        for k in p:
            want = p[k].bfloat16() if k in language_model.QUANTISED else p[k]
            assert torch.equal(q[k], want), k


def test_example_gradients_against_differences(model):
    """Along the gradient of the fp32 vectors (norm weights, residual scales), which reaches them
    through every layer behind: the mean loss over 200 tokens is rounded to 1e-3 or so of its own
    (some ten bf16 roundings of 2^-9 on the way to a logit, averaged over the tokens), so steps
    that change it by 0.2 and 0.4 give the slope to 1 %; the gradient takes as many roundings on
    the way back (2 %); the two steps' difference over 3 is the third-order term.  5 % in all."""
    import language_model
    t_ids, t_logits = language_model.teacher(203, 16, 1, dev())
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.randint(0, 203, (3, 70), generator=g, device=dev(), dtype=torch.int32)
    ids[0, 60:] = -1
    flat = ids.reshape(-1).long()
    weight = (flat >= 0).float()
    weight /= weight.sum()
    at = flat.clamp(min=0)
    args = (ids, t_ids[at].contiguous(), t_logits[at].contiguous(), weight)
    _, _, grads = model.gradients(*args)
    names = ("w_pre", "scale")
    size = sum(float(gr["d" + k].double().square().sum()) for gr in grads for k in names) ** 0.5
    kept = [{k: p[k].clone() for k in names} for p in model.bf16]

    def loss_at(s):
        for p, gr, old in zip(model.bf16, grads, kept):
            for k in names:
                p[k].copy_(old[k] + (s / size) * gr["d" + k])
        return float(model.gradients(*args)[0])
    slopes = []
    for change in (0.2, 0.4):
        s = change / (2 * size)
        slopes.append((loss_at(s) - loss_at(-s)) / (2 * s))
    loss_at(0.0)
    print("  slope %.4f, %.4f against %.4f" % (slopes[0], slopes[1], size), flush=True)
    assert abs(slopes[0] - size) < 0.05 * size + abs(slopes[1] - slopes[0]) / 3
