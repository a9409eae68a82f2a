"""The operators of a layer and of its training step, as measured workloads.

Three operators: the norms before and after a block with its gate and residual
scale (forward and backward), linear attention with a decay for each head
(prompts, gradients, single tokens), and the AdamW step over many tensors at once
with states in 32 or 8 bits.  Each has a plain form in elementary torch
operations (32-bit arithmetic, one rounding at the end) and, with `own` set, the
call of the library's kernels.

    listed()            the named cases
    draw(rng)           one more case of the same ranges
    prepare(case, seed) the tensors a program has in hand before the call
    run(state)          one pass
    work(case)          the bytes and operations a pass cannot do without
    exact(case, seed)   the outputs from the definitions, in 64 bits
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_EPS = 1e-6            # of the norms
_CHUNK = 64            # tokens of a chunk in the plain form of the attention
_BLOCK = 256           # elements that share a scale in 8-bit optimizer states
_E4M3 = 448.0          # the largest value of the 8-bit type
_TINY = 2.0 ** -120    # scales below this are zero
_MOST_BYTES = 4.0e9    # a drawn case costs no more than the largest listed one
_MOST_FLOPS = 2.0e11


def listed():
    return [
        # between two layers of a decode step: 8 sequences, residual and the next layer's norm
        dict(name="norm_step_8x768", op="norm_fwd", rows=8, d=768, io="bf16", x_io="bf16",
             g_io="bf16", gate=False, post=False, scale=False),
        # a training batch (8 x 2048 tokens), an fp32 residual stream, everything on
        dict(name="norm_fwd_8x2048x768", op="norm_fwd", rows=16384, d=768, io="bf16", x_io="f32",
             g_io="bf16", gate=True, post=True, scale=True),
        # odd sizes in fp32
        dict(name="norm_fwd_1021x1003_f32", op="norm_fwd", rows=1021, d=1003, io="f32",
             x_io="f32", g_io="f32", gate=True, post=True, scale=True),
        # the training batch's gradient, the residual's gradient carried in fp32
        dict(name="norm_grad_8x2048x768", op="norm_bwd", rows=16384, d=768, io="bf16",
             x_io="bf16", g_io="f32", gate=True, post=True, scale=True),
        # the long-sequence workload's length and width: a pre-norm layer with a residual scale
        dict(name="norm_grad_65536x2048", op="norm_bwd", rows=65536, d=2048, io="bf16",
             x_io="f32", g_io="bf16", gate=False, post=False, scale=True),
        # a small model's update: 27 tensors, most of them tiny, where launches count
        dict(name="adamw_small_27", op="adamw", layers=2, d=96, inner=192, vocab=1003, bits=32,
             g_io="f32", copy=False),
        # 12 mixer layers and an embedding: bf16 gradients, the weights' bf16 copies with it
        dict(name="adamw_12x768_copy", op="adamw", layers=12, d=768, inner=1536, vocab=50000,
             bits=32, g_io="bf16", copy=True),
        # the same with 8-bit states, odd widths
        dict(name="adamw_12x1001_8bit", op="adamw", layers=12, d=1001, inner=2003, vocab=32003,
             bits=8, g_io="f32", copy=False),
        # one token of each of 8 sequences
        dict(name="linattn_step_8x12x128", op="lin_step", batch=8, L=1, H=12, Hk=12, dk=128,
             dv=128, io="bf16", ragged=False, state=True),
        # a ragged batch of short prompts in fp32, odd head sizes
        dict(name="linattn_fwd_3x333_f32", op="lin_fwd", batch=3, L=333, H=5, Hk=5, dk=40, dv=72,
             io="f32", ragged=True, state=False),
        # one long prompt
        dict(name="linattn_fwd_1x65536x16x128", op="lin_fwd", batch=1, L=65536, H=16, Hk=16,
             dk=128, dv=128, io="bf16", ragged=False, state=True),
        # a training batch's gradient
        dict(name="linattn_grad_8x2048x12x128", op="lin_bwd", batch=8, L=2048, H=12, Hk=12,
             dk=128, dv=128, io="bf16", ragged=False, state=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "adamw", "lin_fwd", "lin_bwd", "lin_step"])
    while True:
        if kind.startswith("norm"):
            io, x_io, g_io = rng.choice([("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                         ("bf16", "bf16", "f32"), ("bf16", "f32", "f32"),
                                         ("bf16", "f32", "bf16")])
            case = dict(op=kind, rows=_log(rng, 1, 65536), d=_log(rng, 64, 8192), io=io,
                        x_io=x_io, g_io=g_io, gate=rng.random() < 0.5, post=rng.random() < 0.5,
                        scale=rng.random() < 0.5)
        elif kind == "adamw":
            d = _log(rng, 64, 1024)
            case = dict(op=kind, layers=rng.randint(1, 12), d=d, inner=2 * d + rng.choice([0, 1]),
                        vocab=_log(rng, 1000, 50000), bits=rng.choice([8, 32]),
                        g_io=rng.choice(["f32", "bf16"]), copy=rng.random() < 0.5)
        else:
            Hk = rng.choice([1, 2, 3, 4, 6, 8, 12, 16])
            step = kind == "lin_step"
            L = 1 if step else _log(rng, 1, 8192 if kind == "lin_bwd" else 65536)
            case = dict(op=kind, batch=_log(rng, 1, 256 if step else 8), L=L,
                        H=Hk * rng.choice([1, 1, 1, 2, 4]), Hk=Hk, dk=8 * _log(rng, 2, 32),
                        dv=8 * _log(rng, 2, 32), io=rng.choice(["bf16", "bf16", "f32"]),
                        ragged=not step and rng.random() < 0.5,
                        state=step or rng.random() < 0.5)
        w = work(case)
        # (fp32 products run at a sixteenth of the bf16 rate)
        most = _MOST_FLOPS / (8 if case.get("io") == "f32" else 1)
        if w["bytes"] <= _MOST_BYTES / (4 if case["op"].startswith("lin") else 1) and \
                w["flops"] <= most:
            return case


# ------------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _shapes(case):
    """The parameters of mixer layers of a width, and of the embedding."""
    d, n = case["d"], case["inner"]
    layer = [(d, n), (d, n), (n, 4), (n, n), (n,), (n, n), (n,), (n, 16), (n, 16), (n,), (n, d),
             (d,), (d,)]
    return [(case["vocab"], d)] + layer * case["layers"]


def _offsets(case):
    """Where each tensor starts in one buffer that holds them all, in whole blocks; its end."""
    at, offsets = 0, []
    for shape in _shapes(case):
        offsets.append(at)
        at += -(-math.prod(shape) // _BLOCK) * _BLOCK
    return offsets, at


def _views(flat, case):
    return [flat[o:o + math.prod(s)].view(s) for s, o in zip(_shapes(case), _offsets(case)[0])]


def _scale_views(flat, case):
    return [flat[o // _BLOCK:o // _BLOCK + -(-math.prod(s) // _BLOCK)]
            for s, o in zip(_shapes(case), _offsets(case)[0])]


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).mul_(std).to(dtype)

    s = {"op": case["op"], "case": case}
    if case["op"].startswith("norm"):
        R, d = case["rows"], case["d"]
        io, x_io, g_io = _DT[case["io"]], _DT[case["x_io"]], _DT[case["g_io"]]
        # the residual stream has grown over the layers before it
        s["x"] = normal(R, d, std=2.0, dtype=x_io)
        s["y"] = normal(R, d, std=0.7, dtype=io)
        s["z"] = normal(R, d, dtype=io) if case["gate"] else None
        s["w_pre"] = 1.0 + normal(d, std=0.1)
        s["w_post"] = 1.0 + normal(d, std=0.1) if case["post"] else None
        s["scale"] = 0.5 + normal(d, std=0.1) if case["scale"] else None
        if case["op"] == "norm_bwd":
            s["dxn"] = normal(R, d, std=1e-2, dtype=g_io)
            s["dx"] = normal(R, d, std=1e-2, dtype=g_io)
        return s
    if case["op"] == "adamw":
        offsets, n = _offsets(case)
        inside = torch.zeros(n, dtype=torch.bool, device=dev)
        for o, shape in zip(offsets, _shapes(case)):
            inside[o:o + math.prod(shape)] = True
        # gradients of very different sizes, tensor by tensor
        size = torch.empty(n // _BLOCK, device=dev).normal_(generator=g).mul_(2.0).exp_()
        size = (size * 1e-3).repeat_interleave(_BLOCK) * inside
        s["p"] = normal(n, std=0.03) * inside
        s["g"] = (normal(n) * size).to(_DT[case["g_io"]])
        s["m"] = normal(n, std=0.3) * size
        s["v"] = (size * (0.3 + normal(n, std=0.3).abs_())).square_()
        s["step"], s["lr"] = 1000, 3e-4
        s["clip"] = torch.full((1,), 0.7, device=dev)  # the coefficient of a clipped global norm
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _encode(s["m"])
            s["v"], s["v_scale"] = _encode(s["v"].sqrt_())
        # the step writes a second set of buffers
        for key in ("p", "m", "v", "m_scale", "v_scale"):
            if key in s:
                s[key + "_next"] = torch.zeros_like(s[key])
        if case["copy"]:
            s["copy_next"] = torch.zeros(n, dtype=torch.bfloat16, device=dev)
        s["lists"] = {k: (_scale_views if "scale" in k else _views)(t, case)
                      for k, t in s.items() if isinstance(t, torch.Tensor) and k != "clip"}
        return s
    B, L, H, Hk = case["batch"], case["L"], case["H"], case["Hk"]
    dk, dv, dt = case["dk"], case["dv"], _DT[case["io"]]
    shape = (B,) if case["op"] == "lin_step" else (B, L)
    s["q"] = normal(*shape, H, dk, dtype=dt)
    s["k"] = normal(*shape, Hk, dk, std=dk ** -0.5, dtype=dt)
    s["v"] = normal(*shape, Hk, dv, dtype=dt)
    # decays from a memory of a few tokens to one of thousands
    s["log_decay"] = -torch.exp2(-1.0 - 10.0 * torch.rand((H,), generator=g, device=dev))
    s["qk_scale"] = dk ** -0.5
    s["state"] = normal(B, H, dk, dv) if case["state"] else None
    s["lengths"] = None
    if case["ragged"]:
        n = torch.randint(0, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[0] = L
        s["lengths"] = n
    if case["op"] == "lin_bwd":
        s["do"] = normal(B, L, H, dv, dtype=dt)
        s["dstate"] = normal(B, H, dk, dv) if case["state"] else None
    if case["op"] == "lin_step":
        s["state_next"] = torch.zeros_like(s["state"])
    return s


# ------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from selective_state_space_naju_amd import binding as nb
    op = s["op"]
    if op == "norm_fwd":
        x, xn = nb.res_norm_fwd(s["x"], s["y"], s["z"], scale=s["scale"], w_post=s["w_post"],
                                w_pre=s["w_pre"], eps=_EPS)
        return {"x": x, "xn": xn}
    if op == "norm_bwd":
        return nb.res_norm_bwd(s["dxn"], s["dx"], s["x"], s["y"], s["z"], scale=s["scale"],
                               w_post=s["w_post"], w_pre=s["w_pre"], eps=_EPS)
    if op == "adamw":
        t = s["lists"]
        nb.adamw_step(t["p"], t["g"], t["m"], t["v"], s["step"], s["lr"], weight_decay=0.1,
                      m_scale=t.get("m_scale"), v_scale=t.get("v_scale"), grad_scale=s["clip"],
                      copies=t.get("copy_next"),
                      out={k: t[k + "_next"] for k in ("p", "m", "v", "m_scale", "v_scale")
                           if k in t})
        return {k: v for k, v in s.items() if k.endswith("_next")}
    if op == "lin_fwd":
        o, state = nb.linattn_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["state"],
                                  s["lengths"], s["qk_scale"])
        return {"o": o, "state": state}
    if op == "lin_bwd":
        return nb.linattn_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["do"], s["state"],
                              s["dstate"], s["lengths"], s["qk_scale"])
    o = nb.linattn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["qk_scale"],
                        state_out=s["state_next"])
    return {"o": o, "state": s["state_next"]}


def _run_plain(s):
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "adamw": _adamw, "lin_fwd": _lin_fwd,
            "lin_bwd": _lin_bwd, "lin_step": _lin_step}[s["op"]](s)


def _inv_rms(x):
    return torch.rsqrt((x * x).mean(dim=1, keepdim=True) + _EPS)


def _norm_fwd(s):
    n = s["y"].float()
    if s["w_post"] is not None:
        n = n * _inv_rms(n) * s["w_post"]
    if s["z"] is not None:
        z = s["z"].float()
        n = n * z / (1.0 + torch.exp(-z))
    if s["scale"] is not None:
        n = n * s["scale"]
    x = s["x"].float() + n
    return {"x": x.to(s["x"].dtype), "xn": (x * _inv_rms(x) * s["w_pre"]).to(s["y"].dtype)}


def _norm_bwd(s):
    x, y, dxn = s["x"].float(), s["y"].float(), s["dxn"].float()
    r = _inv_rms(x)
    xh, e = x * r, dxn * s["w_pre"]
    dx = s["dx"].float() + r * (e - xh * (e * xh).mean(dim=1, keepdim=True))
    out = {"dx": dx.to(s["dx"].dtype), "dw_pre": (dxn * xh).sum(dim=0), "dz": None,
           "dw_post": None, "dscale": None}
    n = y
    if s["w_post"] is not None:
        ry = _inv_rms(y)
        yh = y * ry
        n = yh * s["w_post"]
    gate = 1.0
    if s["z"] is not None:
        z = s["z"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        gate = z * sig
    t = dx
    if s["scale"] is not None:
        out["dscale"] = (dx * n * gate).sum(dim=0)
        t = dx * s["scale"]
    if s["z"] is not None:
        out["dz"] = (t * n * sig * (1.0 + z * (1.0 - sig))).to(s["z"].dtype)
    f = t * gate
    if s["w_post"] is not None:
        out["dw_post"] = (f * yh).sum(dim=0)
        f = f * s["w_post"]
        f = ry * (f - yh * (f * yh).mean(dim=1, keepdim=True))
    out["dy"] = f.to(s["y"].dtype)
    return out


def _encode(x):
    """x as 8-bit floats and a scale for each block."""
    blocks = x.view(-1, _BLOCK)
    scale = blocks.abs().amax(dim=1) / _E4M3
    scale = torch.where(scale < _TINY, torch.zeros_like(scale), scale)
    unit = torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(1)
    codes = torch.where(scale.unsqueeze(1) > 0, blocks / unit, torch.zeros_like(blocks))
    return codes.clamp(-_E4M3, _E4M3).to(torch.float8_e4m3fn).view(-1), scale


def _decode(codes, scale):
    return (codes.float().view(-1, _BLOCK) * scale.unsqueeze(1)).view(-1)


def _adamw(s):
    b1, b2, eps, wd, lr, t = 0.9, 0.999, 1e-8, 0.1, s["lr"], s["step"]
    g = s["g"].float() * s["clip"]
    if "m_scale" in s:
        m, v = _decode(s["m"], s["m_scale"]), _decode(s["v"], s["v_scale"]).square()
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    mhat, vhat = m / (1.0 - b1 ** t), v / (1.0 - b2 ** t)
    p = s["p"] * (1.0 - lr * wd) - lr * mhat / (vhat.sqrt() + eps)
    out = {"p_next": p}
    if "m_scale" in s:
        out["m_next"], out["m_scale_next"] = _encode(m)
        out["v_next"], out["v_scale_next"] = _encode(v.sqrt())
    else:
        out["m_next"], out["v_next"] = m, v
    if "copy_next" in s:
        out["copy_next"] = p.to(torch.bfloat16)
    return out


def _heads(x, H):
    """[B, L, Hk, D] as fp32 [B, H, L, D], a shared head repeated for each of its readers."""
    x = x.float().transpose(1, 2)
    return x.repeat_interleave(H // x.shape[1], dim=1).contiguous()


def _walk(q, k, v, log_decay, state, late):
    """sum_{j <= i} decay^(i - j) (q_i . k_j) v_j + decay^(i + late) q_i . state, chunk by chunk;
    q, k, v fp32 [B, H, L, D].  Exponents are formed as sums, so nothing overflows."""
    B, H, L, dk = q.shape
    dv, C = v.shape[-1], _CHUNK
    n = -(-L // C)
    pad = n * C - L
    q, k, v = (torch.nn.functional.pad(t, (0, 0, 0, pad)).view(B * H, n, C, -1) for t in (q, k, v))
    a = log_decay.repeat(B).view(B * H, 1, 1)
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    gap = (i.unsqueeze(1) - i).unsqueeze(0)
    inner = torch.where(gap >= 0, torch.exp(a * gap.clamp(min=0)), torch.zeros_like(a))
    o = (q @ k.transpose(2, 3).contiguous() * inner.unsqueeze(1)) @ v
    # what each chunk adds to the state at its end, and the state that enters each chunk
    to_end = torch.exp(a * (C - 1 - i).view(1, C, 1)).unsqueeze(1)
    adds = k.transpose(2, 3).contiguous() @ (v * to_end)
    c = torch.arange(n, device=q.device, dtype=torch.float32)
    ago = (c.unsqueeze(1) - 1 - c).unsqueeze(0)
    carry = torch.where(ago >= 0, torch.exp(a * C * ago.clamp(min=0)), torch.zeros_like(a))
    enter = (carry @ adds.view(B * H, n, dk * dv)).view(B * H, n, dk, dv)
    # (a token i of a chunk lies i + 1 steps behind the chunk before it)
    o = o + (q * torch.exp(a * (i + 1).view(1, C, 1)).unsqueeze(1)) @ enter
    o = o.view(B, H, n * C, dv)[:, :, :L]
    if state is not None:
        t = torch.arange(L, device=q.device, dtype=torch.float32) + late
        lead = torch.exp(log_decay.view(1, H, 1, 1) * t.view(1, 1, L, 1))
        o = o + (q.view(B, H, n * C, dk)[:, :, :L] * lead) @ state
    return o


def _sum_to(k, v, log_decay, exponent, there):
    """sum over tokens of decay^exponent k v^T."""
    w = torch.exp(log_decay.view(1, -1, 1, 1) * exponent.view(exponent.shape[0], 1, -1, 1))
    w = torch.where(there.unsqueeze(1).unsqueeze(3), w, torch.zeros_like(w))
    return k.transpose(2, 3).contiguous() @ (v * w)


def _lengths(s, B, L, dev):
    n = s["lengths"]
    n = torch.full((B,), L, dtype=torch.int64, device=dev) if n is None else n.long()
    t = torch.arange(L, device=dev)
    return n, t, t < n.unsqueeze(1)


def _lin_fwd(s):
    q = s["q"]
    B, L, H, _ = q.shape
    n, t, there = _lengths(s, B, L, q.device)
    live = there.view(B, 1, L, 1)
    zero = torch.zeros((), device=q.device)
    qf, kf, vf = (torch.where(live, _heads(x, H), zero) for x in (q, s["k"], s["v"]))
    a = s["log_decay"]
    o = _walk(qf, kf, vf, a, s["state"], 1) * s["qk_scale"]
    last = (n.unsqueeze(1) - 1 - t).clamp(min=0).float()
    state = _sum_to(kf, vf, a, last, there)
    if s["state"] is not None:
        state = state + s["state"] * torch.exp(a * n.float().unsqueeze(1)).view(B, H, 1, 1)
    return {"o": o.transpose(1, 2).to(q.dtype).contiguous(), "state": state}


def _lin_bwd(s):
    q, k = s["q"], s["k"]
    B, L, H, dk = q.shape
    Hk, dv = k.shape[2], s["v"].shape[3]
    n, t, there = _lengths(s, B, L, q.device)
    live = there.view(B, 1, L, 1)
    zero = torch.zeros((), device=q.device)
    qf, kf, vf, gf = (torch.where(live, _heads(x, H), zero) for x in (q, k, s["v"], s["do"]))
    a, sc = s["log_decay"], s["qk_scale"]
    turn = lambda m: None if m is None else m.transpose(2, 3).contiguous()  # noqa: E731
    dq = _walk(gf, vf, kf, a, turn(s["state"]), 1) * sc
    # back in time: the tokens of each row from its last to its first
    back = (n.unsqueeze(1) - 1 - t) % max(1, L)
    flip = lambda x: x.gather(2, back.view(B, 1, L, 1).expand_as(x))  # noqa: E731
    qb, kb, vb, gb = (flip(x) for x in (qf, kf, vf, gf))
    end = s["dstate"] / sc if s["dstate"] is not None else None
    dk_ = torch.where(live, flip(_walk(vb, gb, qb, a, turn(end), 0)), zero) * sc
    dv_ = torch.where(live, flip(_walk(kb, qb, gb, a, end, 0)), zero) * sc
    dstate = _sum_to(qf, gf, a, (t + 1).float().unsqueeze(0).expand(B, L), there) * sc
    if s["dstate"] is not None:
        dstate = dstate + s["dstate"] * torch.exp(a * n.float().unsqueeze(1)).view(B, H, 1, 1)
    dk_ = dk_.view(B, Hk, H // Hk, L, dk).sum(dim=2)
    dv_ = dv_.view(B, Hk, H // Hk, L, dv).sum(dim=2)
    return {"dq": dq.transpose(1, 2).to(q.dtype).contiguous(),
            "dk": dk_.transpose(1, 2).to(q.dtype).contiguous(),
            "dv": dv_.transpose(1, 2).to(q.dtype).contiguous(), "dstate": dstate}


def _lin_step(s):
    q = s["q"]
    B, H, dk = q.shape
    group = H // s["k"].shape[1]
    k, v = (s[x].float().repeat_interleave(group, dim=1) for x in ("k", "v"))
    state = s["state"] * torch.exp(s["log_decay"]).view(1, H, 1, 1)
    state = state + k.unsqueeze(3) * v.unsqueeze(2)
    o = (q.float().unsqueeze(3) * state).sum(dim=2) * s["qk_scale"]
    return {"o": o.to(q.dtype), "state": state}


# --------------------------------------------------------------------- work, exact
def work(case):
    op = case["op"]
    if op.startswith("norm"):
        R, d = case["rows"], case["d"]
        e, ex, eg = (_SIZE[case[k]] for k in ("io", "x_io", "g_io"))
        vectors = 4 * d * (1 + case["post"] + case["scale"])
        if op == "norm_fwd":
            # x and y (and the gate) in, the residual and its norm out
            row = d * (2 * ex + e * (2 + case["gate"]))
            return {"bytes": R * row + vectors, "flops": R * d * 14}
        row = d * (3 * eg + ex + e * (2 + 2 * case["gate"]))
        return {"bytes": R * row + 2 * vectors, "flops": R * d * 40}
    if op == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        each = 8 + _SIZE[case["g_io"]] + (16 if case["bits"] == 32 else 4 + 16 / _BLOCK)
        return {"bytes": n * (each + 2 * case["copy"]), "flops": n * 16}
    B, L, H, Hk, dk, dv = (case[k] for k in ("batch", "L", "H", "Hk", "dk", "dv"))
    e = _SIZE[case["io"]]
    state = 4 * B * H * dk * dv
    fwd = e * B * L * (H * (dk + dv) + Hk * (dk + dv))
    pairs = (_CHUNK + 1) / 2 if L >= _CHUNK else (L + 1) / 2  # of a token inside its chunk
    flops = B * L * H * (2 * pairs * (dk + dv) + 4 * dk * dv)
    if op == "lin_step":
        return {"bytes": fwd + 2 * state, "flops": B * H * 5 * dk * dv}
    if op == "lin_fwd":
        return {"bytes": fwd + state * (2 if case["state"] else 1), "flops": flops}
    grad = e * B * L * (H * (2 * dk + dv) + Hk * 2 * (dk + dv))
    return {"bytes": grad + state * (3 if case["state"] else 1), "flops": 3 * flops}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        return _norm_exact(s, op)
    if op == "adamw":
        return _adamw_exact(case, s)
    if op == "lin_step":
        lam = s["log_decay"].double().exp()
        out, states = [], []
        group = case["H"] // case["Hk"]
        for h in range(case["H"]):
            k, v, q = s["k"][:, h // group].double(), s["v"][:, h // group].double(), \
                s["q"][:, h].double()
            st = torch.addcmul(s["state"][:, h].double() * lam[h], k[:, :, None], v[:, None, :])
            states.append(st)
            out.append(torch.matmul(q[:, None, :], st)[:, 0] * s["qk_scale"])
        return {"o": torch.stack(out, dim=1), "state": torch.stack(states, dim=1)}
    if op == "lin_fwd":
        with torch.no_grad():
            o, state = _lin_definition(s, s["q"].double(), s["k"].double(), s["v"].double(),
                                       None if s["state"] is None else s["state"].double())
        return {"o": o, "state": state}
    ins = [s[k].double().requires_grad_() for k in ("q", "k", "v")]
    B, _, H, dk = s["q"].shape
    st = (s["state"].double() if s["state"] is not None else
          torch.zeros(B, H, dk, s["v"].shape[3], dtype=torch.float64, device=s["q"].device))
    st.requires_grad_()
    o, end = _lin_definition(s, *ins, st)
    loss = (o * s["do"].double()).sum()
    if s["dstate"] is not None:
        loss = loss + (end * s["dstate"].double()).sum()
    dq, dk_, dv_, ds = torch.autograd.grad(loss, ins + [st])
    return {"dq": dq, "dk": dk_, "dv": dv_, "dstate": ds}


def _lin_definition(s, q, k, v, state):
    """The recurrence in 64 bits, 128 tokens at a time."""
    B, L, H, dk = q.shape
    group, dv, dev = H // k.shape[2], v.shape[3], q.device
    a = s["log_decay"].double()
    if state is None:
        state = torch.zeros(B, H, dk, dv, dtype=torch.float64, device=dev)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), L, device=dev)
    outs, C = [], 128
    for c in range(0, L, C):
        T = min(C, L - c)
        t = torch.arange(T, device=dev)
        on = (t + c < n[:, None]).double()[:, None, :, None]
        qc = q[:, c:c + T].permute(0, 2, 1, 3) * on
        kc = k[:, c:c + T].repeat_interleave(group, 2).permute(0, 2, 1, 3) * on
        vc = v[:, c:c + T].repeat_interleave(group, 2).permute(0, 2, 1, 3) * on
        gap = (t[:, None] - t[None, :]).double()
        decay = (a[:, None, None] * gap).exp().tril()
        scores = torch.matmul(qc, kc.permute(0, 1, 3, 2)) * decay
        lead = (a[:, None] * (t + 1.0)).exp()[None, :, :, None]
        outs.append((torch.matmul(scores, vc) + torch.matmul(qc, state) * lead) * s["qk_scale"])
        # tokens that there are from here to the chunk's end, for each row
        left = (n - c).clamp(0, T).double()
        late = (left[:, None] - 1 - t).clamp(min=0)
        fade = (a[None, :, None] * late[:, None, :]).exp()[..., None]
        state = state * (a[None, :] * left[:, None]).exp()[..., None, None] + \
            torch.matmul((kc * fade).permute(0, 1, 3, 2), vc)
    if not outs:
        return torch.zeros(B, 0, H, dv, dtype=torch.float64, device=dev), state
    return torch.cat(outs, dim=2).permute(0, 2, 1, 3), state


def _norm_exact(s, op):
    f = {k: (None if s[k] is None else s[k].double()) for k in ("x", "y", "z", "w_pre", "w_post",
                                                                "scale")}

    def after(x, y, z, w_post, scale):
        if w_post is not None:
            y = y / (y.square().mean(1, keepdim=True) + _EPS).sqrt() * w_post
        if z is not None:
            y = y * (z * torch.sigmoid(z))
        if scale is not None:
            y = y * scale
        return x + y

    def before(x, w):
        return x / (x.square().mean(1, keepdim=True) + _EPS).sqrt() * w
    if op == "norm_fwd":
        x = after(f["x"], f["y"], f["z"], f["w_post"], f["scale"])
        return {"x": x, "xn": before(x, f["w_pre"])}
    # gradients by differentiation, some rows at a time; the sums over rows added up
    names = [k for k in ("y", "z") if f[k] is not None]
    sums = [k for k in ("w_post", "scale") if f[k] is not None]
    rows, total, step = {k: [] for k in ["x"] + names}, {}, max(1, (1 << 25) // s["x"].shape[1])
    for r in range(0, s["x"].shape[0], step):
        part = slice(r, r + step)
        x = f["x"][part].detach().requires_grad_()
        w = f["w_pre"].detach().requires_grad_()
        xn = before(x, w)
        gx, gw = torch.autograd.grad(xn, (x, w), s["dxn"][part].double())
        gx = gx + s["dx"][part].double()
        leaf = {k: f[k][part].detach().requires_grad_() for k in names}
        leaf |= {k: f[k].detach().requires_grad_() for k in sums}
        out = after(torch.zeros_like(gx), leaf["y"], leaf.get("z"), leaf.get("w_post"),
                    leaf.get("scale"))
        got = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), gx)))
        got["w_pre"] = gw
        rows["x"].append(gx)
        for k in names:
            rows[k].append(got[k])
        for k in sums + ["w_pre"]:
            total[k] = total.get(k, 0) + got[k]
    out = {"d" + k: torch.cat(v) for k, v in rows.items()}
    return {"dz": None, "dw_post": None, "dscale": None} | out | \
        {"d" + k: v for k, v in total.items()}


def _adamw_exact(case, s):
    t, lr = s["step"], s["lr"]
    g = s["g"].double() * s["clip"].double()
    m, v = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m = m * s["m_scale"].double().repeat_interleave(_BLOCK)
        v = (v * s["v_scale"].double().repeat_interleave(_BLOCK)) ** 2
    m = m.lerp(g, 1.0 - 0.9)
    v = v.lerp(g ** 2, 1.0 - 0.999)
    ratio = (m / -math.expm1(t * math.log(0.9))) / \
        ((v / -math.expm1(t * math.log(0.999))).sqrt() + 1e-8)
    p = s["p"].double()
    p = p - lr * 0.1 * p - lr * ratio
    out = {"p_next": p}
    if case["bits"] == 8:
        for k, x in (("m", m), ("v", v.sqrt())):
            sc = x.view(-1, _BLOCK).abs().max(dim=1).values / _E4M3
            out[k + "_scale_next"] = sc
            out[k + "_next"] = (x.view(-1, _BLOCK) / sc[:, None]).nan_to_num(0.0).view(-1)
    else:
        out["m_next"], out["v_next"] = m, v
    if "copy_next" in s:
        out["copy_next"] = p
    return out
