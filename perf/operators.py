"""The operators around the mixer layer of a language model, as measured workloads.

Four operators: the token embedding with its gradient, distillation from a
teacher's top logits with its gradient, the processing of logits before a token
is chosen (penalties, biases, grammar masks), and the linear layer with 4-bit
weights that serving uses.  Each has a plain form in elementary torch operations
(32-bit arithmetic, one rounding at the end) and, with `own` set, the call of
the library's kernels.

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

# scale of the embedding rows: sqrt(d_model) brings rows of std 1/sqrt(d_model) to unit size
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}
_MOST_BYTES = 2.0e9  # a drawn case's traffic stays below the largest listed one's


def listed():
    return [
        # the lookup at the head of a decode step: one token of each of 8 sequences
        dict(name="embed_step_8x768", op="embed_fwd", tokens=8, vocab=32000, d=768, io="bf16"),
        # the gradient of a training batch of the mixer workload (8 x 2048 tokens)
        dict(name="embed_grad_8x2048x768", op="embed_bwd", tokens=16384, vocab=50000, d=768,
             io="bf16"),
        # the long-sequence workload's length and width, fp32, a vocabulary of an odd size
        dict(name="embed_grad_65536x2048_f32", op="embed_bwd", tokens=65536, vocab=100003,
             d=2048, io="f32"),
        # an evaluation batch: the loss alone, odd sizes, fp32 logits
        dict(name="distill_loss_129x10007_f32", op="distill_fwd", rows=129, vocab=10007, k=32,
             pad=0, tau=2.0, io="f32"),
        # a training batch: loss and gradient of 8 x 2048 tokens in one call
        dict(name="distill_step_16384x32000", op="distill_fwd_bwd", rows=16384, vocab=32000,
             k=64, pad=0, tau=1.0, io="bf16"),
        # the gradient alone, from the forward's statistics; a large odd vocabulary whose rows
        # lie in a padded matrix
        dict(name="distill_grad_2048x131071", op="distill_bwd", rows=2048, vocab=131071, k=128,
             pad=1, tau=2.0, io="bf16"),
        # one sequence being written: a short history, nothing else
        dict(name="logits_1x32000", op="logits", rows=1, vocab=32000, history=256, biases=0,
             grammar=False, io="bf16"),
        # a small batch with every constraint, odd sizes, fp32
        dict(name="logits_8x50001_f32", op="logits", rows=8, vocab=50001, history=2047,
             biases=16, grammar=True, io="f32"),
        # a full serving batch: long ragged histories, long bias lists, a grammar for each row
        dict(name="logits_256x131072", op="logits", rows=256, vocab=131072, history=4096,
             biases=300, grammar=True, io="bf16"),
        # the mixer's input projection for one token
        dict(name="w4_1x768x1536", op="w4", rows=1, d_in=768, d_out=1536, group=64, zeros=False,
             io="bf16"),
        # odd sizes, small groups with zero points, a few sequences
        dict(name="w4_5x4100x7001", op="w4", rows=5, d_in=4100, d_out=7001, group=32,
             zeros=True, io="bf16"),
        # the output layer of a large vocabulary for a batch of 32
        dict(name="w4_32x4096x131072", op="w4", rows=32, d_in=4096, d_out=131072, group=128,
             zeros=False, io="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "distill_fwd", "distill_bwd", "distill_fwd_bwd",
                     "logits", "w4"])
    io = rng.choice(["bf16", "f32"])
    while True:
        if op.startswith("embed"):
            case = dict(op=op, tokens=_log(rng, 1, 65536), vocab=_log(rng, 1000, 131072),
                        d=_log(rng, 96, 4096), io=io)
        elif op.startswith("distill"):
            case = dict(op=op, rows=_log(rng, 1, 16384), vocab=_log(rng, 1000, 131072),
                        k=_log(rng, 1, 256), pad=rng.choice([0, 0, 1, 8, 57]),
                        tau=rng.choice([1.0, 1.5, 2.0, 4.0]), io=io)
        elif op == "logits":
            case = dict(op=op, rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 131072),
                        history=rng.choice([0, _log(rng, 1, 16384), _log(rng, 1, 16384)]),
                        biases=rng.choice([0, _log(rng, 1, 300)]),
                        grammar=rng.choice([True, False]), io=io)
        else:
            case = dict(op=op, rows=_log(rng, 1, 64), d_in=2 * _log(rng, 48, 4096),
                        d_out=_log(rng, 16, 131072), group=rng.choice([32, 64, 128]),
                        zeros=rng.choice([True, False]), io="bf16")
        w = work(case)
        # (the plain form of a 4-bit product is bound by its operations on unpacked weights)
        if w["bytes"] <= _MOST_BYTES and w["flops"] <= 3.4e10:
            return case


# ------------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _tokens(shape, vocab, g, dev):
    """Token ids of running text: log-uniform ranks (the r-th most frequent token has a share
    of about 1/r), spread over the vocabulary by a fixed stride coprime to it."""
    u = torch.rand(shape, generator=g, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1.0)).long() - 1).clamp_(0, vocab - 1)
    stride = 7919
    while math.gcd(stride, vocab) != 1:
        stride += 2
    return (rank * stride % vocab).to(torch.int32)


def prepare(case, seed):
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[case["io"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev).mul_(std).to(dtype)

    op = case["op"]
    s = {"op": op, "case": case}
    if op.startswith("embed"):
        s["scale"] = math.sqrt(case["d"])
        s["ids"] = _tokens((case["tokens"],), case["vocab"], g, dev)
        # some positions hold no token (padding)
        if case["tokens"] > 64:
            pad = torch.rand((case["tokens"],), generator=g, device=dev) < 0.02
            s["ids"] = torch.where(pad, torch.full_like(s["ids"], -1), s["ids"])
        if op == "embed_fwd":
            s["W"] = normal(case["vocab"], case["d"], std=case["d"] ** -0.5, dtype=dt)
        else:
            s["vocab"] = case["vocab"]
            s["dout"] = normal(case["tokens"], case["d"], std=1e-3, dtype=dt)
    elif op.startswith("distill"):
        R, V, k = case["rows"], case["vocab"], case["k"]
        s["tau"] = case["tau"]
        s["logits"] = normal(R, V + case["pad"], std=2.5, dtype=dt)[:, :V]
        # the teacher's top logits: distinct tokens, descending values
        first = torch.randint(0, V, (R, 1), generator=g, device=dev)
        step = 1 + torch.randint(0, max(1, V // k - 1), (R, 1), generator=g, device=dev)
        s["t_ids"] = ((first + step * torch.arange(k, device=dev)) % V).to(torch.int32)
        t = 4.0 + 3.0 * torch.randn((R, k), generator=g, device=dev).abs()
        t = t.sort(dim=1, descending=True).values
        # lists that end early are filled up with (-1, -inf); a few rows have no list
        n = torch.randint(1, k + 1, (R, 1), generator=g, device=dev)
        u = torch.rand((R, 1), generator=g, device=dev)
        n = torch.where(u < 0.8, torch.full_like(n, k), n)
        n = torch.where(u > 0.99, torch.zeros_like(n), n)
        gone = torch.arange(k, device=dev) >= n
        s["t_logits"] = torch.where(gone, torch.full_like(t, -math.inf), t)
        s["t_ids"] = torch.where(gone, torch.full_like(s["t_ids"], -1), s["t_ids"])
        if op != "distill_fwd":
            w = (torch.rand((R,), generator=g, device=dev) < 0.95).float()  # padding has weight 0
            s["g"] = w / max(1, R)
        if op == "distill_bwd":
            s["lse"] = torch.logsumexp(s["logits"].float() / s["tau"], dim=1)
    elif op == "logits":
        B, V, H = case["rows"], case["vocab"], case["history"]
        s["logits"] = normal(B, V, std=2.5, dtype=dt)
        for key in ("history", "lengths", "repetition", "presence", "frequency", "bias_ids",
                    "bias", "mask"):
            s[key] = None
        if H > 0:
            s["history"] = _tokens((B, H), V, g, dev)
            n = torch.randint(0, H + 1, (B,), generator=g, device=dev, dtype=torch.int32)
            n[0] = H
            s["lengths"] = n
            one = torch.rand((B,), generator=g, device=dev)
            s["repetition"] = 1.0 + 0.5 * one
            s["presence"] = 0.5 * torch.rand((B,), generator=g, device=dev)
            s["frequency"] = 0.2 * torch.rand((B,), generator=g, device=dev)
        if case["biases"] > 0:
            nb = case["biases"]
            first = torch.randint(0, V, (B, 1), generator=g, device=dev)
            step = 1 + torch.randint(0, max(1, V // nb - 1), (B, 1), generator=g, device=dev)
            s["bias_ids"] = ((first + step * torch.arange(nb, device=dev)) % V).to(torch.int32)
            s["bias"] = normal(B, nb, std=5.0)
            # a tenth of the list forbids its token
            ban = torch.rand((B, nb), generator=g, device=dev) < 0.1
            s["bias"] = torch.where(ban, torch.full_like(s["bias"], -math.inf), s["bias"])
        if case["grammar"]:
            words = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g,
                                  device=dev)
            # some rows are tightly constrained, most words of theirs allow nothing
            tight = torch.rand((B, 1), generator=g, device=dev) < 0.5
            few = torch.rand(words.shape, generator=g, device=dev) < 0.05
            words = torch.where(tight & ~few, torch.zeros_like(words), words)
            s["mask"] = words.to(torch.int32)
    else:
        R, K, N, G = case["rows"], case["d_in"], case["d_out"], case["group"]
        ng = (K + G - 1) // G
        s["group"] = G
        s["x"] = normal(R, K, dtype=torch.bfloat16)
        s["qweight"] = torch.randint(0, 256, (N, K // 2), generator=g, device=dev,
                                     dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((N, ng), generator=g, device=dev))
                       * (0.22 * K ** -0.5)).to(torch.bfloat16)
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = torch.randint(5, 11, (N, ng), generator=g, device=dev,
                                       dtype=torch.uint8)
        s["bias"] = normal(N, std=0.5)
    return s


# ------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from selective_state_space_naju_amd import binding as nb
    op = s["op"]
    if op == "embed_fwd":
        return {"out": nb.embed_fwd(s["ids"], s["W"], s["scale"])}
    if op == "embed_bwd":
        return {"dW": nb.embed_bwd(s["ids"], s["dout"], s["vocab"], s["scale"])}
    if op == "distill_fwd":
        loss, lse = nb.distill_fwd(s["logits"], s["t_ids"], s["t_logits"], s["tau"])
        return {"loss": loss, "lse": lse}
    if op == "distill_bwd":
        return {"dlogits": nb.distill_bwd(s["logits"], s["t_ids"], s["t_logits"], s["lse"],
                                          s["g"], s["tau"])}
    if op == "distill_fwd_bwd":
        loss, dlogits = nb.distill_fwd_bwd(s["logits"], s["t_ids"], s["t_logits"], s["g"],
                                           s["tau"])
        return {"loss": loss, "dlogits": dlogits}
    if op == "logits":
        out, best = nb.logits_process(s["logits"], s["history"], s["lengths"],
                                      s["repetition"], s["presence"], s["frequency"],
                                      s["bias_ids"], s["bias"], s["mask"])
        return {"out": out, "best": best}
    return {"y": nb.w4_linear(s["x"], s["qweight"], s["scales"], s["group"], s["zeros"],
                              s["bias"])}


def _run_plain(s):
    op = s["op"]
    if op == "embed_fwd":
        ids, W = s["ids"].long(), s["W"]
        there = ((ids >= 0) & (ids < W.shape[0])).unsqueeze(1)
        rows = W[ids.clamp(0, W.shape[0] - 1)].float() * s["scale"]
        return {"out": (rows * there).to(W.dtype)}
    if op == "embed_bwd":
        ids, V = s["ids"].long(), s["vocab"]
        there = ((ids >= 0) & (ids < V)).unsqueeze(1)
        rows = s["dout"].float() * there
        dW = torch.zeros((V, rows.shape[1]), dtype=torch.float32, device=rows.device)
        return {"dW": dW.index_add_(0, ids.clamp(0, V - 1), rows) * s["scale"]}
    if op.startswith("distill"):
        return _distill_plain(s)
    if op == "logits":
        return _logits_plain(s)
    q = s["qweight"]
    N, K = q.shape[0], 2 * q.shape[1]
    codes = torch.stack((q & 15, q >> 4), dim=2).reshape(N, K).float()
    group = torch.arange(K, device=q.device) // s["group"]
    zero = s["zeros"].float()[:, group] if s["zeros"] is not None else 8.0
    w = (codes - zero) * s["scales"].float()[:, group]
    return {"y": (s["x"].float() @ w.T + s["bias"]).to(torch.bfloat16)}


def _distill_plain(s):
    logits, tau = s["logits"], s["tau"]
    V = logits.shape[1]
    x = logits.float() / tau
    if s["op"] == "distill_bwd":
        lse = s["lse"].unsqueeze(1)
    else:
        top = x.amax(dim=1, keepdim=True)
        lse = top + (x - top).exp().sum(dim=1, keepdim=True).log()
    ids = s["t_ids"].long()
    there = (ids >= 0) & (ids < V) & (s["t_logits"] != -math.inf)
    ids = ids.clamp(0, V - 1)
    some = there.any(dim=1, keepdim=True)
    t = torch.where(there, s["t_logits"] / tau, torch.full_like(s["t_logits"], -math.inf))
    t = t - torch.where(some, t.amax(dim=1, keepdim=True), torch.zeros_like(t[:, :1]))
    total = t.exp().sum(dim=1, keepdim=True)
    p = torch.where(some, t.exp() / total, torch.zeros_like(t))
    out = {}
    if s["op"] != "distill_bwd":
        gap = t - total.log() - (x.gather(1, ids) - lse)
        kl = torch.where(p > 0, p * gap, torch.zeros_like(p)).sum(dim=1)
        out["loss"] = tau * tau * kl
    if s["op"] == "distill_fwd":
        out["lse"] = lse.squeeze(1)
        return out
    diff = (x - lse).exp() * some
    diff.scatter_add_(1, ids, -p)
    out["dlogits"] = (diff * (tau * s["g"]).unsqueeze(1)).to(logits.dtype)
    return out


def _logits_plain(s):
    x = s["logits"].float()
    B, V = x.shape
    if s["history"] is not None:
        hist = s["history"].long()
        there = (torch.arange(hist.shape[1], device=x.device) < s["lengths"].unsqueeze(1))
        there = there & (hist >= 0) & (hist < V)
        count = torch.zeros_like(x).scatter_add_(1, hist.clamp(0, V - 1), there.float())
        seen = count > 0
        r = s["repetition"].unsqueeze(1)
        x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"].unsqueeze(1) * count
        x = x - s["presence"].unsqueeze(1) * seen
    if s["bias"] is not None:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        v = torch.arange(V, device=x.device)
        allowed = (s["mask"][:, v // 32] >> (v % 32)) & 1
        x = torch.where(allowed != 0, x, torch.full_like(x, -math.inf))
    top = x.amax(dim=1, keepdim=True)
    where = torch.where(x == top, torch.arange(V, device=x.device), V).amin(dim=1)
    best = torch.where(top.squeeze(1) > -math.inf, where, torch.full_like(where, -1))
    return {"out": x, "best": best.to(torch.int32)}


# --------------------------------------------------------------------- work, exact
def _distinct(tokens, vocab):
    """Expected number of different tokens among `tokens` log-uniform ranks."""
    r = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log1p(1.0 / r) / math.log(vocab + 1.0)
    return int(round(float((1.0 - torch.exp(tokens * torch.log1p(-p))).sum())))


def work(case):
    op, e = case["op"], _SIZE[case["io"]]
    if op == "embed_fwd":
        T, d = case["tokens"], case["d"]
        return {"bytes": 4 * T + e * d * (T + _distinct(T, case["vocab"])), "flops": T * d}
    if op == "embed_bwd":
        T, d = case["tokens"], case["d"]
        return {"bytes": 4 * T + e * d * T + 4 * d * case["vocab"], "flops": 2 * T * d}
    if op.startswith("distill"):
        R, V, k = case["rows"], case["vocab"], case["k"]
        once = e * R * V
        small = 8 * R * k + 8 * R
        # a subtraction, a scaling, an exponential and a sum for each logit; the gradient's
        # difference and product
        n = {"distill_fwd": (1, 4), "distill_bwd": (2, 4), "distill_fwd_bwd": (2, 6)}[op]
        return {"bytes": n[0] * once + small, "flops": n[1] * R * V}
    if op == "logits":
        B, V = case["rows"], case["vocab"]
        # histories are half full on average
        b = B * V * (e + 4) + 4 * B + 2 * B * case["history"] + 8 * B * case["biases"]
        if case["grammar"]:
            b += 4 * B * ((V + 31) // 32)
        return {"bytes": b, "flops": 4 * B * V}
    R, K, N, G = case["rows"], case["d_in"], case["d_out"], case["group"]
    ng = (K + G - 1) // G
    b = N * K // 2 + N * ng * (3 if case["zeros"] else 2) + 2 * R * K + 2 * R * N + 4 * N
    return {"bytes": b, "flops": 2 * R * K * N}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed_fwd":
        out = torch.zeros((case["tokens"], case["d"]), dtype=torch.float64, device=s["W"].device)
        use = s["ids"] >= 0
        out[use] = s["W"].index_select(0, s["ids"][use].long()).double() * s["scale"]
        return {"out": out}
    if op == "embed_bwd":
        use = s["ids"] >= 0
        dW = torch.zeros((case["vocab"], case["d"]), dtype=torch.float64,
                         device=s["dout"].device)
        dW.index_put_((s["ids"][use].long(),), s["dout"][use].double() * s["scale"],
                      accumulate=True)
        return {"dW": dW}
    if op.startswith("distill"):
        return _distill_exact(case, s)
    if op == "logits":
        return _logits_exact(case, s)
    K, N, G = case["d_in"], case["d_out"], case["group"]
    x, y = s["x"].double(), []
    for n in range(0, N, 16384):
        q = s["qweight"][n:n + 16384]
        w = torch.empty((q.shape[0], K), dtype=torch.float64, device=q.device)
        w[:, 0::2] = torch.bitwise_and(q, 0x0F).double()
        w[:, 1::2] = torch.div(q, 16, rounding_mode="floor").double()
        zero = s["zeros"][n:n + 16384].double() if s["zeros"] is not None else None
        for j in range((K + G - 1) // G):
            cols = slice(j * G, min(K, (j + 1) * G))
            w[:, cols] -= 8.0 if zero is None else zero[:, j:j + 1]
            w[:, cols] *= s["scales"][n:n + 16384, j:j + 1].double()
        y.append(torch.matmul(x, w.t().contiguous()))
    return {"y": torch.cat(y, dim=1) + s["bias"].double()}


def _distill_exact(case, s):
    V, tau, op = case["vocab"], case["tau"], case["op"]
    parts = {"loss": [], "lse": [], "dlogits": []}
    step = max(1, (1 << 26) // V)
    for r in range(0, case["rows"], step):
        logq = s["logits"][r:r + step].double() / tau
        lse = torch.logsumexp(logq, dim=1, keepdim=True)
        if op == "distill_bwd":  # the statistics are an input there
            lse = s["lse"][r:r + step].double().unsqueeze(1)
        logq = logq - lse
        ids = s["t_ids"][r:r + step].long()
        t = (s["t_logits"][r:r + step].double() / tau).masked_fill(ids < 0, -math.inf)
        p = torch.softmax(t, dim=1).nan_to_num(0.0)  # a row without entries is 0/0
        logp = torch.log_softmax(t, dim=1)
        term = torch.xlogy(p, p) if op == "distill_fwd_bwd" else (p * logp).nan_to_num(0.0)
        kl = (term - p * logq.gather(1, ids.clamp(min=0))).sum(dim=1)
        parts["loss"].append(tau ** 2 * kl)
        parts["lse"].append(lse.squeeze(1))
        if op != "distill_fwd":
            ds = logq.exp() * (ids >= 0).any(dim=1, keepdim=True)
            ds = ds.scatter_add(1, ids.clamp(min=0), -p)
            parts["dlogits"].append(ds * tau * s["g"][r:r + step].double().unsqueeze(1))
    names = {"distill_fwd": ("loss", "lse"), "distill_bwd": ("dlogits",),
             "distill_fwd_bwd": ("loss", "dlogits")}[op]
    return {n: torch.cat(parts[n], dim=0) for n in names}


def _logits_exact(case, s):
    out = s["logits"].double()
    V = case["vocab"]
    for b in range(case["rows"]):
        row = out[b]
        if s["history"] is not None:
            seen = s["history"][b, :int(s["lengths"][b])].long()
            count = torch.bincount(seen, minlength=V).double()
            r = s["repetition"][b].double()
            row = torch.where(count > 0, torch.where(row > 0, row / r, row * r), row)
            row = row - s["frequency"][b].double() * count
            row = row - s["presence"][b].double() * (count > 0)
        if s["bias"] is not None:
            row = row.index_add(0, s["bias_ids"][b].long(), s["bias"][b].double())
        if s["mask"] is not None:
            bits = s["mask"][b].long().unsqueeze(1) >> torch.arange(32, device=row.device)
            row = row.masked_fill((bits & 1).reshape(-1)[:V] == 0, -math.inf)
        out[b] = row
    return {"out": out, "best": None}
