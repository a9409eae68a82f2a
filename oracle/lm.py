"""Plain fp64 numpy definitions of the operators around the mixer layer.

Written from the formulas, one row at a time, sharing no code with the HIP
path.  Inputs are float arrays holding the values that the device receives.
"""
from __future__ import annotations

import numpy as np


def embed_fwd(ids, W, scale):
    """out[t] = scale W[ids[t]]; zeros where the id is outside the vocabulary."""
    W = np.asarray(W, dtype=np.float64)
    out = np.zeros((len(ids), W.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < W.shape[0]:
            out[t] = scale * W[v]
    return out


def embed_bwd(ids, dout, vocab, scale):
    """dW[v] = scale sum_{t: ids[t] = v} dout[t]."""
    dout = np.asarray(dout, dtype=np.float64)
    dW = np.zeros((vocab, dout.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            dW[v] += scale * dout[t]
    return dW


def distill(logits, t_ids, t_logits, tau, g=None):
    """loss, lse and (with g) the gradient of the distillation loss, row by row."""
    R, V = logits.shape
    loss, lse, grad = np.zeros(R), np.zeros(R), np.zeros((R, V))
    with np.errstate(all="ignore"):
        for r in range(R):
            x = np.asarray(logits[r], dtype=np.float64) / tau
            top = x.max() if np.isfinite(x.max()) else 0.0
            log_sum = np.log(np.exp(x - top).sum())
            lse[r] = top + log_sum
            use = [j for j, i in enumerate(t_ids[r]) if 0 <= i < V and t_logits[r, j] != -np.inf]
            if not use:
                continue
            idx = t_ids[r, use]
            t = np.asarray(t_logits[r, use], dtype=np.float64) / tau
            e = np.exp(t - t.max())
            p = e / e.sum()
            logp = t - t.max() - np.log(e.sum())
            # (x - lse would lose the sum's logarithm where the logits are huge)
            logq = x - top - log_sum
            if not np.isnan(log_sum):  # (NaN makes the whole row NaN)
                logq[x == -np.inf] = -np.inf
            terms = np.where(p == 0, 0.0, p * (logp - logq[idx]))
            loss[r] = tau * tau * terms.sum()
            if g is not None and g[r] != 0:
                d = np.exp(logq)
                for j, i in enumerate(idx):
                    d[i] -= p[j]
                grad[r] = g[r] * tau * d
    return loss, lse, grad


def logits_process(logits, history=None, lengths=None, repetition=None, presence=None,
                   frequency=None, bias_ids=None, bias=None, mask=None):
    """out, best: penalties, biases and mask, token by token of each row's lists."""
    out = np.array(logits, dtype=np.float64)
    R, V = out.shape
    best = np.full(R, -1, dtype=np.int64)
    for b in range(R):
        counts = {}
        if history is not None:
            n = history.shape[1] if lengths is None else min(max(int(lengths[b]), 0),
                                                             history.shape[1])
            for v in history[b, :n].tolist():
                if 0 <= v < V:
                    counts[v] = counts.get(v, 0) + 1
        for v, c in counts.items():
            x = out[b, v]
            if repetition is not None:
                x = x / float(repetition[b]) if x > 0 else x * float(repetition[b])
            if frequency is not None:
                x -= float(frequency[b]) * c
            if presence is not None:
                x -= float(presence[b])
            out[b, v] = x
        if bias_ids is not None:
            done = set()
            for v, add in zip(bias_ids[b].tolist(), bias[b].tolist()):
                if 0 <= v < V and v not in done:
                    done.add(v)
                    out[b, v] += add
        if mask is not None:
            for v in range(V):
                if not (int(mask[b, v // 32]) >> (v % 32)) & 1:
                    out[b, v] = -np.inf
        x = np.where(np.isnan(out[b]), -np.inf, out[b])
        if V and x.max() > -np.inf:
            best[b] = int(np.flatnonzero(x == x.max())[0])
    return out, best


def w4_weights(qweight, scales, group, zeros=None):
    """The weights [d_out, d_in] that codes, scales and zeros stand for."""
    q = np.asarray(qweight, dtype=np.int64)
    N, half = q.shape
    w = np.zeros((N, 2 * half))
    for i in range(half):
        w[:, 2 * i] = q[:, i] % 16
        w[:, 2 * i + 1] = q[:, i] // 16
    for k in range(2 * half):
        z = 8.0 if zeros is None else np.asarray(zeros[:, k // group], dtype=np.float64)
        w[:, k] = (w[:, k] - z) * np.asarray(scales[:, k // group], dtype=np.float64)
    return w


def w4_linear(x, qweight, scales, group, zeros=None, bias=None, res=None):
    """y = x W^T + bias + res with the weights above."""
    y = np.asarray(x, dtype=np.float64) @ w4_weights(qweight, scales, group, zeros).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    if res is not None:
        y = y + np.asarray(res, dtype=np.float64)
    return y
