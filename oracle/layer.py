"""Plain fp64 numpy definitions of the rest of a layer: norms, decayed linear attention, AdamW.

Written from the formulas, token by token, sharing no code with the HIP path.
Inputs are float arrays holding the values that the device receives.
"""
from __future__ import annotations

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _silu(z):
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-z))
    return z * sig, sig * (1.0 + z * (1.0 - sig))


def res_norm_fwd(x, y=None, z=None, scale=None, w_post=None, w_pre=None, eps=1e-6):
    """x' = x + scale norm(y) w_post SiLU(z), xn = norm(x') w_pre, row by row."""
    x, y, z, scale, w_post, w_pre = (_f(t) for t in (x, y, z, scale, w_post, w_pre))
    new, xn = np.array(x), None if w_pre is None else np.zeros_like(x)
    for t in range(len(x)):
        if y is not None:
            n = y[t]
            if w_post is not None:
                n = n / np.sqrt((n * n).mean() + eps) * w_post
            if z is not None:
                n = n * _silu(z[t])[0]
            if scale is not None:
                n = n * scale
            new[t] = x[t] + n
        if w_pre is not None:
            xn[t] = new[t] / np.sqrt((new[t] * new[t]).mean() + eps) * w_pre
    return new, xn


def _norm_bwd(x, w, d, eps):
    """Gradients of x / sqrt(mean x^2 + eps) * w with respect to x and w, for the gradient d."""
    r = 1.0 / np.sqrt((x * x).mean() + eps)
    e = d * w
    return r * e - r ** 3 * x * (e * x).mean(), d * x * r


def res_norm_bwd(dxn, dx_new, x_new, y=None, z=None, scale=None, w_post=None, w_pre=None,
                 eps=1e-6):
    """dict(dx, dy, dz, dscale, dw_post, dw_pre), None where there is no such input."""
    x, y, z, scale, w_post, w_pre = (_f(t) for t in (x_new, y, z, scale, w_post, w_pre))
    dxn, dx_new = _f(dxn), _f(dx_new)
    out = {"dx": np.zeros_like(x) if dx_new is None else np.array(dx_new)}
    for k, t in (("dy", y), ("dz", z), ("dscale", scale), ("dw_post", w_post), ("dw_pre", w_pre)):
        out[k] = None if t is None else np.zeros_like(t)
    for t in range(len(x)):
        if w_pre is not None:
            dx, dw = _norm_bwd(x[t], w_pre, dxn[t], eps)
            out["dx"][t] += dx
            out["dw_pre"] += dw
        if y is None:
            continue
        g, dg = (1.0, 0.0) if z is None else _silu(z[t])
        s = 1.0 if scale is None else scale
        n = y[t]
        if w_post is not None:
            n = n / np.sqrt((n * n).mean() + eps) * w_post
        d = out["dx"][t]
        if scale is not None:
            out["dscale"] += d * n * g
        if z is not None:
            out["dz"][t] = d * s * n * dg
        if w_post is None:
            out["dy"][t] = d * s * g
        else:
            out["dy"][t], dw = _norm_bwd(y[t], w_post, d * s * g, eps)
            out["dw_post"] += dw
    return out


def linattn_fwd(q, k, v, log_decay, state=None, lengths=None, scale=1.0):
    """S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t; zeros behind a row's
    length.  q [B, L, H, dk], k [B, L, Hk, dk], v [B, L, Hk, dv]; returns o and the last state."""
    q, k, v, a = _f(q), _f(k), _f(v), _f(log_decay)
    B, L, H, dk = q.shape
    group, dv = H // k.shape[2], v.shape[3]
    S = np.zeros((B, H, dk, dv)) if state is None else np.array(_f(state))
    o = np.zeros((B, L, H, dv))
    lam = np.exp(a)
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for h in range(H):
            s = S[b, h]
            for t in range(n):
                s = lam[h] * s + np.outer(k[b, t, h // group], v[b, t, h // group])
                o[b, t, h] = scale * (q[b, t, h] @ s)
            S[b, h] = s
    return o, S


def linattn_bwd(q, k, v, log_decay, do, state=None, dstate=None, lengths=None, scale=1.0):
    """dict(dq, dk, dv, dstate): the adjoint of the state carried back in time."""
    q, k, v, a, do = _f(q), _f(k), _f(v), _f(log_decay), _f(do)
    B, L, H, dk = q.shape
    group, dv = H // k.shape[2], v.shape[3]
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v),
           "dstate": np.zeros((B, H, dk, dv))}
    lam = np.exp(a)
    for b in range(B):
        n = L if lengths is None else min(max(int(lengths[b]), 0), L)
        for h in range(H):
            j = h // group
            s = np.zeros((dk, dv)) if state is None else _f(state)[b, h]
            for t in range(n):
                s = lam[h] * s + np.outer(k[b, t, j], v[b, t, j])
                out["dq"][b, t, h] = scale * (s @ do[b, t, h])
            m = np.zeros((dk, dv)) if dstate is None else np.array(_f(dstate)[b, h])
            for t in range(n - 1, -1, -1):
                m = m + scale * np.outer(q[b, t, h], do[b, t, h])
                out["dk"][b, t, j] += m @ v[b, t, j]
                out["dv"][b, t, j] += m.T @ k[b, t, j]
                m = lam[h] * m
            out["dstate"][b, h] = m
    return out


def adamw(p, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
          grad_scale=1.0):
    """p, m, v after the step, element by element."""
    p, g, m, v = (_f(t) for t in (p, g, m, v))
    g = g * float(grad_scale)
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    mhat, vhat = m / (1.0 - beta1 ** step), v / (1.0 - beta2 ** step)
    with np.errstate(all="ignore"):
        p = p - lr * weight_decay * p - lr * mhat / (np.sqrt(vhat) + eps)
    return p, m, v


def e4m3_values():
    """The finite values of the 8-bit float (4 exponent bits of bias 7, 3 mantissa bits, no
    infinities, the two codes of all ones NaN) that are not negative, by code 0 .. 126."""
    return np.array([(c & 7) / 8.0 * 2.0 ** -6 if c < 8 else
                     (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7) for c in range(127)])
