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
