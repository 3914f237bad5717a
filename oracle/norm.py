"""The norms before and after the layer, oracle side (test infrastructure); fp64.

RMS norm (the normalisation the Jamba pages name): v / sqrt(mean(v^2) + eps) per
token. Before the layer it gives the layer's input; after it, the layer's output
is normalised, gated and added to the residual stream, and the next block's norm
may follow.
"""
from __future__ import annotations

import numpy as np


def rms(v, weight, eps):
    v = np.asarray(v, dtype=np.float64)
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def post(y, residual, weight=None, gate=None, gate_tokens=1, residual_scale=1.0, block_scale=1.0, eps=1e-6,
         next_weight=None, next_eps=None):
    """(out, next or None) as stated above; gate row of token t is t // gate_tokens."""
    n = np.asarray(y, dtype=np.float64) if weight is None else rms(y, weight, eps)
    if gate is not None:
        n = n * np.asarray(gate, dtype=np.float64)[np.arange(len(n)) // gate_tokens]
    out = residual_scale * np.asarray(residual, dtype=np.float64) + block_scale * n
    nxt = None if next_weight is None else rms(out, next_weight, eps if next_eps is None else next_eps)
    return out, nxt
