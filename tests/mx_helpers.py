"""Inputs and derived bounds of the MXFP4 tests.

Error bound of a product (fp32 sums): each product of a 4-bit weight and a bf16
or 4-bit activation is exact (at most 2 + 8 significant bits), and a sum of Kd
terms takes at most Kd additions, each off by at most 2^-23 of the largest
partial sum (a truncating adder; half of that if it rounds), so
    |out - exact| <= Kd * 2^-23 * sum_k |a_k w_k|.
SwiGLU h = silu(g) * u with |silu'| <= 1.1: an error dg, du gives at most
1.1 |u| dg + |silu(g)| du, plus the function itself: the exponential's argument
is off by 2^-23 |g| and its result, the reciprocal and two products by some 2^-22
each: at most (8 + |g|) * 2^-22 of |h|. A bf16 result adds half a step, 2^-8 |out|.
"""
from __future__ import annotations

import numpy as np
import torch

from oracle import mxfp4 as omx

EPS = 2.0 ** -23


def segments(counts, S, rng):
    """expert_offsets for these counts and a shuffled slot list over S slots (rows past the last segment: -1)."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    assert off[-1] <= S
    slots = rng.permutation(S).astype(np.int32)
    slots[off[-1]:] = -1
    return off, slots


def draw_mx(rng, *shape, sigma=0.05, spread=3):
    """MXFP4 codes and scales of random numbers whose blocks differ in magnitude by up to 2^(2*spread)."""
    w = rng.standard_normal(shape) * sigma
    blk = w.reshape(*shape[:-1], shape[-1] // 32, 32)
    blk *= 2.0 ** rng.integers(-spread, spread + 1, blk.shape[:-1])[..., None]
    return omx.quantize(w.astype(np.float32))


def bf16_exact(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def product_bound(a, w, off, rows, w2=None, bf16=False):
    """(exact, bound) of out[r] for r below the last segment; NaN rows past it."""
    Kd = a.shape[1]
    ref = omx.grouped_product(a, w, off, rows, w2)
    mag = omx.grouped_product(np.abs(a), np.abs(w), off, rows)
    if w2 is None:
        bound = Kd * EPS * mag
    else:
        g, u = omx.grouped_product(a, w, off, rows), omx.grouped_product(a, w2, off, rows)
        mag2 = omx.grouped_product(np.abs(a), np.abs(w2), off, rows)
        silu = np.abs(g / (1 + np.exp(-g)))
        bound = 1.1 * np.abs(u) * Kd * EPS * mag + silu * Kd * EPS * mag2 + (8 + np.abs(g)) * 2 * EPS * np.abs(ref)
    if bf16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    return ref, bound + 1e-37


def check(got, ref, bound, last, what):
    got = got.double().cpu().numpy()
    err = np.abs(got[:last] - ref[:last])
    bad = ~(err <= bound[:last])
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst "
                           f"{np.nanmax(err / bound[:last]):.3g} of it at {np.unravel_index(np.nanargmax(err / bound[:last]), err.shape)}")
