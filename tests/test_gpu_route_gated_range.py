"""Gated routing over the range of its logits, against the fp64 oracle.

Logits that fp32 does not hold apart, up to 2^119. The inputs make every 64-bit logit exact, or leave
the largest far above the error of any 64-bit sum, so ids are compared for equality; all logits are taken in 64 bits
there (their fp32 error is past any use), so a weight is off by its rounding to fp32, 2^-24, and as much again for the
64-bit exponentials, sum and division, or by the smallest number of fp32.
"""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from oracle import gate as ogate
from tests.helpers import np64
from tests.test_gpu_route_gated import DT, _gate

pytestmark = pytest.mark.gpu

INF = float("inf")


def _say(msg):
    print(f"[gate-range-test] {msg}", file=sys.stderr, flush=True)


def _exactly(x, wr, bias, K, select=None, what="", **kw):
    """Ids equal to the oracle's, weights to fp32's rounding, with and without a workspace."""
    _say(f"{what} T={x.shape[0]} d={x.shape[1]} E={wr.shape[0]} K={K} {x.dtype} select={select is not None} {kw}")
    b = None if bias is None else torch.from_numpy(bias).cuda()
    with np.errstate(invalid="ignore"):
        rid, rw, l = ogate.route(np64(x), np64(wr), bias, K, select_bias=select, **kw)
    for use_workspace in (True, False):
        ids, w = m.moe_route_gated(x.cuda(), wr.cuda(), b, K, _gate(select, **kw), use_workspace=use_workspace)
        got, gw = ids.cpu().numpy(), np64(w)
        bad = np.argwhere((got != rid).any(1))[:, 0]
        assert bad.size == 0, f"{what}: token {bad[0]}: {got[bad[0]]}, not {rid[bad[0]]} ({bad.size} tokens)"
        assert (np.abs(gw - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149).all(), what
    return l


# d of 64: one block of columns; 8192 bf16 or 4096 fp32 ones of more: few tokens' rows split over workgroups
@pytest.mark.parametrize("E,groups,group_topk,K", [(1, 1, 1, 1), (2, 1, 1, 1), (16, 1, 1, 3), (60, 4, 2, 4), (256, 8, 3, 8)])
@pytest.mark.parametrize("power", [24, 28, 31, 34, 40, 52, 80, 119])
@pytest.mark.parametrize("d", [64, 8192])
def test_softmax_of_logits_finer_than_fp32(E, groups, group_topk, K, power, d):
    """Logits of 2^power (or minus it) and offsets below fp32's step there, so that the largest rounds up for one token and
    down for another: by up to half of 2^(power - 23)."""
    rng = np.random.default_rng(E * 131 + power)
    T = 64
    # 2^power and the offsets are whole units, below 2^53 of them. Between two logits lie less than 690 or more than 800, so a
    # score is a normal number or 0: the smallest ones depend on whose exponential it is.
    unit = 2.0 ** max(0, power - 46)
    step = 2.0 ** (power - 23)
    if power < 32:
        first, second = rng.integers(0, max(2, min(step, 224)), E), rng.integers(0, max(2, min(2 * step, 440)), (E, 8))
    else:
        first = max(1024.0, unit) * rng.integers(0, int(step / max(1024.0, unit)), E)
        second = unit * rng.integers(0, 1 + min(7, int(200 / unit)), (E, 8))
    x, wr = np.zeros((T, d), np.float32), np.zeros((E, d), np.float32)
    x[:, 0] = 2.0 ** (power // 2) * np.where(np.arange(T) < T // 2, 1, -1)
    wr[:, 0] = 2.0 ** (power - power // 2)
    x[:, 32] = 1                                       # the same offsets for all tokens ...
    wr[:, 32] = first
    x[:, 33 + np.arange(8)] = np.eye(8)[np.arange(T) % 8]   # ... and some that differ
    wr[:, 33:41] = second
    x, wr = torch.from_numpy(x), torch.from_numpy(wr)
    small = (0.3 * rng.standard_normal(E)).astype(np.float32)
    some = small.copy()
    some[rng.permutation(E)[:E // 4]] = -INF
    for select, renorm in ((None, True), (None, False), (small, True), (some, False)):
        _exactly(x, wr, None, K, select, f"2^{power}", groups=groups, group_topk=group_topk, top2=E // groups > 1, renorm=renorm)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e8, 2e9, 1e12, 1e20, 1e34])
@pytest.mark.parametrize("E,K", [(2, 1), (16, 4), (64, 4), (256, 8)])
def test_softmax_of_huge_normal_logits(E, K, scale, act):
    """Normal logits of this size: one expert has all the weight, the others' scores are zeros, which tie or go by the bias."""
    rng = np.random.default_rng(E + 7)
    T, d = 300, 256
    x = torch.from_numpy((rng.standard_normal((T, d)) * scale).astype(np.float32)).to(DT[act])
    wr = torch.from_numpy((0.05 * rng.standard_normal((E, d))).astype(np.float32)).to(DT[act])
    l = np.sort(np64(x) @ np64(wr).T, 1)
    # 64-bit sums are off by d 2^-53 of the magnitudes at most: tokens with less than 1000 and as much between any two logits go
    apart = 1000 + 4 * d * 2.0 ** -53 * (np.abs(np64(x)) @ np.abs(np64(wr)).T).max(1)
    keep = np.diff(l, axis=1).min(1) > apart
    assert keep.mean() > (0.9 if scale > 1e9 else 0.2)
    x = x[torch.from_numpy(keep)]
    select = (0.3 * rng.standard_normal(E)).astype(np.float32)
    for sel in (None, select):
        for renorm in (False, True):
            _exactly(x, wr, None, K, sel, f"{scale}", renorm=renorm, scale=2.0)
        _exactly(x, wr, None, K, sel, f"{scale}", groups=2, group_topk=1, top2=E > 2)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("E", [16, 256])
def test_softmax_of_a_row_past_any_exponential(E, act):
    """A token 1e36 times the others, among them, with biases of -inf, of inf and far above any score."""
    rng = np.random.default_rng(E + 3)
    x = torch.from_numpy(rng.standard_normal((5, 128)).astype(np.float32)).to(DT[act])
    wr = torch.from_numpy((0.02 * rng.standard_normal((E, 128))).astype(np.float32)).to(DT[act])
    x[3] = (x[3].float() * 1e36).to(x.dtype)
    top = np.sort(np64(x[3:4]) @ np64(wr).T, 1)
    assert 2.0 ** 110 < abs(top[0, -1]) < 2.0 ** 120 and top[0, -1] - top[0, -3] > 1e30
    bias = np.zeros(E, np.float32)
    bias[1] = -INF
    select = (0.1 * rng.standard_normal(E)).astype(np.float32)
    select[2] = 1e6
    select[3] = INF
    for renorm in (False, True):
        for b, sel in ((bias, select), (None, None), (bias, None), (None, select)):
            _exactly(x[3:4], wr, b, 4, sel, "huge row", renorm=renorm)
            ids, w = m.moe_route_gated(x.cuda(), wr.cuda(), None if b is None else torch.from_numpy(b).cuda(), 4,
                                       _gate(sel, renorm=renorm))
            alone = m.moe_route_gated(x[3:4].cuda(), wr.cuda(), None if b is None else torch.from_numpy(b).cuda(), 4,
                                      _gate(sel, renorm=renorm))
            assert torch.equal(ids[3:4], alone[0]) and torch.equal(w[3:4], alone[1])
            assert (ids >= 0).all() and torch.isfinite(w).all()
