"""The norms before and after the layer on the GPU against fp64.

Bounds, from the arithmetic: a mean of d squares takes at most d additions, each
off by 2^-24, and the squares themselves 2^-24, so the reciprocal root is off by
at most (d / 2 + 4) * 2^-24 relative (half of it for the root; the division and
the root itself one step each); every later product or sum adds 2^-24 of its
result's or its terms' magnitude. The type's rounding adds eps/2 of the value.
"""
import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from oracle import norm as onorm
from tests.helpers import np64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def _half_step(act):
    return float(torch.finfo(DT[act]).eps) / 2


def _draw(rng, *shape, act, scale=1.0, mean=0.0):
    return torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(DT[act])


def _bounds(y, y_err, residual, kw, act):
    """(out, bound, next, bound) with y known up to y_err (elementwise)."""
    d = y.shape[1]
    f64 = {k: (np64(v) if torch.is_tensor(v) else v) for k, v in kw.items()}
    out, nxt = onorm.post(y, np64(residual), **f64)
    a, b = kw.get("residual_scale", 1.0), kw.get("block_scale", 1.0)
    n, n_err = y, y_err
    if kw.get("weight") is not None:
        n = onorm.rms(y, f64["weight"], kw.get("eps", 1e-6))
        rel = (d / 2 + 8) * U
        # an error of y moves an element by its own share, and all of them through the mean
        r = 1 / np.sqrt((y * y).mean(1, keepdims=True) + kw.get("eps", 1e-6))
        shift = np.abs(y * y_err).mean(1, keepdims=True) * r * r
        n_err = np.abs(f64["weight"]) * r * y_err + np.abs(n) * (rel + shift)
    g = 1.0
    if kw.get("gate") is not None:
        g = np.abs(f64["gate"])[np.arange(len(y)) // kw.get("gate_tokens", 1)]
    # the scales are fp32 arguments: half a step each
    terms = np.abs(a * np64(residual)) + np.abs(b) * g * np.abs(n)
    err = np.abs(b) * g * n_err + 6 * U * terms + 1e-37
    bound = err + _half_step(act) * (np.abs(out) + err)
    nbound = None
    if nxt is not None:
        ne = kw.get("next_eps")
        ne = kw.get("eps", 1e-6) if ne is None else ne
        r = 1 / np.sqrt((out * out).mean(1, keepdims=True) + ne)
        shift = np.abs(out * err).mean(1, keepdims=True) * r * r
        e = np.abs(f64["next_weight"]) * r * err + np.abs(nxt) * ((d / 2 + 8) * U + shift) + 1e-37
        nbound = e + _half_step(act) * (np.abs(nxt) + e)
    return out, bound, nxt, nbound


def _check(got, ref, bound, what):
    err = np.abs(np64(got) - ref)
    assert (err <= bound).all(), f"{what}: worst {np.max(err / bound):.3g} of the bound"


# every row length class of the kernel, its edges, and lengths that leave threads without a chunk
SIZES = [(1, 64), (3, 320), (2, 512), (5, 2048), (4, 2112), (1, 4096), (7, 8192), (2, 8256), (3, 16384), (2, 32768),
         (2, 32832), (1, 65536), (600, 192), (1030, 1024), (1025, 4160), (1024, 16384)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES)
def test_norm_pre(T, d, act):
    rng = np.random.default_rng(T + d)
    x, w = _draw(rng, T, d, act=act, scale=3.0), _draw(rng, d, act=act, scale=0.2, mean=1.0)
    x[0] = 0                                                       # a zero row gives zeros
    got = m.moe_norm_pre(x.cuda(), w.cuda(), 1e-5)
    ref = onorm.rms(np64(x), np64(w), 1e-5)
    err = np.abs(ref) * (d / 2 + 8) * U + 1e-37
    _check(got, ref, err + _half_step(act) * (np.abs(ref) + err), "pre")
    assert (got[0] == 0).all()
    inplace = x.cuda()
    assert m.moe_norm_pre(inplace, w.cuda(), 1e-5, out=inplace).data_ptr() == inplace.data_ptr()
    assert torch.equal(inplace, got)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SIZES)
@pytest.mark.parametrize("kind", ["plain", "norm", "gate", "all"])
def test_norm_post(T, d, kind, act):
    rng = np.random.default_rng(T * d + len(kind))
    y, res = _draw(rng, T, d, act=act, scale=2.0), _draw(rng, T, d, act=act)
    kw = {}
    if kind != "plain":
        kw["weight"] = _draw(rng, d, act=act, scale=0.2, mean=1.0)
    if kind in ("gate", "all"):
        kw["gate_tokens"] = max(1, T // 3)
        kw["gate"] = _draw(rng, -(-T // kw["gate_tokens"]), d, act=act)
    if kind == "all":
        kw.update(residual_scale=0.75, block_scale=-1.5, eps=1e-5, next_weight=_draw(rng, d, act=act, mean=1.0),
                  next_eps=1e-3)
    dkw = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in kw.items()}
    out, nxt = m.moe_norm_post(y.cuda(), res.cuda(), **dkw)
    ro, bo, rn, bn = _bounds(np64(y), np.zeros((T, d)), res, kw, act)
    _check(out, ro, bo, "out")
    assert (nxt is None) == (rn is None)
    if nxt is not None:
        _check(nxt, rn, bn, "next")
    for alias in ("residual", "y"):
        yy, rr = y.cuda(), res.cuda()
        o2, n2 = m.moe_norm_post(yy, rr, out=rr if alias == "residual" else yy, **dkw)
        assert torch.equal(o2, out) and (nxt is None or torch.equal(n2, nxt)), alias


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,K", [(1, 64, 1), (3, 2048, 2), (17, 8192, 2), (2, 4160, 8), (65, 320, 3), (2, 65536, 2),
                                   (530, 256, 2)])
def test_combine_post(T, d, K, act):
    rng = np.random.default_rng(T + d + K)
    rows = torch.from_numpy(rng.standard_normal((T * K, d)).astype(np.float32))
    s2r = torch.from_numpy(rng.permutation(T * K).astype(np.int32))
    s2r[rng.integers(0, T * K, max(1, T * K // 7))] = -1            # slots without a row
    s2r[:K] = -1                                                    # and a token without any
    gw = torch.from_numpy(rng.uniform(0.1, 1, (T, K)).astype(np.float32))
    res = _draw(rng, T, d, act=act)
    kw = dict(weight=_draw(rng, d, act=act, mean=1.0, scale=0.1), gate=_draw(rng, T, d, act=act), residual_scale=0.5,
              block_scale=2.0, next_weight=_draw(rng, d, act=act, mean=1.0, scale=0.1))
    r = s2r.view(T, K).numpy()
    terms = np.where((r >= 0)[..., None], np64(gw)[..., None] * np64(rows)[np.maximum(r, 0)], 0.0)
    y = terms.sum(1)
    dkw = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in kw.items()}
    out, nxt = m.moe_combine_post(rows.cuda(), s2r.cuda(), gw.cuda(), res.cuda(), **dkw)
    ro, bo, rn, bn = _bounds(y, 2 * K * U * np.abs(terms).sum(1), res, kw, act)
    _check(out, ro, bo, "out")
    _check(nxt, rn, bn, "next")


@pytest.mark.parametrize("T,d,act", [(16400, 2048, "bf16"), (4100, 8192, "bf16"), (1100, 32768, "bf16"),
                                     (300, 65536, "f32")])
def test_large_outputs(T, d, act):
    """Outputs of 64 MiB and more (stored past the caches) are the same as those of a part of the rows on their own."""
    g = torch.Generator(device="cuda").manual_seed(T)
    y, res = (torch.randn(T, d, generator=g, device="cuda").to(DT[act]) for _ in range(2))
    w = torch.ones(d, dtype=DT[act], device="cuda")
    n = m.moe_norm_pre(y, w)
    out, nxt = m.moe_norm_post(y, res, weight=w, next_weight=w)
    for lo in (0, T // 2, T - 3):
        # few rows take another spread of the row over threads: the sums' order differs, the bound is the same
        rows = slice(lo, lo + 3)
        ro, bo, rn, bn = _bounds(np64(y[rows]), np.zeros((3, d)), res[rows], dict(weight=w.cpu(), next_weight=w.cpu()), act)
        _check(out[rows], ro, bo, "out")
        _check(nxt[rows], rn, bn, "next")
        ref = onorm.rms(np64(y[rows]), np64(w), 1e-6)
        err = np.abs(ref) * (d / 2 + 8) * U + 1e-37
        _check(n[rows], ref, err + _half_step(act) * (np.abs(ref) + err), "pre")


def test_nan_and_infinity_stay_in_their_tokens():
    x = torch.randn(5, 4096, dtype=torch.bfloat16)
    x[1, 7], x[3, 4000] = float("nan"), float("inf")
    w = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    n = m.moe_norm_pre(x.cuda(), w).cpu()
    assert n[1].isnan().all() and n[3, 4000].isnan()
    assert torch.isfinite(n[[0, 2, 4]]).all()
    out, nxt = m.moe_norm_post(x.cuda(), torch.zeros_like(x).cuda(), weight=w, next_weight=w)
    assert torch.isfinite(out[[0, 2, 4]]).all() and torch.isfinite(nxt[[0, 2, 4]]).all()


def test_norm_on_a_side_stream_and_empty():
    x = torch.randn(9, 512, device="cuda")
    w = torch.ones(512, device="cuda")
    a = m.moe_norm_pre(x, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b = m.moe_norm_pre(x, w)
    side.synchronize()
    assert torch.equal(a, b)
    e = torch.empty(0, 512, device="cuda")
    assert m.moe_norm_pre(e, w).shape == (0, 512)
    out, nxt = m.moe_norm_post(e, e, weight=w, next_weight=w)
    assert out.shape == nxt.shape == (0, 512)


def test_refusals_on_the_device():
    y, w = torch.randn(4, 128, device="cuda"), torch.ones(128, device="cuda")
    rows, gw = torch.randn(8, 128, device="cuda"), torch.ones(4, 2, device="cuda")
    s2r = torch.arange(8, dtype=torch.int32, device="cuda")
    ok = m.moe_combine_post(rows, s2r.view(4, 2), gw, y, weight=w)[0]
    assert torch.equal(ok, m.moe_combine_post(rows, s2r, gw, y, weight=w)[0])
    with pytest.raises(ValueError, match="slot_to_row"):
        m.moe_combine_post(rows, s2r[:7], gw, y, weight=w)
    with pytest.raises(TypeError, match="residual"):
        m.moe_norm_post(y, y.to(torch.bfloat16), weight=w)
    with pytest.raises(ValueError, match="gate has shape"):
        m.moe_norm_post(y, y, weight=w, gate=torch.ones(2, 128, device="cuda"), gate_tokens=1)
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_norm_pre(torch.randn(128, 64, device="cuda").t(), torch.ones(128, device="cuda"))
    with pytest.raises(m.MoeError) as e:
        m.moe_norm_pre(y, w, eps=-1.0)
    assert e.value.status == 2
    with pytest.raises(m.MoeError) as e:
        m.moe_norm_post(y, y, weight=w, gate=torch.ones(4, 128, device="cuda"), gate_tokens=0)
    assert e.value.status == 2
