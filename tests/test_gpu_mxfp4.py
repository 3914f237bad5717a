"""MXFP4 on the GPU: quantizer, layouts, the expert FFN's passes with MXFP4 weights, products of MXFP4 by MXFP4."""
import ctypes
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd import _lib, ops
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED, MOE_W_MXFP4
from oracle import moe as omoe
from oracle import mxfp4 as omx
from tests.helpers import np64
from tests.mx_helpers import bf16_exact, check, draw_mx, product_bound, segments

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PATHS = [MOE_PATH_STREAM, MOE_PATH_TILED]


def _say(msg):
    print(f"[mxfp4-test] {msg}", file=sys.stderr, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ quantizer, dequantizer, packer

def _hard_rows(rows, cols, src, seed):
    """Normals of many magnitudes, exact ties, zeros of both signs, the smallest and largest numbers."""
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-40, 41, (rows, cols // 32)).repeat(32, 1)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, -0.25, -0.75, -5.0, -2.5, 0.0, -0.0])
    w[0, :16], w[0, 16:32] = ties, -ties
    if rows > 1:
        w[1, :32] = 0.0
        w[1, 3] = -0.0
    if rows > 2:
        w[2, :32] = 2.0 ** -126 * rng.uniform(-4, 4, 32)       # scale byte 0, subnormals among them
    if rows > 3:
        w[3, :32] = 3.3e38 * rng.uniform(-1, 1, 32)
    if rows > 4:
        w[4, :32] = 2.0 ** -133 * rng.integers(-3, 4, 32)      # the smallest bf16 numbers
    t = torch.from_numpy(w.astype(np.float32))
    return t.to(DT[src])


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (2, 4096), (33, 160), (513, 1056), (2051, 4128)])
def test_quantize_rows_bit_exact(rows, cols, src):
    w = _hard_rows(rows, cols, src, rows * cols)
    q, s = m.moe_quantize_mxfp4(w.cuda())
    rq, rs = omx.quantize(np64(w))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(16, 128), (32, 256), (48, 384), (16, 512), (32, 640), (80, 1152), (16, 4224)])
def test_quantize_tiled_bit_exact(rows, cols, src):
    w = _hard_rows(rows, cols, src, rows + cols)
    q, s = m.moe_quantize_mxfp4(w.cuda(), tiled=True)
    rq, rs = omx.quantize(np64(w))
    tq, ts = omx.tile(rq, rs)
    assert np.array_equal(s.cpu().numpy(), ts)
    assert np.array_equal(q.cpu().numpy(), tq)
    pq, ps = m.moe_pack_mxfp4(dev(rq), dev(rs))
    assert np.array_equal(pq.cpu().numpy(), tq) and np.array_equal(ps.cpu().numpy(), ts)
    back = m.moe_dequantize_mxfp4(q, s, torch.float32, tiled=True)
    assert np.array_equal(back.cpu().numpy().astype(np.float64), omx.dequantize(rq, rs))


def test_quantize_non_finite_blocks():
    w = torch.randn(16, 256)
    w[2, 5], w[3, 40], w[4, 255] = float("inf"), float("nan"), float("-inf")
    for dt in (torch.float32, torch.bfloat16):
        for tiled in (False, True):
            rq, rs = omx.quantize(np64(w.to(dt)))
            if tiled:
                rq, rs = omx.tile(rq, rs)
            q, s = m.moe_quantize_mxfp4(w.to(dt).cuda(), tiled=tiled)
            assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
            v = m.moe_dequantize_mxfp4(q, s, dt, tiled=tiled).cpu()
            assert v[2, :32].isnan().all() and v[3, 32:64].isnan().all() and v[4, 224:].isnan().all()
            assert int(v.isnan().sum()) == 96


@pytest.mark.parametrize("dst", ["bf16", "f32"])
def test_dequantize_every_code_and_scale(dst):
    """Row b holds every pair of codes under scale byte b: exact, or infinite past the type's range, or NaN."""
    q = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    s = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, 16))
    v = m.moe_dequantize_mxfp4(dev(q), dev(s), DT[dst]).float().cpu().numpy().astype(np.float64)
    ref = omx.dequantize(q, s)
    top = float(torch.finfo(DT[dst]).max)
    ref = np.where(np.abs(ref) > top, np.copysign(np.inf, ref), ref)
    assert np.array_equal(v, ref, equal_nan=True)


def test_quantizer_leaves_no_gap_and_takes_empty():
    q, s = m.moe_quantize_mxfp4(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    w = torch.randn(3, 5, 64, device="cuda")
    q, s = m.moe_quantize_mxfp4(w)
    assert q.shape == (3, 5, 32) and s.shape == (3, 5, 2)


# ------------------------------------------------------------------ products

# (counts of rows per expert, unplaced rows, d, f): one row, empty experts, segments that end inside a tile of every
# kernel, reduction steps that leave a partial scale group, sizes that are no multiple of a workgroup's channels
CASES = [
    ([1], 0, 128, 128),
    ([0, 1, 0, 1], 0, 256, 384),
    ([0, 0, 0], 5, 256, 256),
    ([3, 0, 16, 17, 1], 3, 640, 256),
    ([33, 7, 0, 15], 0, 512, 640),
    ([64, 65, 1], 1, 384, 896),
    ([129, 0, 128, 127, 2, 31], 7, 896, 512),
    ([300], 0, 1152, 1408),
    ([0, 257, 0], 2, 2048, 128),
    ([1] * 40 + [0] * 24, 0, 256, 256),
]
# many channel groups (the wide items of the streaming kernel, one and two row blocks, a second pass over the
# weights), long reductions (all its splits, a partial last scale group) and, for the tiled kernel, many rounds of tiles
LARGE = [
    ([9, 0, 1, 16, 17] + [2] * 11, 0, 4096, 256),
    ([20, 0, 33, 16, 17] + [12] * 11, 0, 4096, 128),
    ([9, 0, 1, 16, 17] + [2] * 11, 0, 256, 2048),
    ([20, 0, 33, 16, 17] + [12] * 11, 0, 128, 2048),
    ([3, 0, 18], 1, 4224, 128),
    ([3, 0, 18], 1, 128, 4224),
    ([2] * 40 + [0] * 23 + [130], 0, 128, 4096),
    ([70, 3, 64, 129] + [10] * 12, 0, 384, 12416),
]


def _slots_for(counts, extra, rng, K=2):
    """S = rows of the segments plus unplaced ones, a multiple of K."""
    S = sum(counts) + extra
    S += -S % K
    off, slots = segments(counts, S, rng)
    return S, off, slots


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("counts,extra,d,f", CASES + LARGE)
def test_ffn_passes(counts, extra, d, f, path):
    rng = np.random.default_rng(d + f + sum(counts))
    E, K = len(counts), 2 if len(counts) > 1 else 1
    S, off, slots = _slots_for(counts, extra, rng, K)
    T = S // K
    mats = {}
    for name, (r, c) in (("gate", (f, d)), ("up", (f, d)), ("down", (d, f))):
        mats[name] = draw_mx(rng, E, r, c)
    ex = m.pack_mxfp4_experts(*(dev(mats[k][0]) for k in ("gate", "up", "down")),
                              *(dev(mats[k][1]) for k in ("gate", "up", "down")))
    assert (ex.d, ex.f, ex.E) == (d, f, E)
    W = {k: omx.dequantize(*v) for k, v in mats.items()}
    x = bf16_exact(rng.standard_normal((T, d)))
    h = bf16_exact(rng.standard_normal((S, f)) * rng.standard_normal((S, f)))
    _say(f"counts {counts} d {d} f {f} path {path}")
    doff, dslots = dev(off), dev(slots)
    last = int(off[-1])
    fill = torch.full((S, f), 7.0, dtype=torch.bfloat16, device="cuda")
    got = m.moe_expert_gate_up(x.cuda(), doff, dslots, ex, K, path=path, h=fill)
    ref, bound = product_bound(np64(x), W["gate"], off, slots // K, W["up"], bf16=True)
    check(got, ref, bound, last, "gate/up")
    assert (got[last:] == 7.0).all()
    fill = torch.full((S, d), 7.0, dtype=torch.float32, device="cuda")
    got = m.moe_expert_down(h.cuda(), doff, ex, T, K, path=path, y_rows=fill)
    ref, bound = product_bound(np64(h), W["down"], off, np.arange(S))
    check(got, ref, bound, last, "down")
    assert (got[last:] == 7.0).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,extra,d,f", CASES)
def test_grouped_mm(counts, extra, d, f, gather, swiglu, out, path):
    rng = np.random.default_rng(d * f + sum(counts))
    E = len(counts)
    K = 2 if gather and E > 1 else 1
    S, off, slots = _slots_for(counts, extra, rng, K)
    aq, asc = draw_mx(rng, S // K if gather else S, d, sigma=1.0)
    w, w2 = draw_mx(rng, E, f, d), draw_mx(rng, E, f, d)
    wt, w2t = m.moe_pack_mxfp4(dev(w[0]), dev(w[1])), m.moe_pack_mxfp4(dev(w2[0]), dev(w2[1]))
    _say(f"counts {counts} d {d} f {f} gather {gather} swiglu {swiglu} out {out} path {path}")
    fill = torch.full((S, f), 7.0, dtype=DT[out], device="cuda")
    got = m.moe_grouped_mm_mxfp4(dev(aq), dev(asc), dev(off), *wt, DT[out], sorted_slots=dev(slots) if gather else None,
                                 K=K, w2_q=w2t[0] if swiglu else None, w2_s=w2t[1] if swiglu else None, path=path,
                                 out=fill)
    ref, bound = product_bound(omx.dequantize(aq, asc), omx.dequantize(*w), off,
                               slots // K if gather else np.arange(S), omx.dequantize(*w2) if swiglu else None,
                               bf16=out == "bf16")
    check(got, ref, bound, int(off[-1]), "product")
    assert (got[int(off[-1]):] == 7.0).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,extra,d,f", LARGE)
def test_grouped_mm_large(counts, extra, d, f, swiglu, path):
    test_grouped_mm(counts, extra, d, f, True, swiglu, "f32", path)


@pytest.mark.parametrize("path", PATHS)
def test_nan_and_infinity_stay_in_their_rows(path):
    """A NaN block of a weight row, an infinite activation: only the outputs that read them are not finite."""
    rng = np.random.default_rng(5)
    counts, d, f = [20, 3], 256, 256
    S, off, slots = _slots_for(counts, 0, rng, 1)
    mats = [draw_mx(rng, 2, r, c) for r, c in ((f, d), (f, d), (d, f))]
    mats[0][1][0, 37, 5] = 255                                   # gate: expert 0, channel 37
    mats[2][1][1, 200, 0] = 255                                  # down: expert 1, channel 200
    ex = m.pack_mxfp4_experts(*(dev(q) for q, _ in mats), *(dev(s) for _, s in mats))
    x = bf16_exact(rng.standard_normal((S, d)))
    t = int(slots[22])                                           # the last row's token, of expert 1
    x[t, 9] = float("inf")
    h = m.moe_expert_gate_up(x.cuda(), dev(off), dev(slots), ex, 1, path=path).float().cpu()
    bad = ~torch.isfinite(h)
    assert bad[:20, 37].all() and not bad[:20, :37].any() and not bad[:20, 38:].any()
    assert not bad[20:22].any() and bad[22].any()
    hh = bf16_exact(rng.standard_normal((S, f)))
    y = m.moe_expert_down(hh.cuda(), dev(off), ex, S, 1, path=path).cpu()
    bad = ~torch.isfinite(y)
    assert bad[20:, 200].all() and int(bad.sum()) == 3


@pytest.mark.parametrize("path", PATHS)
def test_nan_block_of_an_activation_row(path):
    """A NaN scale of a row of codes reaches that row's outputs only, from its tokens' slots in both experts."""
    rng = np.random.default_rng(6)
    S, off, slots = _slots_for([18, 40], 0, rng, 2)
    aq, asc = draw_mx(rng, S // 2, 384)
    asc[3, 7] = 255
    w = draw_mx(rng, 2, 256, 384)
    wt = m.moe_pack_mxfp4(dev(w[0]), dev(w[1]))
    got = m.moe_grouped_mm_mxfp4(dev(aq), dev(asc), dev(off), *wt, torch.float32, sorted_slots=dev(slots), K=2, path=path)
    bad = got.isnan().cpu().numpy()
    hit = slots // 2 == 3
    assert bad[hit].all() and not bad[~hit].any() and hit.sum() == 2


def test_log_names_the_schedules(monkeypatch, capfd):
    monkeypatch.setenv("MOE_LOG", "1")
    ex = m.quantize_experts_mxfp4(*(torch.randn(1, 128, 128, device="cuda") for _ in range(3)))
    for T, gate_up, down in ((4, "stream", "stream"), (20, "stream", "stream"), (40, "tiled", "tiled"), (200, "tiled", "tiled")):
        x = torch.randn(T, 128, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        m.moe_expert_ffn_mxfp4(x, off, torch.arange(T, dtype=torch.int32, device="cuda"), ex, 1)
        err = capfd.readouterr().err
        lines = [l for l in err.splitlines() if l.startswith("[moe] moe_expert_ffn_mxfp4")]
        assert len(lines) == 2 and f"; {gate_up} schedule" in lines[0] and f"; {down} schedule" in lines[1], err
    m.moe_mlp_forward(x, ex)
    err = capfd.readouterr().err
    assert "moe_mlp_forward gate/up" in err and "act=bf16 weights=mxfp4" in err and "; tiled schedule" in err


def test_mismatched_widths_are_refused():
    ex = m.quantize_experts_mxfp4(*(torch.randn(2, r, c, device="cuda") for r, c in ((256, 128), (256, 128), (128, 256))))
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    srt = torch.arange(4, dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: m.moe_expert_gate_up(x, off, srt, ex, 1), lambda: m.moe_expert_ffn(x, off, srt, ex, 1),
                 lambda: m.moe_expert_ffn_mxfp4(x, off, srt, ex, 1), lambda: m.moe_forward(x, x[:2], None, ex, 1),
                 lambda: m.moe_expert_down(x[:, :128].contiguous(), off, ex, 4, 1),
                 lambda: m.moe_block_forward(x, x[:2], None, ex, 1, pre_weight=x[0])):
        with pytest.raises(ValueError, match="columns"):
            call()
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_quantize_mxfp4(torch.zeros(64, 64, device="cuda").t())
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm_mxfp4(*m.moe_quantize_mxfp4(x), off, ex.q_gate, ex.s_gate, torch.float32)


def test_two_schedules_agree_and_repeat():
    """Each schedule gives the same bits again, on another stream too."""
    rng = np.random.default_rng(11)
    S, off, slots = _slots_for([40, 0, 70, 18], 0, rng)
    mats = [draw_mx(rng, 4, r, c) for r, c in ((640, 384), (640, 384), (384, 640))]
    ex = m.pack_mxfp4_experts(*(dev(q) for q, _ in mats), *(dev(s) for _, s in mats))
    x = bf16_exact(rng.standard_normal((S // 2, 384))).cuda()
    doff, dslots = dev(off), dev(slots)
    for path in PATHS:
        a = m.moe_expert_ffn(x, doff, dslots, ex, 2, path=path)
        b = m.moe_expert_ffn_mxfp4(x, doff, dslots, ex, 2, path=path)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            a2 = m.moe_expert_ffn(x, doff, dslots, ex, 2, path=path)
            b2 = m.moe_expert_ffn_mxfp4(x, doff, dslots, ex, 2, path=path)
        side.synchronize()
        assert torch.equal(a, a2) and torch.equal(b, b2)


@pytest.mark.parametrize("path", PATHS)
def test_expert_ffn_mxfp4_is_its_four_steps(path):
    """Quantize, product with SwiGLU, quantize, product: bit for bit."""
    rng = np.random.default_rng(12)
    S, off, slots = _slots_for([31, 0, 5, 130], 2, rng)
    mats = [draw_mx(rng, 4, r, c) for r, c in ((512, 256), (512, 256), (256, 512))]
    ex = m.pack_mxfp4_experts(*(dev(q) for q, _ in mats), *(dev(s) for _, s in mats))
    doff, dslots = dev(off), dev(slots)
    last = int(off[-1])
    for dt in (torch.bfloat16, torch.float32):
        x = torch.from_numpy(rng.standard_normal((S // 2, 256))).to(dt).cuda()
        y = m.moe_expert_ffn_mxfp4(x, doff, dslots, ex, 2, path=path)
        xq, xs = m.moe_quantize_mxfp4(x)
        h = m.moe_grouped_mm_mxfp4(xq, xs, doff, ex.q_gate, ex.s_gate, torch.bfloat16, sorted_slots=dslots, K=2,
                                   w2_q=ex.q_up, w2_s=ex.s_up, path=path)
        hq, hs = m.moe_quantize_mxfp4(h)
        y2 = m.moe_grouped_mm_mxfp4(hq, hs, doff, ex.q_down, ex.s_down, torch.float32, path=path)
        assert torch.equal(y[:last], y2[:last])


# ------------------------------------------------------------------ the layer

def _layer(T, d, f, E, seed, dt=torch.bfloat16):
    rng = np.random.default_rng(seed)
    w = [torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.05).to(torch.bfloat16)
         for s in ((E, f, d), (E, f, d), (E, d, f))]
    x = torch.from_numpy(rng.standard_normal((T, d))).to(dt)
    wr = torch.from_numpy(rng.standard_normal((E, d)) * 0.05).to(dt)
    return w, x, wr


@pytest.mark.parametrize("T,path", [(1, MOE_PATH_AUTO), (23, MOE_PATH_AUTO), (23, MOE_PATH_TILED), (700, MOE_PATH_AUTO)])
def test_forward_with_mxfp4_weights(T, path):
    """The layer against fp64 on the decoded weights, at the layer's tolerance, and against its own stages."""
    d, f, E, K = 256, 384, 8, 2
    w, x, wr = _layer(T, d, f, E, T)
    ex = m.quantize_experts_mxfp4(*(t.cuda() for t in w))
    W = {}
    for k, t in zip(("gate", "up", "down"), w):
        q, s = omx.quantize(np64(t))
        W["q_" + k], W["s_" + k] = omx.dequantize(q, s), np.ones(t.shape[:2])
    y, ids, gw = m.moe_forward(x.cuda(), wr.cuda(), None, ex, K, path=path)
    ref = omoe.moe_forward(np64(x), np64(wr), None, W, K, ids=ids.cpu().numpy())["y"]
    tol = 1e-2 * np.abs(ref).max() + 1e-3
    assert np.abs(np64(y) - ref).max() <= tol
    off, srt, s2r = m.moe_permute(ids, E)
    rows = m.moe_expert_ffn(x.cuda(), off, srt, ex, K, path=path)
    assert torch.equal(m.moe_combine(rows, s2r, gw, torch.bfloat16), y)
    if T <= 23:
        y3, _, _ = m.moe_forward_noalloc(x.cuda(), wr.cuda(), None, ex, K, path=path)
        assert torch.equal(y3, y)


@pytest.mark.parametrize("T", [1, 40, 65, 300])
def test_dense_mlp_with_mxfp4_weights(T):
    w, x, _ = _layer(T, 384, 512, 1, T + 1)
    ex = m.quantize_experts_mxfp4(*(t.cuda() for t in w))
    y = m.moe_mlp_forward(x.cuda(), ex)
    W = [omx.dequantize(*omx.quantize(np64(t[0]))) for t in w]
    X = np64(x)
    g = X @ W[0].T
    ref = (g / (1 + np.exp(-g)) * (X @ W[1].T)) @ W[2].T
    assert np.abs(np64(y) - ref).max() <= 1e-2 * np.abs(ref).max() + 1e-3


@pytest.mark.parametrize("fmt", ["mxfp4", "int8"])
@pytest.mark.parametrize("T", [1, 19, 400])
def test_block_forward_is_its_parts(T, fmt):
    """Norm, layer stages and combine_post in one call: the parts' bits; and `next` feeds the block after it."""
    d, f, E, K = 256, 384, 8, 2
    w, res, wr = _layer(T, d, f, E, T + 2)
    dw = [t.cuda() for t in w]
    ex = m.quantize_experts_mxfp4(*dw) if fmt == "mxfp4" else m.quantize_experts(*dw, torch.bfloat16)
    rng = np.random.default_rng(1)
    pre, wt, nw = (torch.from_numpy(1 + 0.1 * rng.standard_normal(d)).to(torch.bfloat16).cuda() for _ in range(3))
    gate = torch.from_numpy(rng.uniform(0, 1, (-(-T // 3), d))).to(torch.bfloat16).cuda()
    res, wr = res.cuda(), wr.cuda()
    kw = dict(weight=wt, gate=gate, gate_tokens=3, residual_scale=0.9, block_scale=0.5, next_weight=nw, next_eps=1e-5)
    keep = res.clone()
    out, nxt, ids, gw = m.moe_block_forward(res, wr, None, ex, K, pre_weight=pre, **kw)
    assert torch.equal(res, keep)
    n = m.moe_norm_pre(res, pre)
    i2, g2 = m.moe_route(n, wr, None, K)
    off, srt, s2r = m.moe_permute(i2, E)
    rows = m.moe_expert_ffn(n, off, srt, ex, K)
    out2, nxt2 = m.moe_combine_post(rows, s2r, g2, res, **kw)
    assert torch.equal(ids, i2) and torch.equal(gw, g2) and torch.equal(out, out2) and torch.equal(nxt, nxt2)
    # a second block, from the first one's next, onto the stream in place
    o2, _, _, _ = m.moe_block_forward(out, wr, None, ex, K, x=nxt, weight=wt)
    stream = out.clone()
    o3, _, _, _ = m.moe_block_forward(stream, wr, None, ex, K, x=nxt, weight=wt, out=stream)
    assert o3.data_ptr() == stream.data_ptr() and torch.equal(o2, o3)


@pytest.mark.parametrize("T", [3, 300])
def test_captured_block_replays(T):
    """A captured block with its own workspace, replayed with eager work between the replays."""
    d, f, E, K = 256, 384, 8, 2
    w, res, wr = _layer(T, d, f, E, 9)
    ex = m.quantize_experts_mxfp4(*(t.cuda() for t in w))
    pre = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    wr, stat = wr.cuda(), res.cuda()
    shape = ops.make_shape(T, d, f, E, K, torch.bfloat16, ex.scale_dtype, MOE_PATH_AUTO, MOE_W_MXFP4)
    ws = torch.empty(ops.block_workspace_size(shape), dtype=torch.uint8, device="cuda")
    run = lambda r, ws_: m.moe_block_forward(r, wr, None, ex, K, pre_weight=pre, weight=pre, next_weight=pre,
                                             workspace=ws_)
    run(stat, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, nxt, ids, gw = run(stat, ws)
        y = m.moe_expert_ffn_mxfp4(nxt, *m.moe_permute(ids, E)[:2], ex, K)
    for i in range(4):
        new = torch.randn(T, d, dtype=torch.bfloat16, device="cuda")
        stat.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        eo, en, ei, ew = run(new, None)
        ey = m.moe_expert_ffn_mxfp4(en, *m.moe_permute(ei, E)[:2], ex, K)
        torch.cuda.synchronize()
        assert torch.equal(out, eo) and torch.equal(nxt, en) and torch.equal(ids, ei) and torch.equal(y, ey), i


def test_empty_batch():
    ex = m.quantize_experts_mxfp4(*(torch.randn(2, 128, 128, device="cuda") for _ in range(3)))
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert m.moe_expert_gate_up(x, off, none, ex, 2).shape == (0, 128)
    assert m.moe_expert_ffn_mxfp4(x, off, none, ex, 2).shape == (0, 128)
    q, s = m.moe_quantize_mxfp4(x)
    assert m.moe_grouped_mm_mxfp4(q, s, off, ex.q_gate, ex.s_gate, torch.float32).shape == (0, 128)


def test_debug_checks_refuse_bad_segments(monkeypatch):
    monkeypatch.setenv("MOE_DEBUG", "1")
    ex = m.quantize_experts_mxfp4(*(torch.randn(2, 128, 128, device="cuda") for _ in range(3)))
    q, s = m.moe_quantize_mxfp4(torch.randn(4, 128, device="cuda"))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    for off, srt in ((i32(0, 2, 5), i32(0, 1, 2, 3)), (i32(0, 3, 2), i32(0, 1, 2, 3)), (i32(0, 2, 4), i32(0, 1, 2, 4))):
        with pytest.raises(m.MoeError) as e:
            m.moe_grouped_mm_mxfp4(q, s, off, ex.q_gate, ex.s_gate, torch.float32, sorted_slots=srt)
        assert e.value.status == 8
        with pytest.raises(m.MoeError) as e:
            m.moe_expert_ffn_mxfp4(torch.randn(4, 128, device="cuda"), off, srt, ex, 1)
        assert e.value.status == 8
