"""Products of int8 rows and int8 matrices on the GPU against the fp64 oracle.

The integer sum is exact; becoming fp32 and taking two scales are three roundings:
a plain result is off by at most 3 u of its magnitude (u = 2^-24). SwiGLU: p0 and
p1 are each off by 3 u; |silu'| <= 1.1; the exponential is good to 2 units in the
last place (4 u), 1 + it, the division and the two products add one rounding each
(some of them halves): at most 12 u of the result besides the two terms of p0 and
p1. For a bf16 result the exponential is the hardware's: its argument, scaled, is off
by 2^-23 |p0|, it and the reciprocal by some 2^-22 each, at most (8 + |p0|) * 2^-22 of
the result in all; and half a step, 2^-8 of the value.
"""
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from oracle import int8 as oint8
from tests.helpers import np64
from tests.mx_helpers import segments

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PATHS = [MOE_PATH_STREAM, MOE_PATH_TILED]
U = 2.0 ** -24


def _say(msg):
    print(f"[int8-test] {msg}", file=sys.stderr, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _draw(rng, rows, E, f, d, scale, sigma=40.0, extreme=False):
    def codes(*shape):
        if extreme:
            return rng.choice(np.array([-128, -127, 127], np.int8), shape)
        return np.clip(np.rint(rng.standard_normal(shape) * sigma), -127, 127).astype(np.int8)
    a_q, a_s = codes(rows, d), (rng.random(rows) * 0.05 + 1e-3).astype(np.float32)
    ws = [(codes(E, f, d), torch.from_numpy((rng.random((E, f)) * 2e-3 / np.sqrt(d)).astype(np.float32)).to(DT[scale]))
          for _ in range(2)]
    return a_q, a_s, ws


def _bound(a_q, a_s, ws, off, rows, swiglu, out):
    n64 = [np64(s) for _, s in ws]
    p0 = oint8.grouped_product(a_q, a_s, ws[0][0], n64[0], off, rows)
    if not swiglu:
        ref, bound = p0, 3.01 * U * np.abs(p0)
    else:
        ref = oint8.grouped_product(a_q, a_s, ws[0][0], n64[0], off, rows, ws[1][0], n64[1])
        p1 = oint8.grouped_product(a_q, a_s, ws[1][0], n64[1], off, rows)
        bound = 1.1 * 3.01 * U * np.abs(p0 * p1) + 15 * U * np.abs(ref)
    if out == "bf16":
        if swiglu:
            bound = bound + (8 + np.abs(p0)) * 2.0 ** -22 * np.abs(ref)
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    return ref, bound + 1e-37


def _run(counts, S, K, d, f, swiglu, out, scale, path, gather, seed, extreme=False):
    rng = np.random.default_rng(seed)
    E = len(counts)
    _say(f"E={E} S={S} K={K} d={d} f={f} swiglu={swiglu} out={out} scale={scale} path={path} gather={gather}")
    off, slots = segments(counts, S, rng)
    n_rows = S // K if gather else S
    rows = np.maximum(slots, 0) // K if gather else np.arange(S)
    a_q, a_s, ws = _draw(rng, n_rows, E, f, d, scale, extreme=extreme)
    packed = [m.moe_pack_rows(dev(q)) for q, _ in ws]
    dst = torch.full((S, f), 7.0, dtype=DT[out], device="cuda")
    got = m.moe_grouped_mm_int8(dev(a_q), dev(a_s), dev(off), packed[0], ws[0][1].cuda(), DT[out],
                                sorted_slots=dev(slots) if gather else None, K=K if gather else 1,
                                w2_q=packed[1] if swiglu else None, w2_s=ws[1][1].cuda() if swiglu else None, path=path,
                                out=dst)
    assert got is dst
    ref, bound = _bound(a_q, a_s, ws, off, rows, swiglu, out)
    last = off[-1]
    err = np.abs(np64(got)[:last] - ref[:last])
    assert (err <= bound[:last]).all(), f"worst {np.max(err / bound[:last]):.3g} of the bound"
    assert (got[last:] == 7.0).all(), "rows past the last segment"
    return got


# (counts, S, K): empty experts, one row, whole and partial row blocks and tiles, rows past the last segment
SEGMENTS = [([1], 1, 1), ([0, 3, 0, 5], 8, 2), ([16, 17, 0, 1], 36, 2), ([33, 0, 64, 2, 30], 130, 2), ([70, 130], 201, 3),
            ([129, 300, 3], 432, 4)]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,S,K", SEGMENTS)
@pytest.mark.parametrize("d,f,scale,out", [(64, 64, "f32", "f32"), (128, 192, "bf16", "bf16"), (448, 704, "f32", "bf16"),
                                           (1024, 320, "bf16", "f32")])
def test_products(counts, S, K, d, f, scale, out, swiglu, path):
    _run(counts, S, K, d, f, swiglu, out, scale, path, True, S + d)
    _run(counts, S, 1, d, f, swiglu, out, scale, path, False, S + d + 1)


@pytest.mark.parametrize("path", PATHS + [MOE_PATH_AUTO])
@pytest.mark.parametrize("d,f", [(4096, 256), (8192, 128), (64, 4160)])
@pytest.mark.parametrize("counts", [[1, 0, 0, 1], [40, 5, 0, 20], [200, 10, 300, 130]])
def test_long_and_wide(counts, d, f, path):
    _run(counts, sum(counts), 1, d, f, False, "f32", "f32", path, False, d + f)
    _run(counts, sum(counts), 1, d, f, True, "bf16", "bf16", path, False, d + f)


# what is taken: (mean rows an expert, E, f, path, the log's words); f / 32 * E items of 32 channels: 2048 is the border
INSTANCES = [(4, 16, 4160, MOE_PATH_AUTO, "16-channel items, 16-row passes, reduction in 4 slices"),
             (5, 16, 4160, MOE_PATH_AUTO, "32-channel items, 32-row passes, reduction in 2 slices"),
             (8, 16, 4160, MOE_PATH_AUTO, "32-channel items, 32-row passes, reduction in 2 slices"),
             (8, 16, 4032, MOE_PATH_AUTO, "16-channel items, 16-row passes, reduction in 4 slices"),
             (9, 16, 4160, MOE_PATH_STREAM, "32-channel items, 64-row passes, reduction in 4 slices"),
             (9, 16, 4160, MOE_PATH_AUTO, "tiled schedule, 128x"),
             (64, 1, 1024, MOE_PATH_AUTO, "32-channel items, 64-row passes, reduction in 4 slices"),
             (65, 1, 1024, MOE_PATH_AUTO, "32-channel items, 64-row passes, reduction in 4 slices"),
             (512, 1, 1024, MOE_PATH_AUTO, "32-channel items, 64-row passes, reduction in 4 slices"),
             (513, 1, 1024, MOE_PATH_AUTO, "tiled schedule, 128x128 tiles"),
             (1700, 1, 64, MOE_PATH_AUTO, "32-channel items, 64-row passes, reduction in 4 slices"),
             (128, 4, 1024, MOE_PATH_AUTO, "32-channel items, 64-row passes, reduction in 4 slices"),
             (129, 4, 1024, MOE_PATH_AUTO, "tiled schedule, 128x128 tiles"),
             (64, 16, 8320, MOE_PATH_AUTO, "tiled schedule, 128x"), (65, 16, 8320, MOE_PATH_AUTO, "tiled schedule, 128x256 tiles"),
             (40, 4, 512, MOE_PATH_TILED, "tiled schedule, 128x128 tiles")]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("rows,E,f,path,words", INSTANCES)
def test_every_instance_and_border(rows, E, f, path, words, out, swiglu, monkeypatch, capfd):
    rng = np.random.default_rng(rows * 31 + E)
    counts = rng.multinomial(rows * E, np.ones(E) / E).tolist()
    monkeypatch.setenv("MOE_LOG", "1")
    _run(counts, rows * E, 1, 192, f, swiglu, out, "bf16", path, True, rows + f)
    line = [l for l in capfd.readouterr().err.splitlines() if "moe_grouped_mm_int8" in l]
    assert len(line) == 1 and words in line[0], line


@pytest.mark.parametrize("path", PATHS)
def test_largest_sums(path):
    """Codes of -128, -127 and 127 only, over the longest reduction: sums up to 2^30."""
    _run([3, 20], 23, 1, 65536, 64, False, "f32", "f32", path, False, 5, extreme=True)


@pytest.mark.parametrize("swiglu", [False, True])
def test_schedules_agree_bit_for_bit(swiglu):
    for counts, d, f in (([3, 0, 7], 320, 192), ([150, 20, 90], 640, 576)):
        a = _run(counts, sum(counts), 1, d, f, swiglu, "f32", "bf16", MOE_PATH_STREAM, False, 11)
        b = _run(counts, sum(counts), 1, d, f, swiglu, "f32", "bf16", MOE_PATH_TILED, False, 11)
        assert torch.equal(a, b)


def test_quantized_tokens_and_graph():
    """As it is used: tokens quantized by the library's quantizer, weights by the layer's, replayed from a graph."""
    rng = np.random.default_rng(12)
    T, d, f, E, K = 40, 512, 384, 8, 2
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(torch.bfloat16).cuda()
    w = torch.from_numpy((0.02 * rng.standard_normal((E, f, d))).astype(np.float32)).to(torch.bfloat16).cuda()
    q, s = m.moe_quantize_pack_rows(w, torch.bfloat16)
    ids, _ = m.moe_route_gated(x, w[:, 0].contiguous(), None, K, m.Gate())
    off, slots, _ = m.moe_permute(ids, E)
    a_q, a_s = m.moe_quantize_rows(x, torch.float32)
    want = m.moe_grouped_mm_int8(a_q, a_s, off, q, s, torch.float32, sorted_slots=slots, K=K)
    rows = slots.cpu().numpy() // K
    ref = np.concatenate([np64(x)[rows[a:b]] @ np64(w)[e].T
                          for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    # a code is off by at most half its row's step: |sum| <= sum |x| ws/2 + sum |w| as/2 + d ws as/4
    srow = np.concatenate([np.tile(np64(s)[e], (b - a, 1)) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    wabs = np.concatenate([np.tile(np.abs(np64(w)[e]).sum(1), (b - a, 1))
                           for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    xs = np64(a_s)[rows][:, None]
    # the channel's scale is rounded to bf16: half a step, 2^-9 of 127 codes, moves a clamped or scaled code too
    bound = (np.abs(np64(x)[rows]).sum(1)[:, None] * srow * 1.01 + wabs * xs / 2 + d * srow * xs)
    assert (np.abs(np64(want) - ref) <= bound).all()
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    src = x.clone()
    with torch.cuda.graph(graph):
        gi, _ = m.moe_route_gated(src, w[:, 0].contiguous(), None, K, m.Gate())
        go, gs, _ = m.moe_permute(gi, E)
        gq, gsc = m.moe_quantize_rows(src, torch.float32)
        m.moe_grouped_mm_int8(gq, gsc, go, q, s, torch.float32, sorted_slots=gs, K=K, out=out)
    for i in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_empty_and_refused():
    z = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt, device="cuda")
    w, s, off = z(2, 64, 128), z(2, 64, dt=torch.float32), z(3, dt=torch.int32)
    assert m.moe_grouped_mm_int8(z(0, 128), z(0, dt=torch.float32), off, w, s, torch.float32).shape == (0, 64)
    a, sc = z(4, 128), z(4, dt=torch.float32)
    out = torch.full((4, 64), 3.0, device="cuda")
    m.moe_grouped_mm_int8(a, sc, off, w, s, torch.float32, out=out)      # every segment empty
    assert (out == 3).all()
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm_int8(a, sc[:3], off, w, s, torch.float32)
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm_int8(a, sc, off[:2], w, s, torch.float32)
    with pytest.raises(TypeError, match="dtype"):
        m.moe_grouped_mm_int8(a, sc.double(), off, w, s, torch.float32)
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm_int8(z(4, 64), sc, off, w, s, torch.float32)
