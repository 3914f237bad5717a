"""MXFP4 calls at the ends of their ranges, on the GPU."""
import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_STREAM, MOE_PATH_TILED
from oracle import mxfp4 as omx
from tests.helpers import np64
from tests.mx_helpers import bf16_exact, check, product_bound, segments

pytestmark = pytest.mark.gpu

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(q, s):
    """fp64 numbers of row-major codes and scale bytes, on their device."""
    grid = torch.tensor([*GRID, *(-v for v in GRID)], dtype=torch.float64, device=q.device)
    v = torch.stack([grid[(q & 15).long()], grid[(q >> 4).long()]], -1).flatten(-2)
    scale = torch.exp2(s.double() - 127)                       # powers of two: exact
    return v * scale.repeat_interleave(32, dim=-1)


def draw(rows, cols, gen, lo=118, hi=124):
    """Random codes, and scales worth 2^-9 .. 2^-4."""
    q = torch.randint(0, 256, (*rows, cols // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s = torch.randint(lo, hi, (*rows, cols // 32), generator=gen, device="cuda", dtype=torch.uint8)
    return q, s


def test_down_rows_past_4_gib():
    """h of 6 GiB: the down pass streams (gate/up, whose x is 8 MiB, stays tiled), rows at both ends of h checked.

    Bound: exact products, fp32 sums of f terms: f * 2^-23 of the sum of magnitudes; and for gate/up that of
    tests/mx_helpers.py with its bf16 rounding.
    """
    T, d, f, E, K = 16384, 256, 24576, 64, 8
    S = T * K
    gen = torch.Generator(device="cuda").manual_seed(1)
    mats = {k: draw((E, r), c, gen) for k, (r, c) in dict(gate=(f, d), up=(f, d), down=(d, f)).items()}
    ex = m.pack_mxfp4_experts(*(mats[k][0] for k in ("gate", "up", "down")), *(mats[k][1] for k in ("gate", "up", "down")))
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (S // E)
    slots = torch.randperm(S, generator=gen, device="cuda").to(torch.int32)
    x = torch.randn(T, d, generator=gen, device="cuda").to(torch.bfloat16)
    h = m.moe_expert_gate_up(x, off, slots, ex, K)
    assert h.numel() * 2 > 1 << 32
    y = m.moe_expert_down(h, off, ex, T, K)
    per = S // E
    for e in (0, 1, E // 2, E - 1):
        W = {k: values(q[e], s[e]) for k, (q, s) in mats.items()}
        for rows in (slice(e * per, e * per + 40), slice((e + 1) * per - 40, (e + 1) * per)):
            a = x[(slots[rows] // K).long()].double()
            g, u = a @ W["gate"].t().contiguous(), a @ W["up"].t().contiguous()
            mg, mu = a.abs() @ W["gate"].abs().t().contiguous(), a.abs() @ W["up"].abs().t().contiguous()
            eps, silu = 2.0 ** -23, g / (1 + torch.exp(-g))
            ref = silu * u
            bound = d * eps * (1.1 * u.abs() * mg + silu.abs() * mu) + (8 + g.abs()) * 2 * eps * ref.abs()
            bound = bound + 2.0 ** -8 * (ref.abs() + bound) + 1e-37
            assert ((h[rows].double() - ref).abs() <= bound).all(), e
            a = h[rows].double()
            ref, mag = a @ W["down"].t().contiguous(), a.abs() @ W["down"].abs().t().contiguous()
            assert ((y[rows].double() - ref).abs() <= f * eps * mag + 1e-37).all(), e


def test_past_4_gib_schedules_in_the_log(monkeypatch, capfd):
    monkeypatch.setenv("MOE_LOG", "1")
    T, d, f, E, K = 16384, 256, 24576, 64, 8
    ex = m.Int8Experts(*(torch.zeros(E, r, c // 2, dtype=torch.uint8, device="cuda") for r, c in ((f, d), (f, d), (d, f))),
                       *(torch.full((E, r, c // 32), 127, dtype=torch.uint8, device="cuda") for r, c in ((f, d), (f, d), (d, f))),
                       fmt=m.MOE_W_MXFP4)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32) * (T * K // E)
    slots = torch.arange(T * K, device="cuda", dtype=torch.int32)
    y = m.moe_expert_ffn(torch.ones(T, d, dtype=torch.bfloat16, device="cuda"), off, slots, ex, K)
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("[moe] moe_expert_ffn")]
    assert "; tiled schedule" in lines[0] and "; stream schedule" in lines[1], lines
    assert (y == 0).all()


def test_norm_outputs_in_place_of_an_input():
    """next may take residual's or y's memory, out the other's: the bits of separate outputs."""
    for dt, d in ((torch.bfloat16, 4096), (torch.float32, 320)):
        g = torch.Generator(device="cuda").manual_seed(d)
        y, res = (torch.randn(70, d, generator=g, device="cuda").to(dt) for _ in range(2))
        w = torch.ones(d, dtype=dt, device="cuda")
        out, nxt = m.moe_norm_post(y, res, weight=w, next_weight=w)
        for swap in (False, True):
            a, b = y.clone(), res.clone()
            o2, n2 = m.moe_norm_post(a, b, weight=w, next_weight=w, out=a if swap else b, next_out=b if swap else a)
            assert torch.equal(o2, out) and torch.equal(n2, nxt)
        with pytest.raises(m.MoeError) as e:
            m.moe_norm_post(y, res, weight=w, next_weight=w, out=out, next_out=out)
        assert e.value.status == 6


# weights' scale bytes, exponent of the activations. Bytes 0 to 2 make weights below bf16's smallest normal number and
# 2^-128 .. 2^-133 such activations; bytes up to 252 are the largest whose every code is a finite bf16 number. The
# other side brings the results back to the normal numbers of fp32, so a flushed operand would be seen.
ENDS = [((0, 0), 100), ((0, 3), 100), ((1, 1), 100), ((2, 2), 100), ((250, 252), -110), ((230, 240), -128),
        ((230, 240), -133)]


@pytest.mark.parametrize("path", [MOE_PATH_STREAM, MOE_PATH_TILED])
@pytest.mark.parametrize("scales,exp", ENDS)
def test_products_at_the_ends_of_the_scales(scales, exp, path):
    """Products stay exact where operands are subnormal or nearly infinite in bf16 (bounds of tests/mx_helpers.py,
    without their absolute term)."""
    counts, d, f, S = [20, 3], 256, 256, 23
    rng = np.random.default_rng(7)
    off, slots = segments(counts, S, rng)
    codes = lambda *shape: (rng.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8))
    mats = [(codes(2, r, c), rng.integers(scales[0], scales[1] + 1, (2, r, c // 32)).astype(np.uint8))
            for r, c in ((f, d), (f, d), (d, f))]
    dev = lambda a: torch.from_numpy(a).cuda()
    ex = m.pack_mxfp4_experts(*(dev(q) for q, _ in mats), *(dev(s) for _, s in mats))
    W = [omx.dequantize(*v) for v in mats]
    h = bf16_exact(np.ldexp(rng.standard_normal((S, f)), exp))
    y = m.moe_expert_down(h.cuda(), dev(off), ex, S, 1, path=path)
    ref, bound = product_bound(np64(h), W[2], off, np.arange(S))
    check(y, ref, bound - 1e-37, S, "down")
    # 4-bit activations of the same magnitude
    aq, byte = codes(S, d), max(0, 127 + exp - 2)
    asc = np.full((S, d // 32), byte, dtype=np.uint8)
    out = m.moe_grouped_mm_mxfp4(dev(aq), dev(asc), dev(off), *m.moe_pack_mxfp4(dev(mats[0][0]), dev(mats[0][1])),
                                 torch.float32, path=path)
    ref, bound = product_bound(omx.dequantize(aq, asc), W[0], off, np.arange(S))
    check(out, ref, bound - 1e-37, S, "product")


@pytest.mark.parametrize("path", [MOE_PATH_STREAM, MOE_PATH_TILED])
def test_weights_past_bf16(path):
    """A weight of 2^128 and more is infinite next to bf16 activations, and exact next to 4-bit ones."""
    w_q = torch.zeros(1, 128, 64, dtype=torch.uint8, device="cuda")
    w_s = torch.full((1, 128, 4), 127, dtype=torch.uint8, device="cuda")
    w_q[0, :, 0] = torch.tensor([1, 3, 5, 6, 7, 14, 15, 0], dtype=torch.uint8, device="cuda").repeat(16)
    w_s[0, :, 0] = 253                                               # 2^126 times the code's number
    grid = torch.tensor([0.5, 1.5, 3, 4, 6, -4, -6, 0], dtype=torch.float64).repeat(16) * 2.0 ** 126
    wt = m.moe_pack_mxfp4(w_q, w_s)
    ex = m.Int8Experts(wt[0], wt[0], wt[0], wt[1], wt[1], wt[1], fmt=m.MOE_W_MXFP4)
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    h = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = torch.tensor([2.0 ** -100, 2.0 ** -20], device="cuda")
    y = m.moe_expert_down(h, off, ex, 2, 1, path=path).cpu().double()
    want = torch.where(grid.abs() >= 2.0 ** 128, torch.copysign(torch.tensor(torch.inf, dtype=torch.float64), grid), grid)
    assert torch.equal(y, h[:, :1].cpu().double() * want)
    a_q = torch.zeros(2, 64, dtype=torch.uint8, device="cuda")
    a_q[:, 0] = 2                                                    # one
    a_s = torch.tensor([[27, 127, 127, 127], [107, 127, 127, 127]], dtype=torch.uint8, device="cuda")
    out = m.moe_grouped_mm_mxfp4(a_q, a_s, off, *wt, torch.float32, path=path).cpu().double()
    assert torch.equal(out, h[:, :1].cpu().double() * grid)


@pytest.mark.parametrize("fmt", ["int8", "mxfp4"])
def test_down_of_a_flat_h(fmt):
    w = [torch.randn(2, r, c, device="cuda").to(torch.bfloat16) for r, c in ((256, 128), (256, 128), (128, 256))]
    ex = m.quantize_experts_mxfp4(*w) if fmt == "mxfp4" else m.quantize_experts(*w, torch.bfloat16)
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    h = torch.randn(8, 256, device="cuda").to(torch.bfloat16)
    y = m.moe_expert_down(h, off, ex, 4, 2)
    for form in (h.view(-1), h.view(4, 2, 256), h.view(16, 128), torch.cat([h, h])):
        assert torch.equal(m.moe_expert_down(form, off, ex, 4, 2), y)


@pytest.mark.parametrize("path", [MOE_PATH_STREAM, MOE_PATH_TILED])
@pytest.mark.parametrize("counts,T,K", [([9], 6, 4), ([20, 33], 40, 8), ([0, 1], 1, 8)])
def test_product_of_a_shard(counts, T, K, path):
    """Fewer experts than slots a token: the slots of experts elsewhere lie past the last segment."""
    rng = np.random.default_rng(T * K)
    S, d, f, E = T * K, 384, 256, len(counts)
    off, slots = segments(counts, S, rng)
    codes = lambda *shape: rng.integers(0, 256, (*shape[:-1], shape[-1] // 2)).astype(np.uint8)
    scales = lambda *shape: rng.integers(118, 124, (*shape[:-1], shape[-1] // 32)).astype(np.uint8)
    a, w = (codes(T, d), scales(T, d)), (codes(E, f, d), scales(E, f, d))
    dev = lambda t: torch.from_numpy(t).cuda()
    out = m.moe_grouped_mm_mxfp4(dev(a[0]), dev(a[1]), dev(off), *m.moe_pack_mxfp4(dev(w[0]), dev(w[1])), torch.float32,
                                 sorted_slots=dev(slots), K=K, path=path, out=torch.full((S, f), 7.0, device="cuda"))
    ref, bound = product_bound(omx.dequantize(*a), omx.dequantize(*w), off, slots // K)
    check(out, ref, bound, int(off[-1]), "product")
    assert (out[int(off[-1]):] == 7.0).all()


# ------------------------------------------------------------------ far rows: the same bits as on their own

def _halves(n, k=64):
    return slice(0, k), slice(n // 2, n // 2 + k), slice(n - k, n)


@pytest.mark.parametrize("rows", [50000, 100000, 140000])
def test_far_rows_of_codes(rows):
    """Codes of 1.5, 3.1 and 4.3 GiB (past 2^31 bytes; past 2^32 the streaming kernel takes them on every schedule):
    exact sums, so every row gives what it gives on its own, on either schedule."""
    d, f = 65536, 128
    gen = torch.Generator(device="cuda").manual_seed(rows)
    a_q, a_s = draw((rows,), d, gen, 120, 122)
    # one element in 64 of a weight row is not zero: at most 1024 products of halves and steps of 2, exact in fp32
    w_q, w_s = draw((1, f), d, gen, 120, 121)
    w_q = torch.where(torch.arange(d // 2, device="cuda") % 32 == 5, w_q & 15, 0).to(torch.uint8)
    wt = m.moe_pack_mxfp4(w_q, w_s)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    out = m.moe_grouped_mm_mxfp4(a_q, a_s, off, *wt, torch.float32, path=MOE_PATH_TILED)
    for r in _halves(rows):
        ref = (values(a_q[r], a_s[r]) @ values(w_q[0], w_s[0]).t().contiguous()).float()
        assert torch.equal(out[r], ref)


def test_far_rows_of_h_on_the_tiled_schedule():
    """h of 3 GiB: byte offsets past 2^31 in the tiled kernel."""
    S, f, d, E = 65536, 24576, 128, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, s = draw((E, d), f, gen)
    wt = m.moe_pack_mxfp4(q, s)
    gate = torch.empty(1, dtype=torch.uint8, device="cuda").expand(E, f, d // 2)
    ex = m.Int8Experts(gate, gate, wt[0], gate, gate, wt[1], fmt=m.MOE_W_MXFP4)
    h = torch.randn(S, f, generator=gen, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 1000, S], dtype=torch.int32, device="cuda")
    y = m.moe_expert_down(h, off, ex, S, 1, path=MOE_PATH_TILED)
    for r in (slice(0, 64), slice(1000, 1064), slice(S - 64, S)):
        a, w = h[r].double(), values(q[0 if r.start == 0 else 1], s[0 if r.start == 0 else 1]).t().contiguous()
        assert ((y[r].double() - a @ w).abs() <= f * 2.0 ** -23 * (a.abs() @ w.abs())).all()


def test_far_rows_of_the_quantizer():
    """2^33 numbers and some more in one call (two launches), both ways; and tiled rows past 2^32 numbers."""
    cols, rows = 1024, (1 << 23) + 100
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in (*_halves(rows), slice((1 << 23) - 32, (1 << 23) + 32)):
        w[r] = torch.randn(64, cols, device="cuda").to(torch.bfloat16)
    q, s = m.moe_quantize_mxfp4(w)
    back = m.moe_dequantize_mxfp4(q, s, torch.bfloat16)
    for r in (*_halves(rows), slice((1 << 23) - 32, (1 << 23) + 32)):
        q1, s1 = m.moe_quantize_mxfp4(w[r])
        assert torch.equal(q[r], q1) and torch.equal(s[r], s1)
        assert torch.equal(back[r], m.moe_dequantize_mxfp4(q1, s1, torch.bfloat16)) and back[r].any()
    del w, q, s, back
    cols, rows = 8192, 16 * 40000
    w = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    for r in _halves(rows):
        w[r] = torch.randn(64, cols, device="cuda").to(torch.bfloat16)
    q, s = m.moe_quantize_mxfp4(w, tiled=True)
    back = m.moe_dequantize_mxfp4(q, s, torch.bfloat16, tiled=True)
    rq, rs = m.moe_quantize_mxfp4(w)
    pq, ps = m.moe_pack_mxfp4(rq, rs)
    assert torch.equal(q, pq) and torch.equal(s, ps)
    for r in _halves(rows):
        q1, s1 = m.moe_quantize_mxfp4(w[r], tiled=True)
        assert torch.equal(q[r], q1) and torch.equal(s[r], s1) and q1.any()
        assert torch.equal(back[r], m.moe_dequantize_mxfp4(q1, s1, torch.bfloat16, tiled=True))


def test_far_tokens_of_the_norms():
    """Past 2^31 elements: a token's numbers are those of the same token in a short batch of the same kernel's spread."""
    T, d = 40000, 65536
    y, res = (torch.zeros(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (y, res):
        for r in _halves(T):
            t[r] = torch.randn(64, d, device="cuda").to(torch.bfloat16)
    w = torch.ones(d, dtype=torch.bfloat16, device="cuda")
    n = m.moe_norm_pre(y, w)
    out, nxt = m.moe_norm_post(y, res, weight=w, next_weight=w)
    for r in _halves(T):
        assert torch.equal(n[r], m.moe_norm_pre(y[r], w)) and n[r].any()
        o1, n1 = m.moe_norm_post(y[r], res[r], weight=w, next_weight=w)
        assert torch.equal(out[r], o1) and torch.equal(nxt[r], n1)
