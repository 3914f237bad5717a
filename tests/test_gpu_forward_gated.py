"""The layer and the block with gated routing and int8 activations: composed bit for bit from their staged calls, and each
stage against the fp64 oracle on what the stage before it gave."""
import os
import sys

import numpy as np
import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd._lib import MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED
from oracle import gate as ogate
from oracle import int8 as oint8
from oracle import moe as omoe
from oracle import quant as oquant
from tests.helpers import np64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _say(msg):
    print(f"[gated-test] {msg}", file=sys.stderr, flush=True)


def _case(T, d, f, E, act="bf16", scale=torch.bfloat16, fmt="int8", seed=0, disabled=0):
    rng = np.random.default_rng(seed + T + d + E)
    n = lambda *s, k=1.0: torch.from_numpy((k * rng.standard_normal(s)).astype(np.float32))
    x, wr = n(T, d).to(DT[act]).cuda(), n(E, d, k=0.05).to(DT[act]).cuda()
    w = [n(E, f, d, k=0.02).to(torch.bfloat16).cuda(), n(E, f, d, k=0.02).to(torch.bfloat16).cuda(),
         n(E, d, f, k=0.02).to(torch.bfloat16).cuda()]
    make = {"int8": lambda: m.quantize_experts(*w, scale), "fp8": lambda: m.quantize_experts_fp8(*w, scale),
            "bf16": lambda: m.pack_bf16_experts(*w), "mxfp4": lambda: m.quantize_experts_mxfp4(*w)}[fmt]
    b = (0.05 * rng.standard_normal(E)).astype(np.float32)
    if disabled:
        b[rng.permutation(E)[:disabled]] = -np.inf
    return x, wr, make(), torch.from_numpy(b).cuda(), w


def _staged(x, wr, bias, ex, K, gate, act_int8, path):
    ids, w = m.moe_route_gated(x, wr, bias, K, gate)
    off, slots, s2r = m.moe_permute(ids, ex.E)
    rows = (m.moe_expert_ffn_int8 if act_int8 else m.moe_expert_ffn)(x, off, slots, ex, K, path=path)
    return m.moe_combine(rows, s2r, w, x.dtype), ids, w, rows, s2r, off, slots


GATES = [dict(score=m.MOE_SCORE_SIGMOID, groups=4, group_topk=2, group_by=m.MOE_GROUP_TOP2, scale=2.5),
         dict(score=m.MOE_SCORE_SOFTMAX, renorm=False)]


@pytest.mark.parametrize("T,d,f,E,K", [(1, 128, 192, 8, 2), (7, 256, 128, 8, 3), (40, 192, 320, 16, 2), (300, 128, 192, 8, 4),
                                       (900, 256, 256, 8, 2)])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("path", [MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED])
def test_layer_is_its_staged_calls(T, d, f, E, K, gate, path):
    for fmt, act, act_int8 in (("int8", "bf16", True), ("int8", "f32", True), ("int8", "bf16", False), ("fp8", "bf16", False),
                               ("bf16", "bf16", False), ("mxfp4", "bf16", False)):
        if fmt == "mxfp4" and (d % 128 or f % 128):
            continue
        for disabled in (0, E - K + 1):       # the second leaves ids of -1
            _say(f"T={T} d={d} f={f} E={E} K={K} {fmt} {act} int8={act_int8} path={path} disabled={disabled}")
            x, wr, ex, b, _ = _case(T, d, f, E, act, fmt=fmt, disabled=disabled)
            g = m.Gate(select_bias=b, **gate)
            y, ids, w = m.moe_forward_gated(x, wr, None, ex, K, g, act_int8, path=path)
            ry, rid, rw = _staged(x, wr, None, ex, K, g, act_int8, path)[:3]
            assert torch.equal(ids, rid) and torch.equal(w, rw)
            assert torch.equal(y, ry)
            assert ((ids == -1).any() == (disabled > 0)) and torch.isfinite(y).all()


@pytest.mark.parametrize("act_int8", [False, True])
def test_block_is_its_staged_calls(act_int8):
    for T in (1, 33, 400):
        x, wr, ex, b, _ = _case(T, 256, 192, 8)
        d = 256
        rng = np.random.default_rng(T)
        v = [torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in range(4)]
        g = m.Gate(select_bias=b, score=m.MOE_SCORE_SIGMOID, scale=1.5)
        bias = b * 0.5
        fg = torch.sigmoid(v[3]).unsqueeze(0)
        kw = dict(weight=v[1], gate=fg, gate_tokens=T, residual_scale=0.9, block_scale=0.5, next_weight=v[2])
        out, nxt, ids, w = m.moe_block_forward_gated(x, wr, bias, ex, 2, g, act_int8, pre_weight=v[0], **kw)
        n = m.moe_norm_pre(x, v[0])
        _, rid, rw, rows, s2r, _, _ = _staged(n, wr, bias, ex, 2, g, act_int8, MOE_PATH_AUTO)
        ro, rn = m.moe_combine_post(rows, s2r, rw, x, **kw)
        assert torch.equal(ids, rid) and torch.equal(w, rw) and torch.equal(out, ro) and torch.equal(nxt, rn)
        # the next block, whose input is `next`, onto the stream itself
        stream = out.clone()
        o2, _, _, _ = m.moe_block_forward_gated(stream, wr, bias, ex, 2, g, act_int8, x=nxt, weight=v[1], out=stream)
        _, _, rw, rows, s2r, _, _ = _staged(nxt, wr, bias, ex, 2, g, act_int8, MOE_PATH_AUTO)
        r2, _ = m.moe_combine_post(rows, s2r, rw, out, weight=v[1])
        assert o2 is stream and torch.equal(o2, r2)


def test_blocks_of_long_rows():
    """Rows that gated routing splits over workgroups: the plain block takes the workspace it names, and both are their
    staged calls."""
    x, wr, ex, _, _ = _case(3, 8192, 64, 4)
    v = torch.ones(8192, dtype=torch.bfloat16, device="cuda")
    n = m.moe_norm_pre(x, v)
    for gate in (None, m.Gate()):
        kw = dict(pre_weight=v, weight=v, residual_scale=0.5)
        if gate is None:
            out, _, ids, w = m.moe_block_forward(x, wr, None, ex, 2, **kw)
            rid, rw = m.moe_route(n, wr, None, 2)
        else:
            out, _, ids, w = m.moe_block_forward_gated(x, wr, None, ex, 2, gate, **kw)
            rid, rw = m.moe_route_gated(n, wr, None, 2, gate)
        assert torch.equal(ids, rid) and torch.equal(w, rw)
        off, slots, s2r = m.moe_permute(rid, 4)
        rows = m.moe_expert_ffn(n, off, slots, ex, 2)
        assert torch.equal(out, m.moe_combine_post(rows, s2r, rw, x, weight=v, residual_scale=0.5)[0])


@pytest.mark.parametrize("T,d,f,E,K", [(5, 192, 256, 8, 2), (120, 320, 448, 12, 3)])
def test_each_stage_against_the_oracle(T, d, f, E, K):
    """Routing, permutation, the tokens' codes, gate/up, h's codes, down and combine, as moe_expert_ffn_int8 chains them."""
    u = 2.0 ** -24
    x, wr, ex, b, w = _case(T, d, f, E)
    g = m.Gate(score=m.MOE_SCORE_SIGMOID, select_bias=b, groups=4, group_topk=2, group_by=m.MOE_GROUP_TOP2, scale=2.5)
    y, ids, tw, rows, s2r, off, slots = _staged(x, wr, None, ex, K, g, True, MOE_PATH_AUTO)
    rid, rw, _ = ogate.route(np64(x), np64(wr), None, K, True, select_bias=b.cpu().numpy(), groups=4, group_topk=2, top2=True,
                             scale=2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    ro, rs, r2 = omoe.permute(rid, E)
    assert all(np.array_equal(a.cpu().numpy(), c) for a, c in ((off, ro), (slots, rs), (s2r, r2)))
    codes = [oquant.quantize_rows(np64(t), "bf16") for t in w]
    xq, xs = oquant.quantize_rows(np64(x), "f32")
    gq, gs = m.moe_quantize_rows(x, torch.float32)
    assert np.array_equal(gq.cpu().numpy(), xq) and np.array_equal(np64(gs), xs)
    h = m.moe_grouped_mm_int8(gq, gs, off, ex.q_gate, ex.s_gate, torch.bfloat16, sorted_slots=slots, K=K, w2_q=ex.q_up,
                              w2_s=ex.s_up)
    src = rs // K
    args = (xq, xs, codes[0][0], codes[0][1], ro, src)
    ref = oint8.grouped_product(*args, codes[1][0], codes[1][1])
    p0, p1 = oint8.grouped_product(*args), oint8.grouped_product(xq, xs, codes[1][0], codes[1][1], ro, src)
    # the bounds of the product's own tests
    bound = 1.1 * 3.01 * u * np.abs(p0 * p1) + (15 * u + (8 + np.abs(p0)) * 2.0 ** -22) * np.abs(ref)
    bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 1e-37
    assert (np.abs(np64(h) - ref) <= bound).all()
    hq, hs = oquant.quantize_rows(np64(h), "f32")
    ref = oint8.grouped_product(hq, hs, codes[2][0], codes[2][1], ro, np.arange(T * K))
    assert (np.abs(np64(rows) - ref) <= 3.01 * u * np.abs(ref) + 1e-37).all()
    # combine: K products and sums in fp32, one rounding to bf16
    ref = (np64(tw)[:, :, None] * np64(rows)[r2].reshape(T, K, d)).sum(1)
    mag = (np.abs(np64(tw))[:, :, None] * np.abs(np64(rows))[r2].reshape(T, K, d)).sum(1)
    assert (np.abs(np64(y) - ref) <= 2 * K * u * mag + 2.0 ** -8 * np.abs(ref) * 1.01 + 1e-37).all()


def test_layer_object_graph_streams_and_debug(monkeypatch):
    x, wr, ex, b, _ = _case(64, 256, 384, 16)
    g = m.Gate(score=m.MOE_SCORE_SIGMOID, select_bias=b, groups=4, group_topk=2, group_by=m.MOE_GROUP_TOP2)
    layer = m.MoeLayer(wr, None, ex, 2, gate=g, act_int8=True)
    y, ids, w = layer.forward(x)
    ry, rid, rw = m.moe_forward_gated(x, wr, None, ex, 2, g, True)
    assert torch.equal(y, ry) and torch.equal(ids, rid) and torch.equal(w, rw)
    small = layer.forward(x[:5].contiguous())[0]
    assert torch.equal(small, m.moe_forward_gated(x[:5].contiguous(), wr, None, ex, 2, g, True)[0])
    plain = m.MoeLayer(wr, None, ex, 2, act_int8=True)          # the default gate: moe_route's choice
    assert torch.equal(plain.forward(x)[1], m.moe_forward(x, wr, None, ex, 2)[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        z = m.moe_forward_gated(x, wr, None, ex, 2, g, True)[0]
    side.synchronize()
    assert torch.equal(z, ry)
    src, dst = x.clone(), torch.empty_like(x)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    layer.forward(src)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(src, y=dst, ids=ids2, w=w2)
    for i in range(3):
        src.copy_(x.roll(i, 0))
        graph.replay()
        torch.cuda.synchronize()
        want = m.moe_forward_gated(x.roll(i, 0).contiguous(), wr, None, ex, 2, g, True)
        assert torch.equal(dst, want[0]) and torch.equal(ids2, want[1]) and torch.equal(w2, want[2])
    monkeypatch.setenv("MOE_DEBUG", "1")
    b2 = b.clone()
    b2[1:] = -float("inf")
    for act_int8 in (False, True):
        y, ids, _ = m.moe_forward_gated(x, wr, None, ex, 2, m.Gate(select_bias=b2), act_int8)
        assert (ids[:, 1] == -1).all() and (ids[:, 0] == 0).all()
    with pytest.raises(m.MoeError, match="CHECK"):
        m.moe_permute(ids, 16)


@pytest.mark.parametrize("gate", [None, m.Gate()])
def test_a_layer_captured_twice_then_grown(gate):
    """Two graphs of one layer replayed on two streams, and a larger batch between: no workspace is shared or lost."""
    x, wr, ex, _, _ = _case(900, 256, 384, 8)
    layer = m.MoeLayer(wr, None, ex, 2, gate=gate, act_int8=gate is not None)
    want = [layer.forward(x[a:a + 40].contiguous())[0].clone() for a in (0, 100)]
    graphs, outs, ins = [], [], []
    for a in (0, 100):
        ins.append(x[a:a + 40].contiguous())
        outs.append(torch.empty_like(ins[-1]))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            layer.forward(ins[-1], y=outs[-1])
    small = layer._ws.numel()
    big = layer.forward(x)[0].clone()
    assert layer._ws.numel() > small
    other = [torch.full((small,), 7, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))
        assert all((o == 7).all() for o in other)
        assert torch.equal(layer.forward(x)[0], big)


def test_schedule_lines(monkeypatch, capfd):
    monkeypatch.setenv("MOE_LOG", "1")
    x, wr, ex, b, _ = _case(600, 256, 4096, 4)
    m.moe_forward_gated(x[:3].contiguous(), wr, None, ex, 2, m.Gate(), True)
    m.moe_forward_gated(x, wr, None, ex, 2, m.Gate(), True)
    m.moe_forward_gated(torch.cat([x, x, x]), wr, None, ex, 2, m.Gate(), True)
    torch.cuda.synchronize()
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("[moe] moe_forward_gated")]
    assert len(lines) == 6 and all("act=int8 weights=int8" in l for l in lines)
    assert "stream schedule, 16-channel items, 16-row passes, reduction in 4 slices" in lines[0]
    # 10 + 4 row tiles by 32 channel tiles are fewer than 512, 29 + 4 are not
    assert "tiled schedule, 128x128 tiles" in lines[2] and "SwiGLU" in lines[2]
    assert "tiled schedule, 128x256 tiles" in lines[4] and "gate/up" in lines[4] and "down" in lines[5]


def test_empty():
    x, wr, ex, b, _ = _case(4, 128, 128, 4)
    y, ids, w = m.moe_forward_gated(x[:0], wr, None, ex, 2, m.Gate(), True)
    assert y.shape == (0, 128) and ids.shape == (0, 2)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert m.moe_expert_ffn_int8(x[:0], torch.zeros(5, dtype=torch.int32, device="cuda"), e, ex, 2).shape == (0, 128)
