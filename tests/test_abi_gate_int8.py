"""Refusals of the gated-routing and int8-activation entry points (CPU: every call returns before a launch)."""
import ctypes
import re

import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd import _lib
from tests.test_abi import HEADER

A, B, MIS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x10008)
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = range(7)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _shape(**kw):
    base = dict(T=32, d=256, f=512, E=16, K=2, act_dtype=1, scale_dtype=1, ffn_path=0, weight_fmt=0)
    base.update(kw)
    return ctypes.byref(_lib.MoeShape(**base))


def _gate(**kw):
    base = dict(select_bias=None, score=0, groups=1, group_topk=1, group_by=0, renorm=1, scale=1.0)
    base.update(kw)
    return ctypes.byref(_lib.MoeGate(**base))


def test_header_constants():
    text = open(HEADER).read()
    for name, val in (("MOE_SCORE_SOFTMAX", 0), ("MOE_SCORE_SIGMOID", 1), ("MOE_GROUP_MAX", 0), ("MOE_GROUP_TOP2", 1)):
        assert re.search(rf"\b{name}\s*=\s*{val}\b", text), name
    assert ctypes.sizeof(_lib.MoeGate) == 32


@pytest.mark.parametrize("shape,gate,status", [
    (dict(E=257), {}, SHAPE), (dict(E=0), {}, SHAPE), (dict(E=300, K=9), {}, SHAPE), (dict(d=100), {}, SHAPE),
    (dict(act_dtype=2), {}, DTYPE), ({}, dict(score=2), SHAPE), ({}, dict(score=-1), SHAPE),
    ({}, dict(groups=0), SHAPE), ({}, dict(groups=3), SHAPE), (dict(E=130), dict(groups=65), SHAPE),
    ({}, dict(groups=4, group_topk=0), SHAPE), ({}, dict(groups=4, group_topk=5), SHAPE), ({}, dict(group_topk=2), SHAPE),
    (dict(K=5), dict(groups=4, group_topk=1), SHAPE), ({}, dict(groups=4, group_by=2), SHAPE),
    ({}, dict(groups=16, group_topk=2, group_by=1), SHAPE), ({}, dict(renorm=2), SHAPE),
    ({}, dict(scale=float("inf")), SHAPE), ({}, dict(scale=float("nan")), SHAPE), ({}, dict(select_bias=MIS), ALIGN),
    (dict(T=0, E=256, K=8), dict(groups=8, group_topk=4, group_by=1), OK), (dict(T=0), dict(group_by=1), OK),
    (dict(T=0, E=1, K=1), dict(group_by=1), OK), (dict(T=0), dict(groups=16, group_topk=2, scale=-2.5), OK),
])
def test_gate_refusals(lib, shape, gate, status):
    assert lib.moe_route_gated(_shape(**shape), _gate(**gate), A, A, None, A, A, None, 0, None) == status
    if status != OK:
        assert lib.moe_last_error()


def test_route_gated_pointers(lib):
    call = lambda x=A, wr=A, b=None, ids=A, w=A, g=_gate(): lib.moe_route_gated(_shape(), g, x, wr, b, ids, w, None, 0, None)
    assert call(g=None) == NULL
    for kw in (dict(x=None), dict(wr=None), dict(ids=None), dict(w=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(x=MIS), dict(wr=MIS), dict(b=MIS), dict(ids=MIS), dict(w=MIS)):
        assert call(**kw) == ALIGN, kw
    assert lib.moe_route_gated(_shape(T=0), _gate(), None, None, None, None, None, None, 0, None) == OK
    n = ctypes.c_size_t(0)
    size = lib.moe_route_gated_workspace_size
    assert size(_shape(E=257), ctypes.byref(n)) == SHAPE and size(_shape(), None) == NULL
    # 64 bf16 columns a block, 16 slices of 16 experts: 8 steps and more are split, up to 1024 tokens
    for kw, want in ((dict(T=1, d=4096), 0), (dict(T=1, d=8192), 8 * (16 * 8 + 17 * 4)), (dict(T=1024, d=8192, E=256), 4 * (1024 * 2048 + 1280 * 4)),
                     (dict(T=1025, d=8192), 0), (dict(T=0, d=8192), 0), (dict(T=17, d=4096, act_dtype=0), 8 * (17 * 128 + 33 * 4))):
        assert size(_shape(**kw), ctypes.byref(n)) == OK and n.value == want, kw
    big = _shape(T=1, d=8192)
    call = lambda ws, b: lib.moe_route_gated(big, _gate(), A, A, None, A, A, ws, ctypes.c_size_t(b), None)
    assert call(A, 8 * 196 - 1) == WORKSPACE and call(MIS, 8 * 196) == ALIGN


def test_grouped_mm_int8(lib):
    out_at = ctypes.c_void_p(1 << 40)
    mm = lambda s, aq=A, asc=A, off=A, srt=A, w=A, ws=A, w2=None, w2s=None, out=out_at: lib.moe_grouped_mm_int8(
        s, aq, asc, off, srt, w, ws, w2, w2s, out, None)
    for fmt in (1, 2, 4):
        assert mm(_shape(weight_fmt=fmt)) == DTYPE
    assert mm(_shape(d=100)) == SHAPE and mm(_shape(f=72)) == SHAPE and mm(_shape(E=65)) == SHAPE
    assert mm(_shape(K=9)) == SHAPE and mm(_shape(scale_dtype=2)) == DTYPE and mm(_shape(ffn_path=3)) == SHAPE
    for kw in (dict(aq=None), dict(asc=None), dict(off=None), dict(w=None), dict(ws=None), dict(out=None),
               dict(w2=A), dict(w2s=A)):
        assert mm(_shape(), **kw) == NULL, kw
    for kw in (dict(aq=MIS), dict(asc=MIS), dict(off=MIS), dict(srt=MIS), dict(w=MIS), dict(ws=MIS), dict(out=MIS),
               dict(w2=MIS, w2s=A), dict(w2=A, w2s=MIS)):
        assert mm(_shape(), **kw) == ALIGN, kw
    # out [64, 512] bf16 may touch no input: rows [32, 256], matrices [16, 512, 256]
    end = (1 << 40) + 64 * 512 * 2
    P = ctypes.c_void_p
    for kw in (dict(aq=P(end - 16)), dict(aq=P((1 << 40) - 32 * 256 + 16)), dict(asc=P(end - 16)), dict(w=P((1 << 40) - 16)),
               dict(ws=out_at), dict(off=out_at), dict(srt=P(end - 256)), dict(w2=out_at, w2s=A), dict(w2=A, w2s=out_at)):
        assert mm(_shape(), **kw) == UNSUPPORTED and b"overlaps" in lib.moe_last_error(), kw
    assert mm(_shape(T=0), None, None, None, None, None, None, None, None, None) == OK


def test_binding_checks():
    """Each call is refused before it reaches the library."""
    x, wr = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x is on cpu"):
        m.moe_route_gated(x, wr, None, 2, m.Gate())
    with pytest.raises(ValueError, match="select_bias is on cpu"):
        m.moe_route_gated(x, wr, None, 2, m.Gate(select_bias=torch.zeros(8)))
    with pytest.raises(ValueError, match="past 2.31"):
        m.moe_route_gated(x, wr, None, 2, m.Gate(groups=1 << 32))
    aq, wq = torch.zeros(4, 128, dtype=torch.int8), torch.zeros(2, 64, 128, dtype=torch.int8)
    a_s, w_s, off = torch.zeros(4), torch.zeros(2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="a_q must be"):
        m.moe_grouped_mm_int8(aq[0], a_s, off, wq, w_s, torch.float32)
    with pytest.raises(ValueError, match="K is the slots"):
        m.moe_grouped_mm_int8(aq, a_s, off, wq, w_s, torch.float32, K=2)
    with pytest.raises(ValueError, match="given together"):
        m.moe_grouped_mm_int8(aq, a_s, off, wq, w_s, torch.float32, w2_q=wq)
    with pytest.raises(TypeError, match="unsupported dtype"):
        m.moe_grouped_mm_int8(aq, a_s, off, wq, w_s, torch.float16)
    with pytest.raises(TypeError, match="unsupported dtype"):
        m.moe_grouped_mm_int8(aq, a_s, off, wq, w_s.half(), torch.float32)
    with pytest.raises(ValueError, match="a_q is on cpu"):
        m.moe_grouped_mm_int8(aq, a_s, off, wq, w_s, torch.float32)


BIG = ctypes.c_size_t(1 << 40)


def _r(v):
    return (v + 255) // 256 * 256


def test_expert_ffn_int8(lib):
    n = ctypes.c_size_t(0)
    size = lib.moe_expert_ffn_int8_workspace_size
    assert size(_shape(weight_fmt=2), ctypes.byref(n)) == DTYPE and size(_shape(), None) == NULL
    assert size(_shape(K=17), ctypes.byref(n)) == SHAPE and size(_shape(E=1), ctypes.byref(n)) == SHAPE
    assert size(_shape(), ctypes.byref(n)) == OK
    assert n.value == _r(32 * 256) + _r(32 * 4) + _r(64 * 512) + _r(64 * 4) + _r(64 * 1024)
    call = lambda ws, b: lib.moe_expert_ffn_int8(_shape(), *([A] * 10), ws, ctypes.c_size_t(b), None)
    assert call(A, n.value - 1) == WORKSPACE and call(None, n.value) == NULL and call(MIS, n.value) == ALIGN
    for i in range(10):
        args = [A] * 10
        args[i] = None
        assert lib.moe_expert_ffn_int8(_shape(), *args, A, n, None) == NULL, i
    assert lib.moe_expert_ffn_int8(_shape(T=0), *([None] * 11), ctypes.c_size_t(0), None) == OK


def test_forward_gated(lib):
    n, fwd, ffn = (ctypes.c_size_t(0) for _ in range(3))
    size = lib.moe_gated_workspace_size
    assert size(_shape(), 2, ctypes.byref(n)) == DTYPE and size(_shape(), 0, None) == NULL
    assert size(_shape(E=65), 0, ctypes.byref(n)) == SHAPE
    for fmt in (1, 2, 4):
        assert size(_shape(weight_fmt=fmt), 1, ctypes.byref(n)) == DTYPE
    assert lib.moe_workspace_size(_shape(), ctypes.byref(fwd)) == OK
    assert lib.moe_expert_ffn_int8_workspace_size(_shape(), ctypes.byref(ffn)) == OK
    assert size(_shape(), 0, ctypes.byref(n)) == OK and n.value == _r(fwd.value)
    assert size(_shape(), 1, ctypes.byref(n)) == OK and n.value == _r(fwd.value) + ffn.value - _r(64 * 1024)

    def call(s=None, g=None, act=1, ptrs=None, ws=A, b=1 << 40, ids=None):
        ptrs = ptrs or [A, A, None, A, A, A, A, A, A, B]
        return lib.moe_forward_gated(s or _shape(), g or _gate(), act, *ptrs, ids, None, ws, ctypes.c_size_t(b), None)
    assert lib.moe_forward_gated(_shape(), None, 0, *([A] * 13), BIG, None) == NULL
    assert call(act=-1) == DTYPE and call(_shape(weight_fmt=2), act=1) == DTYPE
    assert call(_shape(E=128)) == SHAPE and call(g=_gate(groups=5)) == SHAPE and call(g=_gate(select_bias=MIS)) == ALIGN
    assert call(b=n.value - 1) == WORKSPACE and call(ws=None) == NULL and call(ids=MIS) == ALIGN
    assert call(act=0, b=fwd.value - 1) == WORKSPACE
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9):
        ptrs = [A, A, None, A, A, A, A, A, A, B]
        ptrs[i] = None
        assert call(ptrs=ptrs) == NULL, i
        ptrs[i] = MIS
        assert call(ptrs=ptrs) == ALIGN, i
    assert call(ptrs=[A, A, MIS, A, A, A, A, A, A, B]) == ALIGN
    assert lib.moe_forward_gated(_shape(T=0), _gate(), 1, *([None] * 13), ctypes.c_size_t(0), None) == OK


def test_block_forward_gated(lib):
    n, g = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.moe_gated_workspace_size(_shape(), 1, ctypes.byref(g)) == OK
    assert lib.moe_block_gated_workspace_size(_shape(), 1, ctypes.byref(n)) == OK
    assert n.value == _r(g.value) + _r(32 * 256 * 2)
    assert lib.moe_block_gated_workspace_size(_shape(), 3, ctypes.byref(n)) == DTYPE
    post = ctypes.byref(_lib.MoePost(weight=A, gate=None, next_weight=None, gate_tokens=1, residual_scale=1.0,
                                     block_scale=1.0, eps=1e-6, next_eps=1e-6))

    def call(s=None, gate=_gate(), act=1, b=1 << 40, x=None, pre=A):
        return lib.moe_block_forward_gated(s or _shape(), gate, act, A, pre, 1e-6, x, post, A, None, A, A, A, A, A, A, B,
                                           None, None, None, A, ctypes.c_size_t(b), None)
    assert call(gate=None) == NULL and call(gate=_gate(score=7)) == SHAPE and call(act=5) == DTYPE
    assert call(_shape(weight_fmt=1)) == DTYPE
    assert call(b=_r(g.value) + _r(32 * 256 * 2) - 1) == WORKSPACE
    assert call(x=A) == UNSUPPORTED and call(pre=None) == NULL
    assert call(_shape(T=0)) == OK


@pytest.mark.parametrize("T,d", [(3, 8192), (32, 256), (1024, 8192), (2000, 8192)])
def test_blocks_ask_for_the_workspace_they_name(lib, T, d):
    """moe_block_forward asks for moe_block_workspace_size whatever gated routing would split."""
    post = _lib.MoePost(None, None, None, 1, 1.0, 1.0, 1e-6, 1e-6)
    s = _shape(T=T, d=d)
    n, g = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lib.moe_block_workspace_size(s, ctypes.byref(n)) == OK
    far = [ctypes.c_void_p((1 + i) << 40) for i in range(3)]
    call = lambda b: lib.moe_block_forward(s, far[0], A, 1e-6, None, ctypes.byref(post), *[A] * 2, *[A] * 6, far[1], None, None, None,
                                           A, ctypes.c_size_t(b), None)
    assert call(n.value - 1) == WORKSPACE
    assert f"required {n.value}".encode() in lib.moe_last_error()
    assert lib.moe_block_gated_workspace_size(s, 0, ctypes.byref(g)) == OK
    r = ctypes.c_size_t(0)
    assert lib.moe_route_gated_workspace_size(s, ctypes.byref(r)) == OK
    assert n.value + r.value <= g.value <= n.value + r.value + 1024


def test_binding_of_the_layer():
    from tests.test_binding_mxfp4 import D, E, _experts
    x, wr = torch.zeros(4, D, dtype=torch.bfloat16), torch.zeros(E, D, dtype=torch.bfloat16)
    off, srt = torch.zeros(E + 1, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    ex = _experts(m.MOE_W_INT8)
    for bad in (m.MOE_W_FP8, m.MOE_W_MXFP4):
        with pytest.raises(ValueError, match="not in int8"):
            m.moe_expert_ffn_int8(x, off, srt, _experts(bad), 2)
    for call in (lambda: m.moe_expert_ffn_int8(x, off, srt, ex, 2),
                 lambda: m.moe_forward_gated(x, wr, None, ex, 2, m.Gate()),
                 lambda: m.moe_block_forward_gated(x, wr, None, ex, 2, m.Gate(), pre_weight=x[0])):
        with pytest.raises(ValueError, match="not on the current HIP device"):
            call()
    with pytest.raises(ValueError, match="columns"):
        m.moe_forward_gated(x[:, :64].contiguous(), wr, None, ex, 2, m.Gate())
    ex.s_up = ex.s_up[:, :-1].contiguous()
    with pytest.raises(ValueError, match="the experts' s_up"):
        m.moe_forward_gated(x, wr, None, ex, 2, m.Gate())
