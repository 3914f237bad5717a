"""Refusals of the MXFP4 and norm entry points (CPU: every call returns before a launch)."""
import ctypes
import re

import pytest
import torch

import int8_weight_moe_amd as m
from int8_weight_moe_amd import _lib
from tests.test_abi import HEADER

A, B, MIS = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.c_void_p(0x10008)
BIG = ctypes.c_size_t(1 << 40)
OK, NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED = range(7)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _shape(**kw):
    base = dict(T=32, d=256, f=512, E=16, K=2, act_dtype=1, scale_dtype=1, ffn_path=0, weight_fmt=4)
    base.update(kw)
    return ctypes.byref(_lib.MoeShape(**base))


def _post(**kw):
    base = dict(weight=A, gate=None, next_weight=None, gate_tokens=1, residual_scale=1.0, block_scale=1.0, eps=1e-6,
                next_eps=1e-6)
    base.update(kw)
    return ctypes.byref(_lib.MoePost(**base))


def test_header_constants():
    text = open(HEADER).read()
    for name, val in (("MOE_W_MXFP4", 4), ("MOE_MX_ROWS", 0), ("MOE_MX_TILED", 1)):
        assert re.search(rf"\b{name}\s*=\s*{val}\b", text), name
    assert ctypes.sizeof(_lib.MoePost) == 48 and ctypes.sizeof(_lib.MoeShape) == 36


@pytest.mark.parametrize("rows,cols,layout,status", [
    (4, 48, 0, SHAPE), (4, 0, 0, SHAPE), (-1, 64, 0, SHAPE), (4, 1 << 21, 0, SHAPE), (1 << 31, 32, 0, SHAPE),
    (8, 128, 1, SHAPE), (16, 96, 1, SHAPE), (16, 64, 1, SHAPE), (16, 128, 2, SHAPE), (0, 32, 0, OK), (0, 128, 1, OK),
])
def test_quantizer_sizes(lib, rows, cols, layout, status):
    assert lib.moe_quantize_mxfp4(rows, cols, 1, A, layout, A, A, None) == status
    assert lib.moe_dequantize_mxfp4(rows, cols, layout, A, A, 1, A, None) == status
    if layout == 1:
        assert lib.moe_pack_mxfp4(rows, cols, A, A, B, B, None) == status


def test_quantizer_pointers_and_types(lib):
    assert lib.moe_quantize_mxfp4(4, 64, 2, A, 0, A, A, None) == DTYPE
    assert lib.moe_dequantize_mxfp4(4, 64, 0, A, A, -1, A, None) == DTYPE
    for args, st in (((None, 0, A, A), NULL), ((A, 0, None, A), NULL), ((A, 0, A, None), NULL), ((MIS, 0, A, A), ALIGN),
                     ((A, 0, MIS, A), ALIGN), ((A, 0, A, MIS), ALIGN)):
        assert lib.moe_quantize_mxfp4(4, 64, 1, *args, None) == st
    assert lib.moe_dequantize_mxfp4(4, 64, 0, A, A, 1, None, None) == NULL
    assert lib.moe_pack_mxfp4(16, 128, A, A, A, B, None) == UNSUPPORTED
    assert lib.moe_pack_mxfp4(16, 128, A, B, B, B, None) == UNSUPPORTED
    assert lib.moe_pack_mxfp4(16, 128, A, A, B, None, None) == NULL


def test_ffn_with_mxfp4_weights(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_workspace_size(_shape(), ctypes.byref(n)) == OK and n.value > 0
    gate_up = lambda s: lib.moe_expert_gate_up(s, A, A, A, A, A, A, A, A, None, ctypes.c_size_t(0), None)
    down = lambda s: lib.moe_expert_down(s, A, A, A, A, A, None, ctypes.c_size_t(0), None)
    fwd = lambda s: lib.moe_forward(s, A, A, None, A, A, A, A, A, A, A, None, None, A, BIG, None)
    for call in (gate_up, down, fwd):
        assert call(_shape(act_dtype=0)) == UNSUPPORTED
        assert call(_shape(d=192)) == SHAPE and b"128" in lib.moe_last_error()
        assert call(_shape(f=192)) == SHAPE
    # scales are needed
    assert lib.moe_forward(_shape(), A, A, None, A, A, A, A, None, A, A, None, None, A, BIG, None) == NULL
    # the tiled schedule's 32-bit offsets
    assert gate_up(_shape(T=1 << 20, d=4096, K=1, ffn_path=2)) == UNSUPPORTED
    # the code between fp8 and MXFP4 stays unassigned
    assert lib.moe_workspace_size(_shape(weight_fmt=3), ctypes.byref(n)) == DTYPE


def test_grouped_mm(lib):
    mm = lambda s, aq=A, asc=A, off=A, srt=A, w=A, ws=A, w2=None, w2s=None, out=A: lib.moe_grouped_mm_mxfp4(
        s, aq, asc, off, srt, w, ws, w2, w2s, out, None)
    assert mm(_shape(weight_fmt=0)) == DTYPE
    assert mm(_shape(d=192)) == SHAPE and mm(_shape(f=320)) == SHAPE and mm(_shape(E=65)) == SHAPE
    for kw in (dict(aq=None), dict(asc=None), dict(off=None), dict(w=None), dict(ws=None), dict(out=None),
               dict(w2=A), dict(w2s=A)):
        assert mm(_shape(), **kw) == NULL, kw
    for kw in (dict(aq=MIS), dict(asc=MIS), dict(srt=MIS), dict(ws=MIS), dict(out=MIS), dict(w2=MIS, w2s=A)):
        assert mm(_shape(), **kw) == ALIGN, kw
    assert mm(_shape(T=0), None, None, None, None, None, None, None, None, None) == OK


def test_expert_ffn_mxfp4(lib):
    n = ctypes.c_size_t(0)
    assert lib.moe_expert_ffn_mxfp4_workspace_size(_shape(weight_fmt=2), ctypes.byref(n)) == DTYPE
    assert lib.moe_expert_ffn_mxfp4_workspace_size(_shape(), None) == NULL
    assert lib.moe_expert_ffn_mxfp4_workspace_size(_shape(), ctypes.byref(n)) == OK
    r = lambda v: (v + 255) // 256 * 256
    assert n.value == r(32 * 128) + r(32 * 8) + r(64 * 1024) + r(64 * 256) + r(64 * 16)
    call = lambda ws, size: lib.moe_expert_ffn_mxfp4(_shape(), *([A] * 10), ws, ctypes.c_size_t(size), None)
    assert call(A, n.value - 1) == WORKSPACE and call(None, n.value) == NULL and call(MIS, n.value) == ALIGN
    assert lib.moe_expert_ffn_mxfp4(_shape(T=0), *([None] * 11), ctypes.c_size_t(0), None) == OK


def test_norms(lib):
    s = _shape(weight_fmt=0)
    for eps in (-1e-6, float("nan"), float("inf")):
        assert lib.moe_norm_pre(s, A, A, eps, A, None) == SHAPE
        assert lib.moe_norm_post(s, _post(eps=eps), A, A, A, None, None) == SHAPE
        assert lib.moe_norm_post(s, _post(next_weight=A, next_eps=eps), A, A, A, B, None) == SHAPE
    assert lib.moe_norm_pre(s, A, None, 1e-6, A, None) == NULL
    assert lib.moe_norm_pre(s, MIS, A, 1e-6, A, None) == ALIGN
    assert lib.moe_norm_post(s, None, A, A, A, None, None) == NULL
    assert lib.moe_norm_post(s, _post(), None, A, A, None, None) == NULL
    assert lib.moe_norm_post(s, _post(), A, None, A, None, None) == NULL
    assert lib.moe_norm_post(s, _post(next_weight=A), A, A, A, None, None) == NULL
    assert lib.moe_norm_post(s, _post(gate=A, gate_tokens=0), A, A, A, None, None) == SHAPE
    for kw in (dict(weight=MIS), dict(gate=MIS), dict(next_weight=MIS)):
        assert lib.moe_norm_post(s, _post(**kw), A, A, A, A, None) == ALIGN
    assert lib.moe_combine_post(s, _post(), A, None, A, A, A, None, None) == NULL
    assert lib.moe_combine_post(s, _post(), MIS, A, A, A, A, None, None) == ALIGN
    assert lib.moe_combine_post(_shape(K=9, weight_fmt=0), _post(), A, A, A, A, A, None, None) == SHAPE
    z = _shape(T=0, weight_fmt=0)
    assert lib.moe_norm_pre(z, None, None, 1e-6, None, None) == OK
    assert lib.moe_norm_post(z, _post(weight=None), None, None, None, None, None) == OK
    assert lib.moe_combine_post(z, _post(), None, None, None, None, None, None, None) == OK


def test_block(lib):
    n = ctypes.c_size_t(0)
    fw = ctypes.c_size_t(0)
    assert lib.moe_workspace_size(_shape(), ctypes.byref(fw)) == OK
    assert lib.moe_block_workspace_size(_shape(), ctypes.byref(n)) == OK
    assert n.value == (fw.value + 255) // 256 * 256 + 32 * 256 * 2

    def call(s=None, res=A, pre=A, x=None, post=None, rw=A, w=A, out=B, ws=A, size=1 << 40, eps=1e-6):
        return lib.moe_block_forward(s or _shape(), res, pre, eps, x, post or _post(), rw, None, w, A, A, A, A, A, out,
                                     None, None, None, ws, ctypes.c_size_t(size), None)

    assert call(size=n.value - 1) == WORKSPACE
    assert call(x=A) == UNSUPPORTED and call(pre=None) == NULL
    assert call(res=None) == NULL and call(rw=None) == NULL and call(w=None) == NULL and call(out=None) == NULL
    assert call(pre=MIS) == ALIGN and call(pre=None, x=MIS) == ALIGN and call(ws=MIS) == ALIGN
    assert call(eps=-1.0) == SHAPE and call(s=_shape(act_dtype=0)) == UNSUPPORTED and call(s=_shape(d=192)) == SHAPE
    assert call(s=_shape(T=0), res=None, pre=None, rw=None, w=None, out=None, ws=None) == OK


def test_binding_checks_before_the_library():
    """Tensors that are not on the current device, or do not belong together, are refused in Python."""
    q, s = torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="not on the current HIP device"):
        m.moe_dequantize_mxfp4(q, s, torch.bfloat16)
    with pytest.raises(ValueError, match="do not belong together"):
        m.moe_pack_mxfp4(q, s[:, :3])
    with pytest.raises(ValueError, match="multiple of 32"):
        m.moe_quantize_mxfp4(torch.zeros(4, 40))
    with pytest.raises(TypeError):
        m.moe_quantize_mxfp4(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="sorted_slots"):
        m.moe_grouped_mm_mxfp4(q, s, torch.zeros(2, dtype=torch.int32), q[None], s[None], torch.float32, K=2)
    with pytest.raises(ValueError, match="together"):
        m.moe_grouped_mm_mxfp4(q, s, torch.zeros(2, dtype=torch.int32), q[None], s[None], torch.float32, w2_q=q[None])
    with pytest.raises(ValueError, match="not on the current HIP device"):
        m.moe_norm_pre(torch.zeros(2, 64), torch.ones(64))
