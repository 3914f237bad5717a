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
    assert lib.moe_route_gated(_shape(**shape), _gate(**gate), A, A, None, A, A, None) == status
    if status != OK:
        assert lib.moe_last_error()


def test_route_gated_pointers(lib):
    call = lambda x=A, wr=A, b=None, ids=A, w=A, g=_gate(): lib.moe_route_gated(_shape(), g, x, wr, b, ids, w, None)
    assert call(g=None) == NULL
    for kw in (dict(x=None), dict(wr=None), dict(ids=None), dict(w=None)):
        assert call(**kw) == NULL, kw
    for kw in (dict(x=MIS), dict(wr=MIS), dict(b=MIS), dict(ids=MIS), dict(w=MIS)):
        assert call(**kw) == ALIGN, kw
    assert lib.moe_route_gated(_shape(T=0), _gate(), None, None, None, None, None, None) == OK


def test_grouped_mm_int8(lib):
    mm = lambda s, aq=A, asc=A, off=A, srt=A, w=A, ws=A, w2=None, w2s=None, out=A: lib.moe_grouped_mm_int8(
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
