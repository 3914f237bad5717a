"""What the MXFP4 calls accept at the ends of their ranges (CPU: every call returns before a launch).

A call that is accepted is shown by the next check, of a pointer that is missing.
"""
import ctypes

import pytest

from int8_weight_moe_amd import _lib
from tests.test_abi_mxfp4 import A, B, BIG, NULL, SHAPE, UNSUPPORTED, _post, _shape


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _gate_up(lib, s, h=None):
    return lib.moe_expert_gate_up(s, A, A, A, A, A, A, A, h, None, ctypes.c_size_t(0), None)


def _down(lib, s, y=None):
    return lib.moe_expert_down(s, A, A, A, A, y, None, ctypes.c_size_t(0), None)


def _forward(lib, s):
    return lib.moe_forward(s, A, A, None, A, A, A, A, A, A, None, None, None, A, BIG, None)


def _ffn(lib, s):
    return lib.moe_expert_ffn(s, A, A, A, A, A, A, A, A, A, None, A, BIG, None)


def test_rows_past_4_gib_are_streamed_not_refused(lib):
    """Only the rows that a pass reads are under the tiled kernel's 32-bit offsets, and AUTO streams past them."""
    big_h = dict(T=16384, d=256, f=24576, E=64, K=8)            # h of 6 GiB, x of 8 MiB
    big_x = dict(T=1 << 20, d=4096, f=256, E=4, K=1)            # x of 8 GiB, h of 512 MiB
    for kw in (big_h, big_x):
        for call in (_gate_up, _down, _forward, _ffn):
            assert call(lib, _shape(**kw)) == NULL, (kw, call, lib.moe_last_error())
    # on the tiled schedule the pass that reads them is refused, and what holds that pass
    tiled = _shape(ffn_path=2, **big_h)
    assert _gate_up(lib, tiled) == NULL
    for call in (_down, _forward, _ffn):
        assert call(lib, tiled) == UNSUPPORTED
    tiled = _shape(ffn_path=2, **big_x)
    assert _down(lib, tiled) == NULL
    for call in (_gate_up, _forward, _ffn):
        assert call(lib, tiled) == UNSUPPORTED
    # a matrix of 2^32 codes is 2 GiB, and weights are addressed in 64 bits
    for path in (0, 2):
        wide = _shape(T=4096, d=65536, f=65536, E=1, K=1, ffn_path=path)
        assert _gate_up(lib, wide) == NULL and _down(lib, wide) == NULL
    # the int8 comparators keep their limits
    for fmt in (1, 2):
        assert _gate_up(lib, _shape(weight_fmt=fmt, **big_h)) == UNSUPPORTED


@pytest.mark.parametrize("act,size", [(1, 32 * 256 * 2), (0, 32 * 256 * 4)])
def test_norm_outputs_that_overlap_are_refused(lib, act, size):
    """next over out loses out; arrays a few rows apart are read after they are written."""
    s = _shape(weight_fmt=0, act_dtype=act)
    at = lambda n: ctypes.c_void_p(0x10000 + n)
    nxt = _post(next_weight=A)
    far = ctypes.c_void_p(0x40000)
    for d in (16, 512, size - 16):
        assert lib.moe_norm_pre(s, at(d), A, 1e-6, at(0), None) == UNSUPPORTED
        assert lib.moe_norm_pre(s, at(0), A, 1e-6, at(d), None) == UNSUPPORTED
        assert lib.moe_norm_post(s, nxt, far, far, at(0), at(d), None) == UNSUPPORTED       # next, out
        assert lib.moe_norm_post(s, nxt, far, at(d), at(0), far, None) == UNSUPPORTED       # out, residual
        assert lib.moe_norm_post(s, nxt, far, at(d), far, at(0), None) == UNSUPPORTED       # next, residual
        assert lib.moe_norm_post(s, nxt, at(0), far, far, at(d), None) == UNSUPPORTED       # next, y
        assert lib.moe_norm_post(s, _post(), at(0), far, at(d), None, None) == UNSUPPORTED  # out, y
        assert lib.moe_combine_post(s, nxt, A, A, A, far, at(0), at(d), None) == UNSUPPORTED
    assert lib.moe_norm_post(s, nxt, far, far, A, A, None) == UNSUPPORTED
    assert lib.moe_combine_post(s, nxt, A, A, A, far, B, B, None) == UNSUPPORTED
    blk = _shape(act_dtype=1)
    assert lib.moe_block_forward(blk, far, A, 1e-6, None, nxt, A, None, A, A, A, A, A, A, B, B, None, None, A, BIG,
                                 None) == UNSUPPORTED
    # side by side, and in place, pass on to the next check
    assert lib.moe_norm_post(s, nxt, None, at(size), at(0), at(2 * size), None) == NULL
    assert lib.moe_norm_post(s, nxt, None, at(0), at(0), at(size), None) == NULL
    assert lib.moe_norm_post(s, nxt, None, at(0), at(size), at(0), None) == NULL


def test_product_takes_more_slots_a_token_than_experts(lib):
    """A shard with fewer experts than a token has slots; only the calls that route keep K <= E."""
    mm = lambda s: lib.moe_grouped_mm_mxfp4(s, A, A, A, A, A, A, None, None, None, None)
    for E, K in ((1, 2), (2, 8), (7, 8)):
        assert mm(_shape(E=E, K=K)) == NULL
        n = ctypes.c_size_t(0)
        assert lib.moe_expert_ffn_mxfp4_workspace_size(_shape(E=E, K=K), ctypes.byref(n)) == SHAPE
        assert lib.moe_workspace_size(_shape(E=E, K=K), ctypes.byref(n)) == SHAPE
    assert mm(_shape(K=9)) == SHAPE and mm(_shape(E=1, K=9)) == SHAPE and mm(_shape(K=0)) == SHAPE


def test_norm_outputs_over_what_other_tokens_read_are_refused(lib):
    """out or next over the experts' rows, the weights or a shared gate would change what later tokens read."""
    s = _shape(weight_fmt=0)                                            # 32 tokens of 512 bytes; y_rows 64 of 1 KiB
    at = lambda n: ctypes.c_void_p(0x100000 + n)
    far = lambda i: ctypes.c_void_p(0x200000 + 0x10000 * i)
    combine = lambda post, y_rows, out, nxt: lib.moe_combine_post(s, post, y_rows, far(0), far(1), far(2), out, nxt, None)
    both = _post(weight=far(3), next_weight=far(4))
    for d in (0, 16, 64 * 1024 - 16):
        assert combine(both, at(0), at(d), far(5)) == UNSUPPORTED and b"y_rows" in lib.moe_last_error()
        assert combine(both, at(0), far(5), at(d)) == UNSUPPORTED
    assert combine(both, at(32 * 512 - 16), at(0), far(5)) == UNSUPPORTED
    for name, size in (("weight", 512), ("next_weight", 512), ("gate", 11 * 512)):
        arrays = dict(weight=far(3), next_weight=far(4), gate_tokens=3)
        arrays[name] = at(0)
        post = _post(**arrays)
        for out, nxt in ((at(size - 16), far(5)), (far(5), at(size - 16)), (at(-32 * 512 + 16), far(5))):
            assert lib.moe_norm_post(s, post, far(6), far(7), out, nxt, None) == UNSUPPORTED, name
            assert name.encode() in lib.moe_last_error()
            assert combine(post, far(8), out, nxt) == UNSUPPORTED, name
    blk = _shape()
    assert lib.moe_block_forward(blk, far(0), far(1), 1e-6, None, _post(weight=at(0)), A, None, A, A, A, A, A, A, at(16),
                                 None, None, None, A, BIG, None) == UNSUPPORTED
