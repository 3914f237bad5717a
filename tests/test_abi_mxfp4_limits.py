"""What the MXFP4 calls accept at the ends of their ranges (CPU: every call returns before a launch).

A call that is accepted is shown by the next check, of a pointer that is missing.
"""
import ctypes

import pytest

from int8_weight_moe_amd import _lib
from tests.test_abi_mxfp4 import A, BIG, NULL, UNSUPPORTED, _shape


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
