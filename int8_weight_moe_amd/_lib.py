"""ctypes loader for libmoe_int8.so and its C ABI (include/moe_int8.h).

Loading fails loudly when the shared library has not been built: there is no
fallback implementation of any call.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_int8.so")

ABI_VERSION = 8
MOE_OK = 0
STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_DTYPE", 4: "MOE_ERR_ALIGN",
    5: "MOE_ERR_WORKSPACE", 6: "MOE_ERR_UNSUPPORTED", 7: "MOE_ERR_HIP",
    8: "MOE_ERR_CHECK",
}
MOE_F32, MOE_BF16 = 0, 1
MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED = 0, 1, 2
MOE_W_INT8, MOE_W_BF16, MOE_W_FP8, MOE_W_MXFP4 = 0, 1, 2, 4
MOE_MX_ROWS, MOE_MX_TILED = 0, 1
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1
MOE_ACT_AS_IS, MOE_ACT_INT8 = 0, 1

# every symbol the header declares
EXPORTS = (
    "moe_abi_version", "moe_status_str", "moe_last_error", "moe_workspace_size", "moe_ffn_workspace_size",
    "moe_route", "moe_permute", "moe_expert_ffn", "moe_expert_gate_up", "moe_expert_down", "moe_combine", "moe_forward", "moe_quantize_rows",
    "moe_pack_rows", "moe_mlp_workspace_size", "moe_mlp_forward", "moe_quantize_rows_fp8", "moe_down_workspace_size",
    "moe_forward_noalloc", "moe_gate_up_workspace_size", "moe_quantize_pack_rows",
    "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_pack_mxfp4", "moe_grouped_mm_mxfp4",
    "moe_expert_ffn_mxfp4_workspace_size", "moe_expert_ffn_mxfp4", "moe_norm_pre", "moe_norm_post",
    "moe_combine_post", "moe_block_workspace_size", "moe_block_forward",
    "moe_route_gated_workspace_size", "moe_route_gated", "moe_grouped_mm_int8", "moe_expert_ffn_int8_workspace_size", "moe_expert_ffn_int8",
    "moe_gated_workspace_size", "moe_forward_gated", "moe_block_gated_workspace_size", "moe_block_forward_gated",
)


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("f", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("act_dtype", ctypes.c_int32), ("scale_dtype", ctypes.c_int32),
                ("ffn_path", ctypes.c_int32), ("weight_fmt", ctypes.c_int32)]


class MoePost(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("next_weight", ctypes.c_void_p),
                ("gate_tokens", ctypes.c_int32), ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("next_eps", ctypes.c_float)]


class MoeGate(ctypes.Structure):
    _fields_ = [("select_bias", ctypes.c_void_p), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("group_topk", ctypes.c_int32), ("group_by", ctypes.c_int32), ("renorm", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_P = ctypes.c_void_p
_SHAPE = ctypes.POINTER(MoeShape)
_POST = ctypes.POINTER(MoePost)
_GATE = ctypes.POINTER(MoeGate)
_I32, _I64, _F32, _SIZE = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "moe_abi_version": (ctypes.c_int32, []),
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int32]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_workspace_size": (ctypes.c_int32, [_SHAPE, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_ffn_workspace_size": (ctypes.c_int32, [_SHAPE, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_route": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P]),
    "moe_permute": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P]),
    "moe_expert_ffn": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_gate_up": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_gate_up_workspace_size": (ctypes.c_int32, [_SHAPE, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_expert_down": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_down_workspace_size": (ctypes.c_int32, [_SHAPE, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_combine": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P]),
    "moe_forward": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_quantize_rows": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P]),
    "moe_quantize_rows_fp8": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P]),
    "moe_pack_rows": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int32, _P, _P, _P]),
    "moe_quantize_pack_rows": (ctypes.c_int32, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _P, ctypes.c_int32,
                                                ctypes.c_int32, _P, _P, _P]),
    "moe_mlp_workspace_size": (ctypes.c_int32, [_SHAPE, ctypes.POINTER(ctypes.c_size_t)]),
    "moe_mlp_forward": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_forward_noalloc": (ctypes.c_int32, [_SHAPE, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_quantize_mxfp4": (_I32, [_I64, _I32, _I32, _P, _I32, _P, _P, _P]),
    "moe_dequantize_mxfp4": (_I32, [_I64, _I32, _I32, _P, _P, _I32, _P, _P]),
    "moe_pack_mxfp4": (_I32, [_I64, _I32, _P, _P, _P, _P, _P]),
    "moe_grouped_mm_mxfp4": (_I32, [_SHAPE] + [_P] * 10),
    "moe_expert_ffn_mxfp4_workspace_size": (_I32, [_SHAPE, ctypes.POINTER(_SIZE)]),
    "moe_expert_ffn_mxfp4": (_I32, [_SHAPE] + [_P] * 11 + [_SIZE, _P]),
    "moe_route_gated_workspace_size": (_I32, [_SHAPE, ctypes.POINTER(_SIZE)]),
    "moe_route_gated": (_I32, [_SHAPE, _GATE] + [_P] * 6 + [_SIZE, _P]),
    "moe_grouped_mm_int8": (_I32, [_SHAPE] + [_P] * 10),
    "moe_expert_ffn_int8_workspace_size": (_I32, [_SHAPE, ctypes.POINTER(_SIZE)]),
    "moe_expert_ffn_int8": (_I32, [_SHAPE] + [_P] * 11 + [_SIZE, _P]),
    "moe_gated_workspace_size": (_I32, [_SHAPE, _I32, ctypes.POINTER(_SIZE)]),
    "moe_forward_gated": (_I32, [_SHAPE, _GATE, _I32] + [_P] * 13 + [_SIZE, _P]),
    "moe_block_gated_workspace_size": (_I32, [_SHAPE, _I32, ctypes.POINTER(_SIZE)]),
    "moe_block_forward_gated": (_I32, [_SHAPE, _GATE, _I32, _P, _P, _F32, _P, _POST] + [_P] * 13 + [_SIZE, _P]),
    "moe_norm_pre": (_I32, [_SHAPE, _P, _P, _F32, _P, _P]),
    "moe_norm_post": (_I32, [_SHAPE, _POST, _P, _P, _P, _P, _P]),
    "moe_combine_post": (_I32, [_SHAPE, _POST, _P, _P, _P, _P, _P, _P, _P]),
    "moe_block_workspace_size": (_I32, [_SHAPE, ctypes.POINTER(_SIZE)]),
    "moe_block_forward": (_I32, [_SHAPE, _P, _P, _F32, _P, _POST] + [_P] * 13 + [_SIZE, _P]),
}

_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoe_int8.so once and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it first (python -m int8_weight_moe_amd.build). "
            "There is no fallback implementation.")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.moe_abi_version() != ABI_VERSION:
        raise ImportError(f"libmoe_int8 ABI version {lib.moe_abi_version()} != {ABI_VERSION}")
    _lib = lib
    return lib


def check(status: int) -> None:
    if status != MOE_OK:
        raise MoeError(status, _lib.moe_last_error().decode())
