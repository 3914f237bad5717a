"""Python binding of libmoe_int8: argument marshalling only.

Each function takes torch tensors that already live on the current HIP device,
allocates the outputs (torch is the memory and stream provider), and calls the
C entry point of the same name on torch's current stream. Every step of the
layer runs in the library's kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import _lib
from ._lib import (MOE_ACT_AS_IS, MOE_ACT_INT8, MOE_BF16, MOE_F32, MOE_GROUP_MAX, MOE_GROUP_TOP2, MOE_MX_ROWS, MOE_MX_TILED,  # noqa: F401
                   MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_TILED, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MOE_W_BF16,
                   MOE_W_FP8, MOE_W_INT8, MOE_W_MXFP4, MoeError, MoeGate, MoePost, MoeShape)

_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


@dataclasses.dataclass
class Int8Experts:
    """Expert weights of one MoE layer as the FFN kernels read them.

    fmt MOE_W_INT8 (ExpertsInt8, the default): q_gate, q_up [E, f, d] int8 and
    q_down [E, d, f] int8 codes plus per-output-channel scales s_gate, s_up
    [E, f], s_down [E, d] (all fp32 or all bf16). fmt MOE_W_FP8: the same with
    OCP e4m3 codes (uint8 tensors). fmt MOE_W_BF16 (comparator): q_* are the
    bf16 weights themselves and s_* are None. Every q_* holds its bytes in the
    tiled layout of moe_pack_rows; the tensor shape is kept for the sizes.
    fmt MOE_W_MXFP4: q_* [E, out, in/2] uint8 (two codes a byte) and s_* [E, out,
    in/32] uint8 in the tiled layout of moe_quantize_mxfp4.
    """
    q_gate: torch.Tensor
    q_up: torch.Tensor
    q_down: torch.Tensor
    s_gate: Optional[torch.Tensor]
    s_up: Optional[torch.Tensor]
    s_down: Optional[torch.Tensor]
    fmt: int = MOE_W_INT8

    @property
    def E(self) -> int:
        return self.q_gate.shape[0]

    @property
    def f(self) -> int:
        return self.q_gate.shape[1]

    @property
    def d(self) -> int:
        return self.q_gate.shape[2] * (2 if self.fmt == MOE_W_MXFP4 else 1)

    @property
    def scale_dtype(self) -> torch.dtype:
        if self.fmt == MOE_W_MXFP4:
            return torch.bfloat16   # not used: the scales are bytes
        return self.s_gate.dtype if self.s_gate is not None else torch.bfloat16


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe_int8 must be contiguous")
    return t.data_ptr()


def _stream():
    # the handle alone: torch.cuda.current_stream() builds an object a call (1.5 us)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dtype_code(dt: torch.dtype) -> int:
    if dt not in _DT:
        raise TypeError(f"unsupported dtype {dt}")
    return _DT[dt]


def _check_width(name: str, have: int, want: int) -> None:
    if have != want:
        raise ValueError(f"{name} has {have} columns, the experts' weights {want}")


def _check_sizes(*sizes: int) -> None:
    """The library takes sizes of 32 bits; a larger one would be cut, not refused, on the way to it."""
    for v in sizes:
        if v >> 31 > 0:
            raise ValueError(f"size {v} is past 2^31")


# type of the codes; codes a byte; columns a scale covers (0: the row)
_CODES = {MOE_W_INT8: (torch.int8, 1, 0), MOE_W_FP8: (torch.uint8, 1, 0), MOE_W_BF16: (torch.bfloat16, 1, 0),
          MOE_W_MXFP4: (torch.uint8, 2, 32)}


def _weights(experts: Int8Experts, *names: str):
    """Pointers of the codes, then of the scales, of these matrices ("gate", "up", "down"): every tensor has
    the type and shape that the experts' sizes ask for, and is contiguous on the current device."""
    E, f, d, fmt = experts.E, experts.f, experts.d, experts.fmt
    if fmt not in _CODES:
        raise ValueError(f"unknown weight encoding {fmt}")
    code, per_byte, block = _CODES[fmt]
    scale = code if block else experts.scale_dtype
    ts = []
    for name in names:
        out, cols = (d, f) if name == "down" else (f, d)
        ts.append(("q_" + name, getattr(experts, "q_" + name), code, (E, out, cols // per_byte)))
    if fmt != MOE_W_BF16:
        for name in names:
            out, cols = (d, f) if name == "down" else (f, d)
            ts.append(("s_" + name, getattr(experts, "s_" + name), scale,
                       (E, out, cols // block) if block else (E, out)))
    for name, t, dtype, shape in ts:
        if t is None or t.dtype != dtype or t.shape != shape:
            have = None if t is None else f"{t.dtype} {tuple(t.shape)}"
            raise ValueError(f"the experts' {name} is {have}, not {dtype} {shape}")
    ptrs = [_arg(name, t, None) for name, t, _, _ in ts]
    return ptrs if fmt != MOE_W_BF16 else ptrs + [None] * len(names)


def _ffn_weights(experts: Int8Experts, *names: str):
    """_weights for MXFP4; the pointers as they are for the other encodings."""
    if experts.fmt == MOE_W_MXFP4:
        return _weights(experts, *names)
    return [_ptr(getattr(experts, k + name)) for k in ("q_", "s_") for name in names]


def make_shape(T: int, d: int, f: int, E: int, K: int, act: torch.dtype, scale: torch.dtype,
               path: int = MOE_PATH_AUTO, fmt: int = MOE_W_INT8) -> MoeShape:
    _check_sizes(T, d, f, E, K)
    return MoeShape(T, d, f, E, K, _dtype_code(act), _dtype_code(scale), path, fmt)


def _lib_handle():
    return _lib.load()


def workspace_size(shape: MoeShape) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def ffn_workspace_size(shape: MoeShape) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_ffn_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_route(x: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor], K: int):
    """Router + top-K gate. Returns (topk_ids int32 [T,K], topk_w fp32 [T,K])."""
    lib = _lib_handle()
    T, d = x.shape
    E = router_w.shape[0]
    shape = make_shape(T, d, 64, E, K, x.dtype, torch.float32)
    ids = torch.empty((T, K), dtype=torch.int32, device=x.device)
    w = torch.empty((T, K), dtype=torch.float32, device=x.device)
    _lib.check(lib.moe_route(ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(bias), _ptr(ids), _ptr(w),
                             _stream()))
    return ids, w


def moe_permute(topk_ids: torch.Tensor, E: int):
    """Returns (expert_offsets [E+1], sorted_slots [T*K], slot_to_row [T*K]), all int32."""
    lib = _lib_handle()
    T, K = topk_ids.shape
    shape = MoeShape(T, 64, 64, E, K, MOE_BF16, MOE_BF16, MOE_PATH_AUTO)
    dev = topk_ids.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_slots = torch.empty(T * K, dtype=torch.int32, device=dev)
    slot_to_row = torch.empty(T * K, dtype=torch.int32, device=dev)
    _lib.check(lib.moe_permute(ctypes.byref(shape), _ptr(topk_ids), _ptr(offsets), _ptr(sorted_slots),
                               _ptr(slot_to_row), _stream()))
    return offsets, sorted_slots, slot_to_row


def moe_expert_ffn(x: torch.Tensor, expert_offsets: torch.Tensor, sorted_slots: torch.Tensor,
                   experts: Int8Experts, K: int, path: int = MOE_PATH_AUTO,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expert SwiGLU FFNs on the permuted rows. Returns y_rows fp32 [T*K, d] (sorted-row order)."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    y_rows = torch.empty((T * K, d), dtype=torch.float32, device=x.device)
    need = ffn_workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_expert_ffn(
        ctypes.byref(shape), _ptr(x), _ptr(expert_offsets), _ptr(sorted_slots),
        *_ffn_weights(experts, "gate", "up", "down"), _ptr(y_rows), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream()))
    return y_rows


def gate_up_workspace_size(shape: MoeShape) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_gate_up_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_expert_gate_up(x: torch.Tensor, expert_offsets: torch.Tensor, sorted_slots: torch.Tensor,
                       experts: Int8Experts, K: int, path: int = MOE_PATH_AUTO,
                       h: Optional[torch.Tensor] = None, use_workspace: bool = True,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gate/up pass: h [T*K, f] bf16 (sorted-row order). With use_workspace the call
    gets the workspace it can use (`workspace` if given, else a new one: the tiled
    schedule's tile claim words); without it every tile follows the static order
    (same result, bit for bit)."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    if h is None:
        h = torch.empty((T * K, experts.f), dtype=torch.bfloat16, device=x.device)
    ws = None
    need = gate_up_workspace_size(shape) if use_workspace else 0
    if need:
        ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_expert_gate_up(
        ctypes.byref(shape), _ptr(x), _ptr(expert_offsets), _ptr(sorted_slots), *_ffn_weights(experts, "gate", "up"),
        _ptr(h), _ptr(ws),
        ctypes.c_size_t(ws.numel() if ws is not None else 0), _stream()))
    return h


def down_workspace_size(shape: MoeShape) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_down_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_expert_down(h: torch.Tensor, expert_offsets: torch.Tensor, experts: Int8Experts, T: int, K: int,
                    act: torch.dtype = torch.bfloat16, path: int = MOE_PATH_AUTO,
                    y_rows: Optional[torch.Tensor] = None, split_workspace: bool = True,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Down pass: y_rows [T*K, d] fp32 from h [T*K, f] bf16. With split_workspace the
    call gets the workspace it can use (`workspace` if given, else a new one: the
    stream schedule's partial sums of a split reduction, none for most stream
    shapes, or the tiled schedule's tile claim words); without it a split
    reduction stays inside one workgroup and tiles follow the static order (same
    result, bit for bit)."""
    lib = _lib_handle()
    have, need = h.numel(), T * K * experts.f   # h is read as T*K rows whatever its shape
    if have != need and (have < need or (h.dim() == 2 and h.shape[1] != experts.f)):
        raise ValueError(f"h has {have} numbers {tuple(h.shape)}, not {T * K} rows of {experts.f} columns")
    shape = make_shape(T, experts.d, experts.f, experts.E, K, act, experts.scale_dtype, path, experts.fmt)
    if y_rows is None:
        y_rows = torch.empty((T * K, experts.d), dtype=torch.float32, device=h.device)
    ws = None
    need = down_workspace_size(shape) if split_workspace else 0
    if need:
        ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=h.device)
    _lib.check(lib.moe_expert_down(ctypes.byref(shape), _ptr(h), _ptr(expert_offsets),
                                   *_ffn_weights(experts, "down"), _ptr(y_rows), _ptr(ws),
                                   ctypes.c_size_t(ws.numel() if ws is not None else 0), _stream()))
    return y_rows


def moe_combine(y_rows: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor,
                out_dtype: torch.dtype) -> torch.Tensor:
    """y[t] = sum_k topk_w[t,k] * y_rows[slot_to_row[t*K+k]]. Returns y [T, d] in out_dtype."""
    lib = _lib_handle()
    T, K = topk_w.shape
    d = y_rows.shape[1]
    shape = make_shape(T, d, 64, max(K, 1), K, out_dtype, torch.float32)
    y = torch.empty((T, d), dtype=out_dtype, device=y_rows.device)
    _lib.check(lib.moe_combine(ctypes.byref(shape), _ptr(y_rows), _ptr(slot_to_row), _ptr(topk_w), _ptr(y),
                               _stream()))
    return y


@dataclasses.dataclass
class Gate:
    """How a router's scores become the choice of experts and their weights (moe_route_gated).

    score MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID; select_bias [E] fp32 is added to
    the scores for the choice only (-inf takes an expert out of service); groups of
    E / groups consecutive experts, of which the group_topk of the largest value stay
    (group_by MOE_GROUP_MAX: the largest choice value of the group, MOE_GROUP_TOP2:
    the sum of its two largest); renorm: the weights are divided by their sum; scale
    multiplies them.
    """
    score: int = MOE_SCORE_SOFTMAX
    select_bias: Optional[torch.Tensor] = None
    groups: int = 1
    group_topk: int = 1
    group_by: int = MOE_GROUP_MAX
    renorm: bool = True
    scale: float = 1.0

    def struct(self, E: int) -> MoeGate:
        _check_sizes(self.groups, self.group_topk)
        return MoeGate(_arg("select_bias", self.select_bias, torch.float32, (E,)), self.score, self.groups,
                       self.group_topk, self.group_by, 1 if self.renorm else 0, self.scale)


class MoeLayer:
    """A resident MoE layer: router weights, int8 experts and a reusable workspace. With a gate the tokens are
    routed by it, and with act_int8 the experts' products take int8 activations (moe_forward_gated). A forward captured
    into a graph has a workspace of its own in the graph's memory: graphs neither share one nor lose it to a larger batch."""

    def __init__(self, router_w: torch.Tensor, bias: Optional[torch.Tensor], experts: Int8Experts, K: int,
                 gate: Optional[Gate] = None, act_int8: bool = False):
        self.router_w = router_w
        self.bias = bias
        self.experts = experts
        self.K = K
        self.gate = Gate() if gate is None and act_int8 else gate
        self.act_int8 = act_int8
        self._ws = None

    def workspace(self, shape: MoeShape) -> torch.Tensor:
        need = max(workspace_size(shape) if self.gate is None else gated_workspace_size(shape, self.act_int8), 256)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.router_w.device)
        return self._ws

    def forward(self, x: torch.Tensor, path: int = MOE_PATH_AUTO, y: Optional[torch.Tensor] = None,
                ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None):
        ws = None if torch.cuda.is_current_stream_capturing() else self.workspace(self.shape(x, path))
        if self.gate is not None:
            return moe_forward_gated(x, self.router_w, self.bias, self.experts, self.K, self.gate, self.act_int8,
                                     path=path, y=y, ids=ids, w=w, workspace=ws)
        return moe_forward(x, self.router_w, self.bias, self.experts, self.K, path=path, y=y, ids=ids, w=w, workspace=ws)

    def shape(self, x: torch.Tensor, path: int = MOE_PATH_AUTO) -> MoeShape:
        e = self.experts
        return make_shape(x.shape[0], x.shape[1], e.f, e.E, self.K, x.dtype, e.scale_dtype, path, e.fmt)


def moe_forward(x: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor], experts: Int8Experts,
                K: int, path: int = MOE_PATH_AUTO, y: Optional[torch.Tensor] = None,
                ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None):
    """The whole layer. Returns (y [T, d] in x.dtype, topk_ids [T, K], topk_w [T, K])."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    dev = x.device
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=dev)
    if ids is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(workspace_size(shape), 256), dtype=torch.uint8, device=dev)
    _lib.check(lib.moe_forward(
        ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(bias),
        *_ffn_weights(experts, "gate", "up", "down"), _ptr(y), _ptr(ids),
        _ptr(w), _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream()))
    return y, ids, w


def moe_forward_noalloc(x: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor],
                        experts: Int8Experts, K: int, path: int = MOE_PATH_AUTO, y: torch.Tensor = None,
                        ids: torch.Tensor = None, w: torch.Tensor = None):
    """The whole layer on the library's fixed per-GPU scratch (no workspace argument;
    the C call allocates nothing). Outputs y, ids and w must be given by the caller
    that cannot allocate; they are allocated here only when omitted."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    dev = x.device
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=dev)
    if ids is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
    _lib.check(lib.moe_forward_noalloc(
        ctypes.byref(shape), _ptr(x), _ptr(router_w), _ptr(bias),
        *_ffn_weights(experts, "gate", "up", "down"), _ptr(y), _ptr(ids),
        _ptr(w), _stream()))
    return y, ids, w


def moe_mlp_forward(x: torch.Tensor, experts: Int8Experts, path: int = MOE_PATH_AUTO,
                    y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense int8-weight SwiGLU MLP (one expert, E = K = 1). Returns y [T, d] in x.dtype."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    if experts.E != 1:
        raise ValueError("the dense MLP takes one expert (E = 1)")
    shape = make_shape(T, d, experts.f, 1, 1, x.dtype, experts.scale_dtype, path, experts.fmt)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=x.device)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _lib.check(lib.moe_mlp_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
        workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_mlp_forward(
        ctypes.byref(shape), _ptr(x), *_ffn_weights(experts, "gate", "up", "down"), _ptr(y), _ptr(workspace),
        ctypes.c_size_t(workspace.numel()), _stream()))
    return y


def moe_quantize_rows(w: torch.Tensor, scale_dtype: torch.dtype):
    """ExpertsInt8 quantizer on the GPU: w [..., cols] (fp32/bf16) -> (q int8 [..., cols], s [...])."""
    lib = _lib_handle()
    cols = w.shape[-1]
    rows = w.numel() // cols
    q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
    s = torch.empty(w.shape[:-1], dtype=scale_dtype, device=w.device)
    _lib.check(lib.moe_quantize_rows(ctypes.c_int64(rows), ctypes.c_int32(cols), _dtype_code(w.dtype), _ptr(w),
                                     _dtype_code(scale_dtype), _ptr(q), _ptr(s), _stream()))
    return q, s


def moe_quantize_rows_fp8(w: torch.Tensor, scale_dtype: torch.dtype):
    """FP8 comparator quantizer on the GPU: w [..., cols] -> (e4m3 code bytes uint8 [..., cols], s [...])."""
    lib = _lib_handle()
    cols = w.shape[-1]
    rows = w.numel() // cols
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty(w.shape[:-1], dtype=scale_dtype, device=w.device)
    _lib.check(lib.moe_quantize_rows_fp8(ctypes.c_int64(rows), ctypes.c_int32(cols), _dtype_code(w.dtype), _ptr(w),
                                         _dtype_code(scale_dtype), _ptr(q), _ptr(s), _stream()))
    return q, s


def moe_quantize_pack_rows(w: torch.Tensor, scale_dtype: torch.dtype, fmt: int = MOE_W_INT8):
    """Quantize w [..., rows, cols] (int8 or fp8 e4m3 codes) straight into the tiled layout:
    (codes [..., rows, cols] in the tiled byte order, scales [..., rows]), one pass."""
    lib = _lib_handle()
    cols = w.shape[-1]
    rows = w.numel() // cols
    q = torch.empty(w.shape, dtype=torch.int8 if fmt == MOE_W_INT8 else torch.uint8, device=w.device)
    s = torch.empty(w.shape[:-1], dtype=scale_dtype, device=w.device)
    _lib.check(lib.moe_quantize_pack_rows(ctypes.c_int64(rows), ctypes.c_int32(cols), _dtype_code(w.dtype), _ptr(w),
                                          _dtype_code(scale_dtype), ctypes.c_int32(fmt), _ptr(q), _ptr(s), _stream()))
    return q, s


def moe_pack_rows(q: torch.Tensor) -> torch.Tensor:
    """Row-major int8 codes [..., rows, cols] -> the tiled layout (same shape, permuted bytes)."""
    lib = _lib_handle()
    cols = q.shape[-1]
    rows = q.numel() // cols
    out = torch.empty_like(q)
    _lib.check(lib.moe_pack_rows(ctypes.c_int64(rows), ctypes.c_int32(cols), _ptr(q), _ptr(out), _stream()))
    return out


def pack_bf16_experts(w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor) -> Int8Experts:
    """bf16 expert weights (the unquantized comparator) -> the tiled layout of their bytes."""
    out = []
    for w in (w_gate, w_up, w_down):
        if w.dtype != torch.bfloat16:
            raise TypeError("pack_bf16_experts takes bf16 weights")
        b = w.contiguous().view(torch.int8)           # [..., rows, 2*cols] bytes
        out.append(moe_pack_rows(b).view(torch.bfloat16))
    return Int8Experts(out[0], out[1], out[2], None, None, None, fmt=MOE_W_BF16)


def pack_experts(q_gate: torch.Tensor, q_up: torch.Tensor, q_down: torch.Tensor, s_gate: torch.Tensor,
                 s_up: torch.Tensor, s_down: torch.Tensor) -> Int8Experts:
    """Row-major int8 codes + scales -> Int8Experts in the kernels' tiled layout."""
    return Int8Experts(moe_pack_rows(q_gate), moe_pack_rows(q_up), moe_pack_rows(q_down), s_gate, s_up, s_down)


def quantize_experts_fp8(w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                         scale_dtype: torch.dtype) -> Int8Experts:
    """FP8 comparator: quantize the (out, in) expert weights to e4m3 codes in the tiled layout (one pass)."""
    out, scales = [], []
    for w in (w_gate, w_up, w_down):
        q, s = moe_quantize_pack_rows(w, scale_dtype, MOE_W_FP8)
        out.append(q)
        scales.append(s)
    return Int8Experts(out[0], out[1], out[2], scales[0], scales[1], scales[2], fmt=MOE_W_FP8)


def quantize_experts(w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                     scale_dtype: torch.dtype) -> Int8Experts:
    """Load-time ExpertsInt8: quantize the (out, in) expert weights straight into the tiled layout (one pass)."""
    out = []
    scales = []
    for w in (w_gate, w_up, w_down):
        q, s = moe_quantize_pack_rows(w, scale_dtype, MOE_W_INT8)
        out.append(q)
        scales.append(s)
    return Int8Experts(out[0], out[1], out[2], scales[0], scales[1], scales[2])


# ---------------------------------------------------------------- MXFP4 and the norms around the layer

def _arg(name: str, t: Optional[torch.Tensor], dtype: Optional[torch.dtype], shape=None):
    """Pointer of a contiguous tensor of this type and shape on the current device (None: NULL)."""
    if t is None:
        return None
    # the device's index is looked up at the call: a torch without GPU support has no such function
    if ((dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape) and t.is_contiguous()
            and t.is_cuda and t.get_device() == torch._C._cuda_getDevice()):
        return t.data_ptr()
    if not t.is_cuda or t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, not on the current HIP device")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, not {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    raise ValueError("tensors passed to libmoe_int8 must be contiguous")


def moe_quantize_mxfp4(w: torch.Tensor, tiled: bool = False):
    """w [..., cols] (fp32/bf16) -> (codes uint8 [..., cols/2], scale bytes uint8 [..., cols/32]),
    row-major or in the tiled layout the kernels read weights in."""
    lib = _lib_handle()
    if w.dim() < 1 or w.shape[-1] % 32:
        raise ValueError(f"the last dimension of {tuple(w.shape)} is not a multiple of 32")
    cols = w.shape[-1]
    _check_sizes(cols)
    rows = w.numel() // cols if cols else 0
    q = torch.empty((*w.shape[:-1], cols // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((*w.shape[:-1], cols // 32), dtype=torch.uint8, device=w.device)
    _lib.check(lib.moe_quantize_mxfp4(rows, cols, _dtype_code(w.dtype), _arg("w", w, None),
                                      MOE_MX_TILED if tiled else MOE_MX_ROWS, _ptr(q), _ptr(s), _stream()))
    return q, s


def _mx_shape(q: torch.Tensor, s: torch.Tensor):
    cols = q.shape[-1] * 2
    if q.dim() < 1 or cols % 32 or tuple(s.shape) != (*q.shape[:-1], cols // 32):
        raise ValueError(f"codes {tuple(q.shape)} and scales {tuple(s.shape)} do not belong together")
    _check_sizes(cols)
    return (q.numel() // q.shape[-1] if cols else 0), cols


def moe_dequantize_mxfp4(q: torch.Tensor, s: torch.Tensor, dtype: torch.dtype, tiled: bool = False) -> torch.Tensor:
    """The numbers [..., cols] in `dtype` that codes and scales stand for."""
    lib = _lib_handle()
    rows, cols = _mx_shape(q, s)
    code = _dtype_code(dtype)
    w = torch.empty((*q.shape[:-1], cols), dtype=dtype, device=q.device)
    _lib.check(lib.moe_dequantize_mxfp4(rows, cols, MOE_MX_TILED if tiled else MOE_MX_ROWS,
                                        _arg("q", q, torch.uint8), _arg("s", s, torch.uint8), code, _ptr(w),
                                        _stream()))
    return w


def moe_pack_mxfp4(q: torch.Tensor, s: torch.Tensor):
    """Row-major codes and scales (a checkpoint's) -> (codes, scales) in the tiled layout, same shapes."""
    lib = _lib_handle()
    rows, cols = _mx_shape(q, s)
    qt, st = torch.empty_like(q), torch.empty_like(s)
    _lib.check(lib.moe_pack_mxfp4(rows, cols, _arg("q", q, torch.uint8), _arg("s", s, torch.uint8), _ptr(qt),
                                  _ptr(st), _stream()))
    return qt, st


def quantize_experts_mxfp4(w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor) -> Int8Experts:
    """Load time: (out, in) expert weights -> MXFP4 in the tiled layout (one pass)."""
    g, u, d = (moe_quantize_mxfp4(w, tiled=True) for w in (w_gate, w_up, w_down))
    return Int8Experts(g[0], u[0], d[0], g[1], u[1], d[1], fmt=MOE_W_MXFP4)


def pack_mxfp4_experts(q_gate: torch.Tensor, q_up: torch.Tensor, q_down: torch.Tensor, s_gate: torch.Tensor,
                       s_up: torch.Tensor, s_down: torch.Tensor) -> Int8Experts:
    """Row-major MXFP4 codes and scales -> Int8Experts in the kernels' tiled layout."""
    g, u, d = (moe_pack_mxfp4(q, s) for q, s in ((q_gate, s_gate), (q_up, s_up), (q_down, s_down)))
    return Int8Experts(g[0], u[0], d[0], g[1], u[1], d[1], fmt=MOE_W_MXFP4)


def moe_grouped_mm_mxfp4(a_q: torch.Tensor, a_s: torch.Tensor, expert_offsets: torch.Tensor, w_q: torch.Tensor,
                         w_s: torch.Tensor, out_dtype: torch.dtype, sorted_slots: Optional[torch.Tensor] = None,
                         K: int = 1, w2_q: Optional[torch.Tensor] = None, w2_s: Optional[torch.Tensor] = None,
                         path: int = MOE_PATH_AUTO, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Products grouped by expert, both operands in MXFP4.

    a_q [rows, d/2], a_s [rows, d/32] row-major; w_q [E, f, d/2], w_s [E, f, d/32]
    tiled. With sorted_slots [rows*K] sorted row r reads a's row
    sorted_slots[r] // K, else its own row r (K = 1). With w2_*: silu(W a) *
    (W2 a). Returns out [rows*K, f] in out_dtype (rows past the last segment are
    left as they are: uninitialised unless `out` is given)."""
    lib = _lib_handle()
    if a_q.dim() != 2 or w_q.dim() != 3:
        raise ValueError("a_q must be [rows, d/2] and w_q [E, f, d/2]")
    rows, d = a_q.shape[0], a_q.shape[1] * 2
    E, f = w_q.shape[0], w_q.shape[1]
    if sorted_slots is None and K != 1:
        raise ValueError("K is the slots per row of sorted_slots: 1 without it")
    if (w2_q is None) != (w2_s is None):
        raise ValueError("w2_q and w2_s are given together")
    _check_sizes(rows, d, f, E, K)
    shape = MoeShape(rows, d, f, E, K, _dtype_code(out_dtype), MOE_BF16, path, MOE_W_MXFP4)
    if out is None:
        out = torch.empty((rows * K, f), dtype=out_dtype, device=a_q.device)
    u8, w_shape, s_shape = torch.uint8, (E, f, d // 2), (E, f, d // 32)
    _lib.check(lib.moe_grouped_mm_mxfp4(
        ctypes.byref(shape), _arg("a_q", a_q, u8), _arg("a_s", a_s, u8, (rows, d // 32)),
        _arg("expert_offsets", expert_offsets, torch.int32, (E + 1,)),
        _arg("sorted_slots", sorted_slots, torch.int32, (rows * K,)), _arg("w_q", w_q, u8, w_shape),
        _arg("w_s", w_s, u8, s_shape), _arg("w2_q", w2_q, u8, w_shape), _arg("w2_s", w2_s, u8, s_shape),
        _arg("out", out, out_dtype, (rows * K, f)), _stream()))
    return out


def moe_expert_ffn_mxfp4(x: torch.Tensor, expert_offsets: torch.Tensor, sorted_slots: torch.Tensor,
                         experts: Int8Experts, K: int, path: int = MOE_PATH_AUTO,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expert SwiGLU FFNs with weights and activations in MXFP4. Returns y_rows fp32 [T*K, d]."""
    lib = _lib_handle()
    if experts.fmt != MOE_W_MXFP4:
        raise ValueError("the experts are not in MXFP4")
    T, d = x.shape
    _check_width("x", d, experts.d)
    weights = _weights(experts, "gate", "up", "down")
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_expert_ffn_mxfp4_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    y_rows = torch.empty((T * K, d), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_expert_ffn_mxfp4(
        ctypes.byref(shape), _arg("x", x, None),
        _arg("expert_offsets", expert_offsets, torch.int32, (experts.E + 1,)),
        _arg("sorted_slots", sorted_slots, torch.int32, (T * K,)), *weights, _ptr(y_rows),
        _arg("workspace", workspace, torch.uint8), ctypes.c_size_t(workspace.numel()), _stream()))
    return y_rows


# ---------------------------------------------------------------- gated routing, int8 activations

def moe_route_gated(x: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor], K: int, gate: Gate,
                    ids: Optional[torch.Tensor] = None, w: Optional[torch.Tensor] = None, use_workspace: bool = True,
                    workspace: Optional[torch.Tensor] = None):
    """Router with a Gate: x [T, d], router_w [E, d] (E up to 256), bias [E] fp32 added to the logits or None.
    Returns (topk_ids int32 [T, K], topk_w fp32 [T, K]); ids of -1 (weight 0) where fewer than K experts can
    be taken. With use_workspace the call gets the workspace it can use (`workspace` if given, else a new one:
    few tokens' rows are split over workgroups)."""
    lib = _lib_handle()
    T, d = x.shape
    E = router_w.shape[0]
    shape = make_shape(T, d, 64, E, K, x.dtype, torch.float32)
    g = gate.struct(E)
    dev = x.device
    if ids is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
    if use_workspace and workspace is None:
        n = ctypes.c_size_t(0)
        _lib.check(lib.moe_route_gated_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
        if n.value:
            workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    ws = workspace if use_workspace else None
    _lib.check(lib.moe_route_gated(ctypes.byref(shape), ctypes.byref(g), _arg("x", x, None),
                                   _arg("router_w", router_w, x.dtype, (E, d)), _arg("bias", bias, torch.float32, (E,)),
                                   _arg("ids", ids, torch.int32, (T, K)), _arg("w", w, torch.float32, (T, K)),
                                   _arg("workspace", ws, torch.uint8), 0 if ws is None else ws.numel(), _stream()))
    return ids, w


def moe_grouped_mm_int8(a_q: torch.Tensor, a_s: torch.Tensor, expert_offsets: torch.Tensor, w_q: torch.Tensor,
                        w_s: torch.Tensor, out_dtype: torch.dtype, sorted_slots: Optional[torch.Tensor] = None,
                        K: int = 1, w2_q: Optional[torch.Tensor] = None, w2_s: Optional[torch.Tensor] = None,
                        path: int = MOE_PATH_AUTO, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Products grouped by expert of int8 rows and int8 matrices, with a scale for each row and each channel.

    a_q [rows, d] int8, a_s [rows] fp32 (moe_quantize_rows with fp32 scales); w_q
    [E, f, d] tiled codes (moe_pack_rows), w_s [E, f] fp32 or bf16. With sorted_slots
    [rows*K] sorted row r reads a's row sorted_slots[r] // K, else its own row r (K =
    1). With w2_*: silu(W a) * (W2 a). Returns out [rows*K, f] in out_dtype (rows past
    the last segment are left as they are: uninitialised unless `out` is given)."""
    lib = _lib_handle()
    if a_q.dim() != 2 or w_q.dim() != 3:
        raise ValueError("a_q must be [rows, d] and w_q [E, f, d]")
    rows, d = a_q.shape
    E, f = w_q.shape[0], w_q.shape[1]
    if sorted_slots is None and K != 1:
        raise ValueError("K is the slots per row of sorted_slots: 1 without it")
    if (w2_q is None) != (w2_s is None):
        raise ValueError("w2_q and w2_s are given together")
    _check_sizes(rows, d, f, E, K)
    shape = MoeShape(rows, d, f, E, K, _dtype_code(out_dtype), _dtype_code(w_s.dtype), path, MOE_W_INT8)
    if out is None:
        out = torch.empty((rows * K, f), dtype=out_dtype, device=a_q.device)
    i8, i32, w_shape, s_shape = torch.int8, torch.int32, (E, f, d), (E, f)
    _lib.check(lib.moe_grouped_mm_int8(
        ctypes.byref(shape), _arg("a_q", a_q, i8), _arg("a_s", a_s, torch.float32, (rows,)),
        _arg("expert_offsets", expert_offsets, i32, (E + 1,)), _arg("sorted_slots", sorted_slots, i32, (rows * K,)),
        _arg("w_q", w_q, i8, w_shape), _arg("w_s", w_s, w_s.dtype, s_shape), _arg("w2_q", w2_q, i8, w_shape),
        _arg("w2_s", w2_s, w_s.dtype, s_shape), _arg("out", out, out_dtype, (rows * K, f)), _stream()))
    return out


def moe_expert_ffn_int8(x: torch.Tensor, expert_offsets: torch.Tensor, sorted_slots: torch.Tensor,
                        experts: Int8Experts, K: int, path: int = MOE_PATH_AUTO,
                        workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expert SwiGLU FFNs with weights and activations in int8. Returns y_rows fp32 [T*K, d]."""
    lib = _lib_handle()
    if experts.fmt != MOE_W_INT8:
        raise ValueError("the experts are not in int8")
    T, d = x.shape
    _check_width("x", d, experts.d)
    weights = _weights(experts, "gate", "up", "down")
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_expert_ffn_int8_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    y_rows = torch.empty((T * K, d), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(n.value, 256), dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_expert_ffn_int8(
        ctypes.byref(shape), _arg("x", x, None),
        _arg("expert_offsets", expert_offsets, torch.int32, (experts.E + 1,)),
        _arg("sorted_slots", sorted_slots, torch.int32, (T * K,)), *weights, _ptr(y_rows),
        _arg("workspace", workspace, torch.uint8), ctypes.c_size_t(workspace.numel()), _stream()))
    return y_rows


def gated_workspace_size(shape: MoeShape, act_int8: bool = False) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_gated_workspace_size(ctypes.byref(shape), MOE_ACT_INT8 if act_int8 else MOE_ACT_AS_IS,
                                            ctypes.byref(n)))
    return n.value


def moe_forward_gated(x: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor], experts: Int8Experts,
                      K: int, gate: Gate, act_int8: bool = False, path: int = MOE_PATH_AUTO,
                      y: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
                      w: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The whole layer with a Gate, and with act_int8 the experts' products in int8 by int8 (int8 weights).
    Returns (y [T, d] in x.dtype, topk_ids [T, K], topk_w [T, K])."""
    lib = _lib_handle()
    T, d = x.shape
    _check_width("x", d, experts.d)
    weights = _weights(experts, "gate", "up", "down")
    shape = make_shape(T, d, experts.f, experts.E, K, x.dtype, experts.scale_dtype, path, experts.fmt)
    g = gate.struct(experts.E)
    need = gated_workspace_size(shape, act_int8)
    if y is None:
        y = torch.empty((T, d), dtype=x.dtype, device=x.device)
    if ids is None:
        ids = torch.empty((T, K), dtype=torch.int32, device=x.device)
    if w is None:
        w = torch.empty((T, K), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    _lib.check(lib.moe_forward_gated(
        ctypes.byref(shape), ctypes.byref(g), MOE_ACT_INT8 if act_int8 else MOE_ACT_AS_IS, _arg("x", x, None),
        _arg("router_w", router_w, x.dtype, (experts.E, d)), _arg("bias", bias, torch.float32, (experts.E,)), *weights,
        _arg("y", y, x.dtype, (T, d)), _arg("ids", ids, torch.int32, (T, K)), _arg("w", w, torch.float32, (T, K)),
        _arg("workspace", workspace, torch.uint8), ctypes.c_size_t(workspace.numel()), _stream()))
    return y, ids, w


def moe_norm_pre(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """RMS norm before the layer: x / sqrt(mean(x^2) + eps) * weight, [T, d] in x.dtype. out may be x."""
    lib = _lib_handle()
    T, d = x.shape
    shape = make_shape(T, d, 64, 1, 1, x.dtype, torch.float32)
    if out is None:
        out = torch.empty_like(x)
    _lib.check(lib.moe_norm_pre(ctypes.byref(shape), _arg("x", x, None), _arg("weight", weight, x.dtype, (d,)), eps,
                                _arg("out", out, x.dtype, (T, d)), _stream()))
    return out


def _post(T: int, d: int, dtype: torch.dtype, weight, gate, gate_tokens: int, residual_scale: float,
          block_scale: float, eps: float, next_weight, next_eps: Optional[float]) -> MoePost:
    # past T all tokens share one row, whatever its size; below 1 the library refuses it
    gate_tokens = min(max(gate_tokens, 0), 0x7fffffff)
    rows = (-(-T // gate_tokens), d) if gate_tokens >= 1 else None
    return MoePost(_arg("weight", weight, dtype, (d,)), _arg("gate", gate, dtype, rows),
                   _arg("next_weight", next_weight, dtype, (d,)), gate_tokens, residual_scale, block_scale, eps,
                   eps if next_eps is None else next_eps)


def _post_outputs(residual, out, next_weight, next_out):
    if out is None:
        out = torch.empty_like(residual)
    if next_weight is not None and next_out is None:
        next_out = torch.empty_like(residual)
    return out, next_out if next_weight is not None else None


def moe_norm_post(y: torch.Tensor, residual: torch.Tensor, weight: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, gate_tokens: int = 1, residual_scale: float = 1.0,
                  block_scale: float = 1.0, eps: float = 1e-6, next_weight: Optional[torch.Tensor] = None,
                  next_eps: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  next_out: Optional[torch.Tensor] = None):
    """After the layer, y [T, d] its output: out = residual_scale * residual + block_scale * gate *
    (rms(y) * weight), and with next_weight also next = rms(out) * next_weight, in one pass.

    Without weight y is not normalised; gate [ceil(T / gate_tokens), d] is shared by gate_tokens
    consecutive tokens a row (None: 1). Returns (out, next or None) in y.dtype; out may be residual or y."""
    lib = _lib_handle()
    T, d = y.shape
    shape = make_shape(T, d, 64, 1, 1, y.dtype, torch.float32)
    p = _post(T, d, y.dtype, weight, gate, gate_tokens, residual_scale, block_scale, eps, next_weight, next_eps)
    res = _arg("residual", residual, y.dtype, (T, d))
    out, nxt = _post_outputs(residual, out, next_weight, next_out)
    _lib.check(lib.moe_norm_post(ctypes.byref(shape), ctypes.byref(p), _arg("y", y, None), res,
                                 _arg("out", out, y.dtype, (T, d)), _arg("next_out", nxt, y.dtype, (T, d)),
                                 _stream()))
    return out, nxt


def moe_combine_post(y_rows: torch.Tensor, slot_to_row: torch.Tensor, topk_w: torch.Tensor, residual: torch.Tensor,
                     weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                     gate_tokens: int = 1, residual_scale: float = 1.0, block_scale: float = 1.0, eps: float = 1e-6,
                     next_weight: Optional[torch.Tensor] = None, next_eps: Optional[float] = None,
                     out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None):
    """moe_norm_post with y = sum_k topk_w[t, k] * y_rows[slot_to_row[t*K + k]] (as moe_combine, unrounded)."""
    lib = _lib_handle()
    T, K = topk_w.shape
    d = y_rows.shape[1]
    if slot_to_row.numel() != T * K:
        raise ValueError(f"slot_to_row has {slot_to_row.numel()} entries, not {T * K}")
    dt = residual.dtype
    shape = make_shape(T, d, 64, max(K, 1), K, dt, torch.float32)
    p = _post(T, d, dt, weight, gate, gate_tokens, residual_scale, block_scale, eps, next_weight, next_eps)
    res = _arg("residual", residual, dt, (T, d))
    out, nxt = _post_outputs(residual, out, next_weight, next_out)
    _lib.check(lib.moe_combine_post(
        ctypes.byref(shape), ctypes.byref(p), _arg("y_rows", y_rows, torch.float32, (T * K, d)),
        _arg("slot_to_row", slot_to_row, torch.int32), _arg("topk_w", topk_w, torch.float32), res,
        _arg("out", out, dt, (T, d)), _arg("next_out", nxt, dt, (T, d)), _stream()))
    return out, nxt


def block_workspace_size(shape: MoeShape) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_block_workspace_size(ctypes.byref(shape), ctypes.byref(n)))
    return n.value


def moe_block_forward(residual: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor],
                      experts: Int8Experts, K: int, pre_weight: Optional[torch.Tensor] = None, pre_eps: float = 1e-6,
                      x: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, gate_tokens: int = 1, residual_scale: float = 1.0,
                      block_scale: float = 1.0, eps: float = 1e-6, next_weight: Optional[torch.Tensor] = None,
                      next_eps: Optional[float] = None, path: int = MOE_PATH_AUTO,
                      out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None):
    """A block on the residual stream [T, d]: norm (pre_weight; or x, already normalised), the layer, then
    moe_combine_post. Returns (out, next or None, topk_ids [T, K], topk_w [T, K])."""
    lib = _lib_handle()
    T, d = residual.shape
    dt = residual.dtype
    _check_width("residual", d, experts.d)
    weights = _weights(experts, "gate", "up", "down")
    shape = make_shape(T, d, experts.f, experts.E, K, dt, experts.scale_dtype, path, experts.fmt)
    p = _post(T, d, dt, weight, gate, gate_tokens, residual_scale, block_scale, eps, next_weight, next_eps)
    res = _arg("residual", residual, dt)
    out, nxt = _post_outputs(residual, out, next_weight, next_out)
    ids = torch.empty((T, K), dtype=torch.int32, device=residual.device)
    w = torch.empty((T, K), dtype=torch.float32, device=residual.device)
    need = block_workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=residual.device)
    _lib.check(lib.moe_block_forward(
        ctypes.byref(shape), res, _arg("pre_weight", pre_weight, dt, (d,)), pre_eps, _arg("x", x, dt, (T, d)),
        ctypes.byref(p), _arg("router_w", router_w, dt, (experts.E, d)),
        _arg("bias", bias, torch.float32, (experts.E,)), *weights, _arg("out", out, dt, (T, d)),
        _arg("next_out", nxt, dt, (T, d)), _ptr(ids), _ptr(w),
        _arg("workspace", workspace, torch.uint8), ctypes.c_size_t(workspace.numel()), _stream()))
    return out, nxt, ids, w


def block_gated_workspace_size(shape: MoeShape, act_int8: bool = False) -> int:
    lib = _lib_handle()
    n = ctypes.c_size_t(0)
    _lib.check(lib.moe_block_gated_workspace_size(ctypes.byref(shape), MOE_ACT_INT8 if act_int8 else MOE_ACT_AS_IS,
                                                  ctypes.byref(n)))
    return n.value


def moe_block_forward_gated(residual: torch.Tensor, router_w: torch.Tensor, bias: Optional[torch.Tensor],
                            experts: Int8Experts, K: int, route: Gate, act_int8: bool = False,
                            pre_weight: Optional[torch.Tensor] = None, pre_eps: float = 1e-6,
                            x: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                            gate: Optional[torch.Tensor] = None, gate_tokens: int = 1, residual_scale: float = 1.0,
                            block_scale: float = 1.0, eps: float = 1e-6, next_weight: Optional[torch.Tensor] = None,
                            next_eps: Optional[float] = None, path: int = MOE_PATH_AUTO,
                            out: Optional[torch.Tensor] = None, next_out: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """moe_block_forward with the layer of moe_forward_gated; `route` is its Gate, `gate` the factor of the
    layer's output as there. Returns (out, next or None, topk_ids [T, K], topk_w [T, K])."""
    lib = _lib_handle()
    T, d = residual.shape
    dt = residual.dtype
    _check_width("residual", d, experts.d)
    weights = _weights(experts, "gate", "up", "down")
    shape = make_shape(T, d, experts.f, experts.E, K, dt, experts.scale_dtype, path, experts.fmt)
    g = route.struct(experts.E)
    p = _post(T, d, dt, weight, gate, gate_tokens, residual_scale, block_scale, eps, next_weight, next_eps)
    res = _arg("residual", residual, dt)
    out, nxt = _post_outputs(residual, out, next_weight, next_out)
    ids = torch.empty((T, K), dtype=torch.int32, device=residual.device)
    w = torch.empty((T, K), dtype=torch.float32, device=residual.device)
    need = block_gated_workspace_size(shape, act_int8)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=residual.device)
    _lib.check(lib.moe_block_forward_gated(
        ctypes.byref(shape), ctypes.byref(g), MOE_ACT_INT8 if act_int8 else MOE_ACT_AS_IS, res,
        _arg("pre_weight", pre_weight, dt, (d,)), pre_eps, _arg("x", x, dt, (T, d)), ctypes.byref(p),
        _arg("router_w", router_w, dt, (experts.E, d)), _arg("bias", bias, torch.float32, (experts.E,)), *weights,
        _arg("out", out, dt, (T, d)), _arg("next_out", nxt, dt, (T, d)), _ptr(ids), _ptr(w),
        _arg("workspace", workspace, torch.uint8), ctypes.c_size_t(workspace.numel()), _stream()))
    return out, nxt, ids, w
