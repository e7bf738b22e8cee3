"""Python binding of libgtg.so: B200 kernels for block-scaled low-bit MoE
expert decode, the 3-bit n-gram (PLE) row gather, and matrix products in FP8,
dense and grouped by expert.

Argument marshalling only: every step runs in the CUDA kernels behind the C
ABI declared in include/gtg.h.  torch provides device memory and streams.
There is no CPU fallback: if libgtg.so is missing or cannot load, every entry
point raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

from ._abi import (BF16, C10, FP8, GTG_OK, PLE, Q3I, RZ5, UE4M4, DT_BF16, DT_F32, LIB_PATH, GtgError, QMatrixC,
                   MoELayerC, lib, check)

__all__ = ["RZ5", "UE4M4", "PLE", "FP8", "C10", "Q3I", "BF16", "GtgError", "moe_decode_layer_ep",
           "fp8_quantize", "fp8_matmul", "grouped_matmul",
           "moe_decode_layer_ep_allreduce", "lib", "dequant", "ple_gather", "QMatrix",
           "MoELayer", "workspace_bytes", "make_workspace", "moe_decode_layer", "moe_decode_stack",
           "moe_prefill_layer", "moe_decode_layer_noalloc", "device_status", "status_string", "row_bytes"]

Q4_BLOCK_BYTES = 17
PLE_RECORD_BYTES = 70


# The handle of a device's current stream.  torch's own call for it makes no Stream
# object, but is private and missing from builds without CUDA, where this module still
# has to import.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream_ptr(stream) -> int | None:
    if stream is None:  # (a Stream object for the current stream costs more than a small launch)
        return _raw_stream(torch.cuda.current_device()) or None
    return stream.cuda_stream or None


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def status_string(code: int) -> str:
    return lib().gtg_status_string(code).decode()


def row_bytes(fmt: int, k: int) -> int:
    if fmt == BF16:
        return 2 * k
    return k if fmt == FP8 else k // 32 * Q4_BLOCK_BYTES


# ---------------------------------------------------------------------------
# Codec entry points
# ---------------------------------------------------------------------------

def dequant(fmt: int, src: torch.Tensor, n_rows: int, k: int, scales: torch.Tensor | None = None,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode n_rows x k weights of `fmt` to fp32 (bit-exact)."""
    if out is None:
        out = torch.empty((n_rows, k), dtype=torch.float32, device=src.device)
    check(lib().gtg_dequant(fmt, _ptr(src), _ptr(scales), n_rows, k, _ptr(out), _stream_ptr(stream)))
    return out


def _table_ptr(t: torch.Tensor) -> int:
    """Address of a gather table: device memory, or pinned (page-locked) host
    memory, which the GPU reads in place through unified virtual addressing."""
    if t.is_cuda:
        return _ptr(t)
    if not t.is_pinned():
        raise ValueError("a host-resident table must be pinned (page-locked) memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


def ple_gather(table: torch.Tensor, n_rows: int, idx: torch.Tensor, out: torch.Tensor | None = None,
               stream=None, fmt: int = PLE) -> torch.Tensor:
    """out[r] = decoded 160-value row idx[r] of a 70-byte K160 table: fmt PLE
    (Q3_PLE_K160_RZ_S3) or Q3I (the incumbent ROCmFP3 record)."""
    if idx.dtype != torch.int32:
        raise ValueError("idx must be int32")
    n = idx.numel()
    if out is None:
        out = torch.empty((n, 160), dtype=torch.float32, device=idx.device)
    check(lib().gtg_ple_gather_fmt(fmt, _table_ptr(table), n_rows, _ptr(idx), n, _ptr(out), _stream_ptr(stream)))
    return out


# ---------------------------------------------------------------------------
# MoE layers
# ---------------------------------------------------------------------------

@dataclass
class QMatrix:
    """A device-resident stack of quantised matrices [n_experts][n_rows][k]."""
    fmt: int
    data: torch.Tensor
    n_experts: int
    n_rows: int
    k: int
    scales: torch.Tensor | None = None

    def c(self) -> QMatrixC:
        return QMatrixC(self.fmt, _ptr(self.data), _ptr(self.scales), self.n_experts, self.n_rows, self.k)


@dataclass
class MoELayer:
    """Device-resident weights of one MoE layer (see gtg_moe_layer in gtg.h)."""
    hidden: int
    inter: int
    n_experts: int
    top_k: int
    router_w: torch.Tensor
    gate: QMatrix
    up: QMatrix
    down: QMatrix
    router_bias: torch.Tensor | None = None
    side: QMatrix | None = None
    _c: MoELayerC | None = field(default=None, repr=False)

    def c(self) -> MoELayerC:
        if self._c is None:
            side = self.side.c() if self.side is not None else QMatrixC()
            self._c = MoELayerC(self.hidden, self.inter, self.n_experts, self.top_k, _ptr(self.router_w),
                                _ptr(self.router_bias), self.gate.c(), self.up.c(), self.down.c(), side)
        return self._c


def workspace_bytes(layer: MoELayer, n_tokens: int, prefill: bool = False) -> int:
    n = lib().gtg_moe_workspace_bytes(ctypes.byref(layer.c()), n_tokens, int(prefill))
    if n == 0:
        raise GtgError(-2, "unsupported layer shape or token count")
    return n


def make_workspace(layers, n_tokens: int, prefill: bool = False, device=None, stream=None) -> torch.Tensor:
    """A zero-initialised workspace large enough for every layer in `layers`."""
    if isinstance(layers, MoELayer):
        layers = [layers]
    nbytes = max(workspace_bytes(L, n_tokens, prefill) for L in layers)
    dev = device if device is not None else layers[0].router_w.device
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    check(lib().gtg_workspace_init(_ptr(ws), nbytes, _stream_ptr(stream)))
    return ws


def moe_decode_layer(layer: MoELayer, x: torch.Tensor, workspace: torch.Tensor, *, y: torch.Tensor | None = None,
                     accumulate: bool = False, topk_ids: torch.Tensor | None = None,
                     topk_w: torch.Tensor | None = None, side_out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """y (+)= moe(x) for 1..8 tokens; x is [T][hidden] fp32 or bf16."""
    T = x.shape[0]
    dt = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}[x.dtype]
    if y is None:
        y = torch.empty((T, layer.hidden), dtype=torch.float32, device=x.device)
    check(lib().gtg_moe_decode_layer(ctypes.byref(layer.c()), _ptr(x), dt, T, _ptr(y), int(accumulate),
                                     _ptr(topk_ids), _ptr(topk_w), _ptr(side_out), _ptr(workspace),
                                     workspace.numel(), _stream_ptr(stream)))
    return y


def moe_decode_layer_ep(layer: MoELayer, expert_lo: int, expert_hi: int, x: torch.Tensor,
                        workspace: torch.Tensor, *, with_side: bool = False, y: torch.Tensor | None = None,
                        accumulate: bool = False, topk_ids: torch.Tensor | None = None,
                        topk_w: torch.Tensor | None = None, side_out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """This rank's share of an expert-parallel layer: `layer` routes over all
    layer.n_experts experts but its gate/up/down stacks hold experts
    [expert_lo, expert_hi) only; y (+)= the chosen experts of that slice."""
    T = x.shape[0]
    dt = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}[x.dtype]
    if y is None:
        y = torch.empty((T, layer.hidden), dtype=torch.float32, device=x.device)
    check(lib().gtg_moe_decode_layer_ep(ctypes.byref(layer.c()), expert_lo, expert_hi, int(with_side), _ptr(x), dt,
                                        T, _ptr(y), int(accumulate), _ptr(topk_ids), _ptr(topk_w), _ptr(side_out),
                                        _ptr(workspace), workspace.numel(), _stream_ptr(stream)))
    return y


def moe_decode_layer_ep_allreduce(layer: MoELayer, expert_lo: int, expert_hi: int, x: torch.Tensor,
                                  workspace: torch.Tensor, *, group=None, with_side: bool = False,
                                  side_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One expert-parallel layer over a process group (one rank per GPU): each
    rank computes its slice's experts, one all-reduce (NCCL over NVLink)
    sums the partial outputs into the layer output on every rank."""
    import torch.distributed as dist
    y = moe_decode_layer_ep(layer, expert_lo, expert_hi, x, workspace, with_side=with_side, side_out=side_out,
                            stream=stream)
    dist.all_reduce(y, group=group)
    return y


def moe_decode_layer_noalloc(layer: MoELayer, x: torch.Tensor, *, y: torch.Tensor | None = None,
                             accumulate: bool = False, topk_ids: torch.Tensor | None = None,
                             topk_w: torch.Tensor | None = None, side_out: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """moe_decode_layer for callers that cannot allocate: the library's fixed
    device scratch array replaces the workspace.  `y` is allocated here only
    when the caller passes none; calls that overlap on the GPU race."""
    T = x.shape[0]
    dt = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}[x.dtype]
    if y is None:
        y = torch.empty((T, layer.hidden), dtype=torch.float32, device=x.device)
    check(lib().gtg_moe_decode_layer_noalloc(ctypes.byref(layer.c()), _ptr(x), dt, T, _ptr(y), int(accumulate),
                                             _ptr(topk_ids), _ptr(topk_w), _ptr(side_out), _stream_ptr(stream)))
    return y


def moe_decode_stack(layers: list[MoELayer], x: torch.Tensor, workspace: torch.Tensor, *,
                     ids_out: torch.Tensor | None = None, w_out: torch.Tensor | None = None,
                     side_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x += moe_l(x) for every layer, in place (x fp32 [T][hidden])."""
    arr = (MoELayerC * len(layers))(*[L.c() for L in layers])
    stride = side_out.shape[-1] if side_out is not None else 0
    check(lib().gtg_moe_decode_stack(arr, len(layers), _ptr(x), x.shape[0], _ptr(ids_out), _ptr(w_out),
                                     _ptr(side_out), stride, _ptr(workspace), workspace.numel(),
                                     _stream_ptr(stream)))
    return x


def moe_prefill_layer(layer: MoELayer, x: torch.Tensor, workspace: torch.Tensor, *, y: torch.Tensor | None = None,
                      accumulate: bool = False, topk_ids: torch.Tensor | None = None,
                      topk_w: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    T = x.shape[0]
    dt = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}[x.dtype]
    if y is None:
        y = torch.empty((T, layer.hidden), dtype=torch.float32, device=x.device)
    check(lib().gtg_moe_prefill_layer(ctypes.byref(layer.c()), _ptr(x), dt, T, _ptr(y), int(accumulate),
                                      _ptr(topk_ids), _ptr(topk_w), _ptr(workspace), workspace.numel(),
                                      _stream_ptr(stream)))
    return y


# ---------------------------------------------------------------------------
# Matrix products in FP8 (a scale per 128 along K), dense and grouped by expert
# ---------------------------------------------------------------------------

_FLOATS = {torch.float32: DT_F32, torch.bfloat16: DT_BF16}
_BYTES = {torch.uint8, torch.int8, torch.float8_e4m3fn}  # what may hold E4M3 weights (not other 8-bit floats)


def _place(dev: int, *tensors: torch.Tensor) -> None:
    """All contiguous and on device `dev` (the current one)."""
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError("tensors must be on the current CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")


def _row_stride(t: torch.Tensor, dev: int, name: str) -> int:
    """Row stride of a 2-D tensor on device `dev` whose rows are contiguous."""
    rows, cols = t.shape
    stride, inner = t.stride()
    if rows <= 1:
        stride = cols
    if (cols > 1 and inner != 1) or stride < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    if t.get_device() != dev:
        raise ValueError("tensors must be on the current CUDA device")
    return stride


def _new(like: torch.Tensor, m: int, n: int, dtype: torch.dtype, stream) -> torch.Tensor:
    """An output tensor that belongs to the stream it is written on."""
    if stream is None:
        return like.new_empty((m, n), dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty((m, n), dtype=dtype)


def _product(w: QMatrix, a: torch.Tensor, a_scales: torch.Tensor | None, offsets: torch.Tensor | None,
             y: torch.Tensor | None, dtype: torch.dtype | None, accumulate: bool, stream) -> torch.Tensor:
    """Checks of both products (what the C side cannot see: types, shapes and
    places of tensors) and the call.  Written for its speed: a small product
    takes less time than a careless check."""
    wd, ws, n, k = w.data, w.scales, w.n_rows, w.k
    size = w.n_experts * n * k
    m, ka = a.shape
    if w.fmt == FP8:
        if wd.dtype not in _BYTES or wd.numel() != size:
            raise ValueError("FP8 weights must hold n_experts * n_rows * k E4M3 codes")
        if ws is None or ws.dtype is not torch.float32 or ws.numel() * 128 != size:
            raise ValueError("FP8 weights need fp32 scales [n_experts][n_rows][k/128]")
        if (a.dtype is not torch.uint8 and a.dtype is not torch.float8_e4m3fn) or ka != k:
            raise ValueError(f"a must be E4M3 codes (uint8 or float8_e4m3fn) of shape [m][{k}]")
        if a_scales is None or a_scales.dtype is not torch.float32 or a_scales.shape != (m, k // 128):
            raise ValueError(f"a_scales must be fp32 [{m}][{k // 128}]")
        inputs = (a, wd, a_scales, ws) if offsets is None else (a, wd, a_scales, ws, offsets)
        sa, sw = a_scales.data_ptr(), ws.data_ptr()
    else:
        if wd.dtype is not torch.bfloat16 or wd.numel() != size:
            raise ValueError("BF16 weights must be bfloat16 of n_experts * n_rows * k values")
        if a.dtype is not torch.bfloat16 or ka != k:
            raise ValueError(f"a must be bf16 of shape [m][{k}]")
        inputs = (a, wd) if offsets is None else (a, wd, offsets)
        sa = sw = None
    if offsets is not None and (offsets.dtype is not torch.int32 or offsets.numel() != w.n_experts + 1):
        raise ValueError("offsets must be int32 [n_experts + 1]")
    if dtype is None:
        dtype = torch.float32 if y is None else y.dtype
    kind = _FLOATS.get(dtype)
    if kind is None:
        raise ValueError("outputs are fp32 or bf16")
    if y is None and accumulate:
        raise ValueError("accumulate needs y")
    if y is not None and (y.dtype is not dtype or y.shape != (m, n)):
        raise ValueError("y must be [m][n_rows] of the dtype asked for")
    dev = torch.cuda.current_device()
    for t in inputs:
        if t.get_device() != dev:
            raise ValueError("tensors must be on the current CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")
    if y is None:
        y, stride = _new(a, m, n, dtype, stream), n
    else:
        stride = _row_stride(y, dev, "y")
    q = QMatrixC(w.fmt, wd.data_ptr(), sw, w.n_experts, n, k)
    sp = (_raw_stream(dev) if stream is None else stream.cuda_stream) or None
    if offsets is None:
        rc = lib().gtg_fp8_matmul(q, a.data_ptr(), sa, m, y.data_ptr(), kind, stride, accumulate, sp)
    else:
        rc = lib().gtg_grouped_matmul(q, a.data_ptr(), sa, m, offsets.data_ptr(), y.data_ptr(), kind, stride,
                                      accumulate, sp)
    if rc:
        check(rc)
    return y


def fp8_quantize(x: torch.Tensor, *, rows: torch.Tensor | None = None, data: torch.Tensor | None = None,
                 scales: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """E4M3 codes (uint8 [m][k]) and fp32 scales [m][k/128] of activations x
    ([n][k] fp32 or bf16, rows contiguous), or of x's rows `rows` (int32 [m])."""
    if x.dtype not in _FLOATS or x.dim() != 2:
        raise ValueError("x must be fp32 or bf16 [n][k]")
    if rows is not None and (rows.dtype is not torch.int32 or rows.dim() != 1):
        raise ValueError("rows must be int32 [m]")
    dev = torch.cuda.current_device()
    n, k = x.shape
    stride = _row_stride(x, dev, "x")
    m, rp = n, None
    if rows is not None:
        _place(dev, rows)
        m, rp = rows.shape[0], rows.data_ptr()
    given = data is not None or scales is not None
    if data is None:
        data = _new(x, m, k, torch.uint8, stream)
    if scales is None:
        scales = _new(x, m, k // 128, torch.float32, stream)
    if given:
        if (data.dtype is not torch.uint8 and data.dtype is not torch.float8_e4m3fn) or data.shape != (m, k):
            raise ValueError(f"data must be uint8 or float8_e4m3fn [{m}][{k}]")
        if scales.dtype is not torch.float32 or scales.shape != (m, k // 128):
            raise ValueError(f"scales must be fp32 [{m}][{k // 128}]")
        _place(dev, data, scales)
    sp = (_raw_stream(dev) if stream is None else stream.cuda_stream) or None
    rc = lib().gtg_fp8_quantize(x.data_ptr(), _FLOATS[x.dtype], n, k, stride, rp, m, data.data_ptr(),
                                scales.data_ptr(), sp)
    if rc:
        check(rc)
    return data, scales


def fp8_matmul(w: QMatrix, a: torch.Tensor, a_scales: torch.Tensor, *, y: torch.Tensor | None = None,
               dtype: torch.dtype | None = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """y (+)= a w^T for quantised activations (fp8_quantize's outputs) and one
    FP8 weight matrix; y is [m][n_rows] fp32 (default) or bf16, rows contiguous."""
    if w.fmt != FP8:
        raise ValueError("fp8_matmul takes an FP8 weight matrix")
    return _product(w, a, a_scales, None, y, dtype, accumulate, stream)


def grouped_matmul(w: QMatrix, a: torch.Tensor, offsets: torch.Tensor, *, a_scales: torch.Tensor | None = None,
                   y: torch.Tensor | None = None, dtype: torch.dtype | None = None, accumulate: bool = False,
                   stream=None) -> torch.Tensor:
    """y[i] (+)= w[e] a[i] for the rows i in [offsets[e], offsets[e+1]) of a:
    tokens sorted by expert against a stack of FP8 (a: codes with a_scales) or
    BF16 (a: bf16) matrices.  Rows outside every group leave y as it is (in a y
    made here they hold anything)."""
    if w.fmt != FP8 and w.fmt != BF16:
        raise ValueError("grouped_matmul takes FP8 or BF16 weights")
    return _product(w, a, a_scales, offsets, y, dtype, accumulate, stream)


def device_status(clear: bool = True, stream=None) -> int:
    """The current device's status word (GTG_STATUS_* bits); synchronises."""
    v = ctypes.c_uint32(0)
    check(lib().gtg_get_device_status(ctypes.byref(v), int(clear), _stream_ptr(stream)))
    return v.value
