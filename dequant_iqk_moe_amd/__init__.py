"""IQ_K routed-expert kernels for MI355X -- thin Python binding over ``libiqk.so``.

Every call here is argument marshalling for the C ABI declared in
``include/iqk.h`` (same names without the ``iqk_`` prefix).  All arithmetic
runs in the library's HIP kernels (or its host relayout); PyTorch supplies
device memory and the current stream only.  If ``libiqk.so`` has not been
built, importing this package raises ``ImportError`` -- there is no CPU
fallback.

Operations follow the "mlx-iqk" package description: the relayout of
"Format" (``pack_relayout`` / ``unpack_relayout``), the float32
reconstruction of "Format" (``dequant``), and the switch-linear call of
"Surface" (``moe_gemv`` for few token-expert pairs, ``moe_prefill`` =
``route`` + ``dequant`` + ``grouped_gemm`` for many).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import numpy as np
import torch
import torch.autograd.forward_ad as _forward_ad

__all__ = [
    "IQ2_KS", "IQ2_K", "IQ1_S_R4", "IqkError", "IqkValueError", "Weights",
    "row_bytes", "plane_offsets", "pack_relayout", "unpack_relayout", "dequant", "moe_gemv",
    "route", "grouped_gemm", "prefill_workspace_bytes", "moe_prefill", "floor_gemv",
    "floor_dequant", "stream_read", "stream_write", "library_path",
    "router_topk", "router_topk_grad", "Fp8Weights", "fp8_quantize", "fp8_linear",
    "fp8_linear_workspace_bytes", "moe_fp8", "moe_fp8_workspace_bytes", "fp8_path",
    "moe_sort", "moe_sort_workspace_bytes", "moe_unsort", "moe_unsort_grad", "Int8Weights", "int8_quantize", "int8_linear",
    "int8_linear_workspace_bytes", "int8_grouped", "int8_grouped_workspace_bytes", "int8_path",
    "block_norm", "block_norm_grad", "block_norm_grad_workspace_bytes",
]

IQ2_KS, IQ2_K, IQ1_S_R4 = 1, 2, 3
FORMAT_NAMES = {"iq2_ks": IQ2_KS, "iq2_k": IQ2_K, "iq1_s_r4": IQ1_S_R4}
_F32, _F16, _BF16, _E4M3, _INT8 = 0, 1, 2, 3, 4
_DT = {torch.float32: _F32, torch.float16: _F16, torch.bfloat16: _BF16}

_E_ARG, _E_FORMAT, _E_SHAPE, _E_WIDTH, _E_ROWS4, _E_SIZE, _E_TABLE, _E_HIP = -1, -2, -3, -4, -5, -6, -7, -8
_VALUE_ERRORS = {_E_ARG, _E_FORMAT, _E_SHAPE, _E_ROWS4, _E_SIZE}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libiqk.so")


class IqkError(RuntimeError):
    """Unsupported request (no instance for a width, table not int8-exact) or a HIP error."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"[iqk {code}] {msg}")
        self.code = code


class IqkValueError(ValueError):
    """Bad arguments: format, shape, sizes, row groups."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"[iqk {code}] {msg}")
        self.code = code


class _Weights(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("experts", ctypes.c_int64), ("out", ctypes.c_int64),
                ("in_", ctypes.c_int64), ("streams", ctypes.c_void_p), ("streams_bytes", ctypes.c_size_t)]


class _Fp8Weights(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int64), ("out", ctypes.c_int64), ("in_", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("codes_bytes", ctypes.c_size_t), ("scales", ctypes.c_void_p),
                ("scales_count", ctypes.c_size_t)]


class _Int8Weights(ctypes.Structure):
    _fields_ = _Fp8Weights._fields_


class _Block(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("eps", ctypes.c_float),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("next_weight", ctypes.c_void_p)]


def library_path() -> str:
    return _LIB_PATH


def _load():
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built; run `python dequant_iqk_moe_amd/build.py`")
    L = ctypes.CDLL(_LIB_PATH)
    p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    f32 = ctypes.c_float
    W, F, I, B = (ctypes.POINTER(c) for c in (_Weights, _Fp8Weights, _Int8Weights, _Block))
    sig = {
        "iqk_row_bytes": (sz, [i32, i64]),
        "iqk_plane_offsets": (i32, [i32, i64, i64, p, p]),
        "iqk_pack_relayout": (i32, [i32, p, sz, i64, i64, p, sz]),
        "iqk_unpack_relayout": (i32, [i32, p, sz, i64, i64, p, sz]),
        "iqk_dequant": (i32, [W, i64, i64, p, p, i32, p, p]),
        "iqk_moe_gemv": (i32, [W, p, p, p, i32, i32, p, i64, i32, p, p]),
        "iqk_moe_gemv_swiglu": (i32, [W, p, p, p, i32, i32, p, i64, i32, p, p]),
        "iqk_moe_gemv_combine": (i32, [W, p, p, p, i32, i32, p, p, i64, i32, p, p]),
        "iqk_moe_gemv_grouped_workspace": (i32, [W, i64, i32, p]),
        "iqk_moe_gemv_grouped": (i32, [W, p, p, p, i32, i32, p, i64, i32, i32, p, sz, p, p]),
        "iqk_moe_auto_workspace": (i32, [W, i64, i32, p]),
        "iqk_moe_auto": (i32, [W, p, p, p, i32, i32, p, i64, i32, p, sz, p, p, p]),
        "iqk_moe_auto_noalloc": (i32, [W, p, p, p, i32, i32, p, i64, i32, p, p, p]),
        "iqk_swiglu": (i32, [p, i64, i64, p, p]),
        "iqk_combine": (i32, [p, p, i64, i32, i64, p, p]),
        "iqk_route": (i32, [p, i64, i64, i32, p, p, p, p]),
        "iqk_grouped_gemm": (i32, [p, i64, i64, i64, p, i32, i64, i32, p, p, p, p]),
        "iqk_moe_prefill_workspace": (i32, [W, i64, i32, p]),
        "iqk_moe_prefill": (i32, [W, p, p, p, i32, p, i64, i32, i32, p, sz, p, p]),
        "iqk_moe_prefill_fused_workspace": (i32, [W, i64, i32, p]),
        "iqk_moe_prefill_fused": (i32, [W, p, p, p, i32, p, i64, i32, i32, p, sz, p, p]),
        "iqk_floor_gemv": (i32, [W, p, p, p, i32, i32, p, i64, i32, p, p]),
        "iqk_floor_dequant": (i32, [W, i64, i64, i32, p, p]),
        "iqk_stream_read": (i32, [p, sz, p, sz, p]),
        "iqk_stream_write": (i32, [p, sz, ctypes.c_uint32, i32, p]),
        "iqk_router_topk": (i32, [p, i32, i64, i64, i32, i32, p, i32, i32, i32, i32, f32, p, p, p]),
        "iqk_router_topk_grad": (i32, [p, i32, p, p, i64, i64, i32, i32, i32, f32, p, p]),
        "iqk_fp8_quantize": (i32, [p, i32, i64, i64, p, p, p]),
        "iqk_fp8_linear_workspace": (i32, [F, i64, p]),
        "iqk_fp8_linear": (i32, [F, p, i32, p, i64, p, sz, p, i32, p]),
        "iqk_fp8_path": (i32, [F, i64, i32, i32, p]),
        "iqk_moe_fp8_workspace": (i32, [F, i64, i32, i32, p]),
        "iqk_moe_fp8": (i32, [F, p, i32, p, i32, p, i64, i32, i32, p, sz, p, i32, p]),
        "iqk_moe_sort_workspace": (i32, [i64, i32, i64, p]),
        "iqk_moe_sort": (i32, [p, i32, p, i64, i32, i64, i64, p, sz, p, p, p, p]),
        "iqk_moe_unsort": (i32, [p, i32, p, p, i64, i32, i64, p, i32, p]),
        "iqk_moe_unsort_grad": (i32, [p, i32, p, i32, p, p, i64, i32, i64, p, p, p]),
        "iqk_int8_quantize": (i32, [p, i32, i64, i64, p, p, p]),
        "iqk_int8_linear_workspace": (i32, [I, i64, i32, p]),
        "iqk_int8_linear": (i32, [I, p, i32, p, i64, p, sz, p, i32, p]),
        "iqk_int8_grouped_workspace": (i32, [I, i64, i32, p]),
        "iqk_int8_grouped": (i32, [I, p, i32, p, p, i64, p, sz, p, i32, p]),
        "iqk_int8_path": (i32, [I, i64, i32, p]),
        "iqk_block_norm": (i32, [B, p, p, p]),
        "iqk_block_norm_grad_workspace": (i32, [B, p]),
        "iqk_block_norm_grad": (i32, [B, p, p, p, p, p, p, p, p, sz, p]),
        "iqk_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    return L


_lib = _load()


def _check(rc: int):
    if rc == 0:
        return
    msg = _lib.iqk_last_error().decode()
    if rc in _VALUE_ERRORS:
        raise IqkValueError(rc, msg)
    raise IqkError(rc, msg)


def _fmt(fmt) -> int:
    if isinstance(fmt, str):
        return FORMAT_NAMES[fmt.lower()]
    return int(fmt)


# the current stream's handle without the Stream object around it (3 us less per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


GRID_NUMEL = 2048 * 8  # the IQ1_S_R4 grid: 2048 entries of 8 int8 values


def _dev(t: torch.Tensor | None, what: str, dtype=None, numel: int | None = None):
    """Device pointer of a contiguous tensor, after checking its dtype and,
    when `numel` is given, its element count (the kernels read or write
    exactly that many elements; a shorter buffer would be overrun)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise IqkValueError(_E_ARG, f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise IqkValueError(_E_ARG, f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise IqkValueError(_E_ARG, f"{what} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise IqkValueError(_E_SIZE, f"{what} has {t.numel()} elements, expected {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _grid(grid: torch.Tensor | None):
    return _dev(grid, "grid", torch.int8, GRID_NUMEL)


def _ids(ids: torch.Tensor):
    if ids.dim() != 2:
        raise IqkValueError(_E_ARG, "ids must be [T, k]")
    return _dev(ids, "ids", torch.int32)


def _host_values(values):
    if values is None:
        return None, None
    v = np.ascontiguousarray(np.asarray(values, np.float32).ravel())
    if v.size != 8:
        raise IqkValueError(_E_ARG, "the value table has 8 entries")
    return v, v.ctypes.data_as(ctypes.c_void_p)


def row_bytes(fmt, n: int) -> int:
    return int(_lib.iqk_row_bytes(_fmt(fmt), n))


def plane_offsets(fmt, rows: int, n: int):
    off = (ctypes.c_int64 * 5)()
    tot = ctypes.c_int64()
    _check(_lib.iqk_plane_offsets(_fmt(fmt), rows, n, off, ctypes.byref(tot)))
    return list(off), tot.value


def pack_relayout(fmt, wire: np.ndarray, rows: int, n: int) -> np.ndarray:
    """Host relayout wire -> canonical streams (byte-exact permutation)."""
    w = np.ascontiguousarray(wire, np.uint8).ravel()
    out = np.empty(w.size, np.uint8)
    _check(_lib.iqk_pack_relayout(_fmt(fmt), w.ctypes.data_as(ctypes.c_void_p), w.size, rows, n,
                                  out.ctypes.data_as(ctypes.c_void_p), out.size))
    return out


def unpack_relayout(fmt, streams: np.ndarray, rows: int, n: int) -> np.ndarray:
    s = np.ascontiguousarray(streams, np.uint8).ravel()
    out = np.empty(s.size, np.uint8)
    _check(_lib.iqk_unpack_relayout(_fmt(fmt), s.ctypes.data_as(ctypes.c_void_p), s.size, rows, n,
                                    out.ctypes.data_as(ctypes.c_void_p), out.size))
    return out


@dataclass
class Weights:
    """Expert-stacked stream tensor: `experts` x [out, in_features] in one
    device uint8 tensor laid out as the canonical streams."""

    fmt: int
    experts: int
    out: int
    in_features: int
    streams: torch.Tensor

    @staticmethod
    def from_wire(fmt, experts: int, out: int, in_features: int, wire: np.ndarray, device="cuda") -> "Weights":
        s = pack_relayout(fmt, wire, experts * out, in_features)
        return Weights(_fmt(fmt), experts, out, in_features, torch.from_numpy(s).to(device))

    def _c(self) -> _Weights:
        if not self.streams.is_cuda or self.streams.dtype != torch.uint8 or not self.streams.is_contiguous():
            raise IqkValueError(_E_ARG, "streams must be a contiguous device uint8 tensor")
        return _Weights(_fmt(self.fmt), self.experts, self.out, self.in_features,
                        self.streams.data_ptr(), self.streams.numel())


def dequant(w: Weights, values=None, grid: torch.Tensor | None = None, out_dtype=torch.float32,
            row0: int = 0, nrows: int | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    nrows = w.experts * w.out - row0 if nrows is None else nrows
    if out is None:
        out = torch.empty((nrows, w.in_features), dtype=out_dtype, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    if out.dtype not in _DT:
        raise IqkValueError(_E_ARG, "out must be float32, float16 or bfloat16")
    _check(_lib.iqk_dequant(ctypes.byref(cw), row0, nrows, vp, _grid(grid),
                            _DT[out.dtype], _dev(out, "out", numel=nrows * w.in_features), _stream(stream)))
    return out


def _x_args(x: torch.Tensor, T: int, x_slots: int, n: int):
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise IqkValueError(_E_ARG, "x must be float32 or bfloat16")
    if x.numel() != T * x_slots * n:
        raise IqkValueError(_E_SIZE, f"x has {x.numel()} elements, expected T*x_slots*in = {T * x_slots * n}")
    return _dev(x, "x"), _DT[x.dtype]


def moe_gemv(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
             x_slots: int = 1, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fused decode matvec: y[T, k, out] (float32)."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if y is None:
        y = torch.empty((T, k, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_gemv(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                             _ids(ids), T, k, _dev(y, "y", torch.float32, T * k * w.out), _stream(stream)))
    return y


def moe_gemv_swiglu(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
                    x_slots: int = 1, h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gate/up matvec with the SwiGLU epilogue: h[T, k, out // 2] (bf16),
    h = silu(gate) * up with gate rows [0, I) and up rows [I, 2I)."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if h is None:
        h = torch.empty((T, k, w.out // 2), dtype=torch.bfloat16, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_gemv_swiglu(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                                    _ids(ids), T, k, _dev(h, "h", torch.bfloat16, T * k * (w.out // 2)),
                                    _stream(stream)))
    return h


def moe_gemv_combine(w: Weights, x: torch.Tensor, ids: torch.Tensor, route_w: torch.Tensor, values=None,
                     grid: torch.Tensor | None = None, x_slots: int | None = None, y: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Down matvec with the router-weighted combine: y[T, out] (float32),
    y[t] = sum_j route_w[t, j] * W_{ids[t, j]} x[t, j].  x_slots defaults to k."""
    T, k = ids.shape
    x_slots = k if x_slots is None else x_slots
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if y is None:
        y = torch.empty((T, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_gemv_combine(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                                     _ids(ids), _dev(route_w, "route_w", torch.float32, T * k), T, k,
                                     _dev(y, "y", torch.float32, T * w.out), _stream(stream)))
    return y


def gemv_grouped_workspace_bytes(w: Weights, T: int, k: int) -> int:
    b = ctypes.c_size_t()
    cw = _Weights(_fmt(w.fmt), w.experts, w.out, w.in_features, None, 0)
    _check(_lib.iqk_moe_gemv_grouped_workspace(ctypes.byref(cw), T, k, ctypes.byref(b)))
    return b.value


def moe_gemv_grouped(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
                     x_slots: int = 1, sorted: bool = False, workspace: torch.Tensor | None = None,
                     y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Grouped decode matvec: route, then one decode pass per selected expert
    shared by all of its pairs.  y[T, k, out] (float32); pairs with an
    invalid id get NaN rows."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if workspace is None:
        workspace = torch.empty(gemv_grouped_workspace_bytes(w, T, k), dtype=torch.uint8, device=w.streams.device)
    if y is None:
        y = torch.zeros((T, k, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_gemv_grouped(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                                     _ids(ids), T, k, int(bool(sorted)),
                                     _dev(workspace, "workspace", torch.uint8), workspace.numel(),
                                     _dev(y, "y", torch.float32, T * k * w.out), _stream(stream)))
    return y


def swiglu(y_gu: torch.Tensor, h: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """h = silu(gate) * up (bf16) from a gate/up projection's output
    y_gu [..., 2I] (float32; gate columns first)."""
    if y_gu.dtype != torch.float32 or y_gu.shape[-1] % 2:
        raise IqkValueError(_E_ARG, "y_gu must be float32 [..., 2I]")
    I = y_gu.shape[-1] // 2
    P = y_gu.numel() // (2 * I)
    if h is None:
        h = torch.empty((*y_gu.shape[:-1], I), dtype=torch.bfloat16, device=y_gu.device)
    _check(_lib.iqk_swiglu(_dev(y_gu, "y_gu", torch.float32), P, I, _dev(h, "h", torch.bfloat16, P * I),
                           _stream(stream)))
    return h


def combine(y: torch.Tensor, route_w: torch.Tensor, yc: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """yc[t] = sum_j route_w[t, j] * y[t, j] (float32, slot order) from y [T, k, out]."""
    T, k, out = y.shape
    if yc is None:
        yc = torch.empty((T, out), dtype=torch.float32, device=y.device)
    _check(_lib.iqk_combine(_dev(y, "y", torch.float32), _dev(route_w, "route_w", torch.float32, T * k), T, k, out,
                            _dev(yc, "yc", torch.float32, T * out), _stream(stream)))
    return yc


AUTO_PATHS = ("gemv", "grouped_gemv", "fused_prefill")


def moe_auto(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
             x_slots: int = 1, workspace: torch.Tensor | None = None, y: torch.Tensor | None = None,
             stream=None) -> tuple[torch.Tensor, str]:
    """The routed projection with the path picked by pairs per expert
    (per-pair matvec, grouped matvec or fused prefill); returns (y, path)."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if workspace is None:
        b = ctypes.c_size_t()
        cw0 = _Weights(_fmt(w.fmt), w.experts, w.out, w.in_features, None, 0)
        _check(_lib.iqk_moe_auto_workspace(ctypes.byref(cw0), T, k, ctypes.byref(b)))
        workspace = torch.empty(b.value, dtype=torch.uint8, device=w.streams.device)
    if y is None:
        y = torch.zeros((T, k, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    path = ctypes.c_int(-1)
    _check(_lib.iqk_moe_auto(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                             _ids(ids), T, k, _dev(workspace, "workspace", torch.uint8),
                             workspace.numel(), _dev(y, "y", torch.float32, T * k * w.out), ctypes.byref(path),
                             _stream(stream)))
    return y, AUTO_PATHS[path.value]


def moe_auto_noalloc(w: Weights, x: torch.Tensor, ids: torch.Tensor, y: torch.Tensor, values=None,
                     grid: torch.Tensor | None = None, x_slots: int = 1, stream=None) -> str:
    """moe_auto without a workspace and without any allocation: the
    library's fixed device scratch holds the routing arrays (calls that
    overlap on one GPU race).  y [T, k, out] float32 is the caller's;
    returns the path taken."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    _v, vp = _host_values(values)
    cw = w._c()
    path = ctypes.c_int(-1)
    _check(_lib.iqk_moe_auto_noalloc(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots, _ids(ids), T, k,
                                     _dev(y, "y", torch.float32, T * k * w.out), ctypes.byref(path),
                                     _stream(stream)))
    return AUTO_PATHS[path.value]


def floor_gemv(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
               x_slots: int = 1, sink: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Deleted-decode floor of moe_gemv (same loads; integer accumulator out)."""
    T, k = ids.shape
    xp, xdt = _x_args(x, T, x_slots, w.in_features)
    if sink is None:
        sink = torch.empty((T, k, w.out), dtype=torch.int32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_floor_gemv(ctypes.byref(cw), vp, _grid(grid), xp, xdt, x_slots,
                               _ids(ids), T, k, _dev(sink, "sink", torch.int32, T * k * w.out),
                               _stream(stream)))
    return sink


def floor_dequant(w: Weights, out_dtype=torch.bfloat16, row0: int = 0, nrows: int | None = None,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    nrows = w.experts * w.out - row0 if nrows is None else nrows
    if out is None:
        out = torch.empty((nrows, w.in_features), dtype=out_dtype, device=w.streams.device)
    cw = w._c()
    if out.dtype not in _DT:
        raise IqkValueError(_E_ARG, "out must be float32, float16 or bfloat16")
    _check(_lib.iqk_floor_dequant(ctypes.byref(cw), row0, nrows, _DT[out.dtype],
                                  _dev(out, "out", numel=nrows * w.in_features), _stream(stream)))
    return out


def stream_read(buf: torch.Tensor, sink: torch.Tensor, stream=None) -> torch.Tensor:
    nbytes = buf.numel() * buf.element_size()
    _check(_lib.iqk_stream_read(_dev(buf, "buf"), nbytes, _dev(sink, "sink", torch.int32), sink.numel(),
                                _stream(stream)))
    return sink


def stream_write(buf: torch.Tensor, value: int = 0, runs: int = 1, stream=None) -> torch.Tensor:
    """Plain streaming write of `value` into every 32-bit word of buf (the
    write ceiling of the dequantization producer); each wave writes `runs`
    consecutive 1 KiB runs (1: the fastest shape, 8: the bf16 producer's)."""
    nbytes = buf.numel() * buf.element_size()
    _check(_lib.iqk_stream_write(_dev(buf, "buf"), nbytes, int(value) & 0xFFFFFFFF, int(runs), _stream(stream)))
    return buf


def route(ids: torch.Tensor, E: int, sorted: bool = False, stream=None):
    """Stable expert sort of the pairs: (counts[E], offsets[E+1], perm[P]) int32 device tensors."""
    P = ids.numel()
    dev = ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(P, 1), dtype=torch.int32, device=dev)
    _check(_lib.iqk_route(_dev(ids, "ids", torch.int32), P, E, int(bool(sorted)), _dev(counts, "counts"),
                          _dev(offsets, "offsets"), _dev(perm, "perm"), _stream(stream)))
    return counts, offsets, perm[:P]


def grouped_gemm(W: torch.Tensor, x: torch.Tensor, T: int, k: int, offsets: torch.Tensor, perm: torch.Tensor,
                 x_slots: int = 1, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """MFMA grouped GEMM over dense bf16 experts W [E, out, in] for routed pairs."""
    E, out, n = W.shape
    if x.dtype != torch.bfloat16 or x.numel() != T * x_slots * n:
        raise IqkValueError(_E_SIZE, "x must be bf16 [T, x_slots, in]")
    if y is None:
        y = torch.zeros((T, k, out), dtype=torch.float32, device=W.device)
    if perm.numel() < T * k:
        raise IqkValueError(_E_SIZE, f"perm has {perm.numel()} elements, expected at least T*k = {T * k}")
    _check(_lib.iqk_grouped_gemm(_dev(W, "W", torch.bfloat16), E, out, n, _dev(x, "x"), x_slots, T, k,
                                 _dev(offsets, "offsets", torch.int32, E + 1), _dev(perm, "perm", torch.int32),
                                 _dev(y, "y", torch.float32, T * k * out), _stream(stream)))
    return y


def prefill_workspace_bytes(w: Weights, T: int, k: int) -> int:
    b = ctypes.c_size_t()
    cw = _Weights(_fmt(w.fmt), w.experts, w.out, w.in_features, None, 0)
    _check(_lib.iqk_moe_prefill_workspace(ctypes.byref(cw), T, k, ctypes.byref(b)))
    return b.value


def moe_prefill(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
                x_slots: int = 1, sorted: bool = False, workspace: torch.Tensor | None = None,
                y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prefill: route + one-pass dequant of all experts to bf16 + MFMA grouped GEMM."""
    T, k = ids.shape
    if x.dtype != torch.bfloat16 or x.numel() != T * x_slots * w.in_features:
        raise IqkValueError(_E_SIZE, "x must be bf16 [T, x_slots, in]")
    if workspace is None:
        workspace = torch.empty(prefill_workspace_bytes(w, T, k), dtype=torch.uint8, device=w.streams.device)
    if y is None:
        y = torch.zeros((T, k, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_prefill(ctypes.byref(cw), vp, _grid(grid), _dev(x, "x"), x_slots,
                                _ids(ids), T, k, int(bool(sorted)),
                                _dev(workspace, "workspace", torch.uint8), workspace.numel(),
                                _dev(y, "y", torch.float32, T * k * w.out), _stream(stream)))
    return y


def prefill_fused_workspace_bytes(w: Weights, T: int, k: int) -> int:
    b = ctypes.c_size_t()
    cw = _Weights(_fmt(w.fmt), w.experts, w.out, w.in_features, None, 0)
    _check(_lib.iqk_moe_prefill_fused_workspace(ctypes.byref(cw), T, k, ctypes.byref(b)))
    return b.value


def moe_prefill_fused(w: Weights, x: torch.Tensor, ids: torch.Tensor, values=None, grid: torch.Tensor | None = None,
                      x_slots: int = 1, sorted: bool = False, workspace: torch.Tensor | None = None,
                      y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prefill with the dequantization fused into the MFMA grouped GEMM
    (route + one kernel; no dense weight copy)."""
    T, k = ids.shape
    if x.dtype != torch.bfloat16 or x.numel() != T * x_slots * w.in_features:
        raise IqkValueError(_E_SIZE, "x must be bf16 [T, x_slots, in]")
    if workspace is None:
        workspace = torch.empty(prefill_fused_workspace_bytes(w, T, k), dtype=torch.uint8, device=w.streams.device)
    if y is None:
        y = torch.zeros((T, k, w.out), dtype=torch.float32, device=w.streams.device)
    _v, vp = _host_values(values)
    cw = w._c()
    _check(_lib.iqk_moe_prefill_fused(ctypes.byref(cw), vp, _grid(grid), _dev(x, "x"), x_slots,
                                      _ids(ids), T, k, int(bool(sorted)),
                                      _dev(workspace, "workspace", torch.uint8), workspace.numel(),
                                      _dev(y, "y", torch.float32, T * k * w.out), _stream(stream)))
    return y


def _stream_object(stream):
    """The stream given as an object or as a handle.  The handle 0 is the default stream's (ExternalStream(0) is a new
    stream that nothing orders behind the others)."""
    if hasattr(stream, "cuda_stream"):
        return stream
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor of the stream the call runs on (the caching allocator may
    give a tensor's memory away while another stream still writes it)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream)):
        return torch.empty(shape, dtype=dtype, device=device)


# ---------------------------------------------------------------------------
# expert selection
# ---------------------------------------------------------------------------

_SCORING = {"softmax": 0, "sigmoid": 1}


def _scoring(name: str) -> int:
    if name not in _SCORING:
        raise IqkValueError(_E_ARG, f"scoring must be one of {sorted(_SCORING)}, got {name!r}")
    return _SCORING[name]


def _logits(logits: torch.Tensor):
    if logits.dim() != 2 or logits.dtype not in _DT:
        raise IqkValueError(_E_ARG, "logits must be [T, E] in float32, float16 or bfloat16")
    return _dev(logits, "logits"), _DT[logits.dtype]


def router_topk(logits: torch.Tensor, k: int, scoring: str = "softmax", bias: torch.Tensor | None = None,
                n_group: int = 1, topk_group: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
                ids: torch.Tensor | None = None, weights: torch.Tensor | None = None, stream=None):
    """The k experts of each token and their weights, (ids int32 [T, k],
    weights float32 [T, k]), from router logits [T, E].  scoring: "softmax"
    or "sigmoid"; bias [E] (float32) shifts the choice only; n_group > 1 keeps
    the best topk_group groups of experts, by the best or (group_top=2) the
    best two of each; renorm divides the weights by their sum.  Where logits
    require a gradient the weights carry it (through router_topk_grad), as a
    new tensor over the caller's buffer if one is given."""
    lp, dt = _logits(logits)
    T, E = logits.shape
    if not 1 <= k <= E:
        raise IqkValueError(_E_ARG, f"k = {k} outside [1, {E}]")
    if getattr(_forward_ad, "_current_level", 0) >= 0:
        _refuse_tangents(logits)
    given = [t for t in (ids, weights) if t is not None]
    if ids is None:
        ids = _empty((T, k), torch.int32, logits.device, stream)
    if weights is None:
        weights = _empty((T, k), torch.float32, logits.device, stream)
    _check(_lib.iqk_router_topk(lp, dt, T, E, k, _scoring(scoring), _dev(bias, "bias", torch.float32, E), n_group,
                                topk_group, group_top, int(bool(renorm)), scale,
                                _dev(ids, "ids", torch.int32, T * k), _dev(weights, "weights", torch.float32, T * k),
                                _stream(stream)))
    for t in given:  # a gradient of an earlier call that still needs a caller's buffer can tell
        if not t.is_inference():
            torch.autograd.graph.increment_version(t)
    if logits.requires_grad and torch.is_grad_enabled():
        weights = _RouterWeights.apply(logits, ids, weights.detach(), scoring, renorm, scale)
    return ids, weights


class _RouterWeights(torch.autograd.Function):
    """Joins weights that router_topk has computed to the logits they came from."""

    @staticmethod
    def forward(ctx, logits, ids, weights, scoring, renorm, scale):
        ctx.save_for_backward(logits, ids)
        ctx.mark_dirty(weights)
        ctx.args = scoring, renorm, scale
        return weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_weights):
        logits, ids = ctx.saved_tensors
        return router_topk_grad(logits, ids, d_weights.contiguous(), *ctx.args), None, None, None, None, None


def router_topk_grad(logits: torch.Tensor, ids: torch.Tensor, d_weights: torch.Tensor, scoring: str = "softmax",
                     renorm: bool = True, scale: float = 1.0, d_logits: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Gradient of router_topk's weights with respect to the logits (of their
    dtype), the chosen ids held fixed."""
    lp, dt = _logits(logits)
    T, E = logits.shape
    ip = _ids(ids)
    if ids.shape[0] != T:
        raise IqkValueError(_E_SIZE, f"ids has {ids.shape[0]} rows, logits {T}")
    k = ids.shape[1]
    if d_logits is None:
        d_logits = _empty(logits.shape, logits.dtype, logits.device, stream)
    _check(_lib.iqk_router_topk_grad(lp, dt, ip, _dev(d_weights, "d_weights", torch.float32, T * k), T, E, k,
                                     _scoring(scoring), int(bool(renorm)), scale,
                                     _dev(d_logits, "d_logits", logits.dtype, T * E), _stream(stream)))
    return d_logits


# ---------------------------------------------------------------------------
# products in 8-bit floating point, a scale for each block of 128
# ---------------------------------------------------------------------------

_XDT = {**_DT, torch.float8_e4m3fn: _E4M3}


def _blocks(n: int) -> int:
    return -(-n // 128)


@dataclass
class Fp8Weights:
    """8-bit weights: codes [experts, out, in] (torch.float8_e4m3fn) with
    scales [experts, ceil(out / 128), ceil(in / 128)] (float32), one per
    128 x 128 block."""

    codes: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        if self.codes.dim() != 3 or self.codes.dtype != torch.float8_e4m3fn:
            raise IqkValueError(_E_ARG, "codes must be float8_e4m3fn [experts, out, in]")
        if self.codes.numel() == 0:
            raise IqkValueError(_E_ARG, "codes hold no values")
        self.experts, self.out, self.in_features = self.codes.shape
        if self.scales.dtype != torch.float32 or tuple(self.scales.shape) != (
                self.experts, _blocks(self.out), _blocks(self.in_features)):
            raise IqkValueError(_E_SIZE, "scales must be float32 [experts, ceil(out / 128), ceil(in / 128)]")

    def _c(self) -> _Fp8Weights:
        cp, sp = _dev(self.codes, "codes"), _dev(self.scales, "scales")
        return _Fp8Weights(self.experts, self.out, self.in_features, cp, self.codes.numel(), sp, self.scales.numel())


def fp8_quantize(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """x [..., n] -> (codes float8_e4m3fn [..., n], scales float32
    [..., ceil(n / 128)]), one scale per 1 x 128 block."""
    if x.dtype not in _DT:
        raise IqkValueError(_E_ARG, "x must be float32, float16 or bfloat16")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise IqkValueError(_E_ARG, "x must be [..., n] with n > 0")
    n = x.shape[-1]
    rows = x.numel() // n
    if codes is None:
        codes = _empty(x.shape, torch.float8_e4m3fn, x.device, stream)
    if scales is None:
        scales = _empty((*x.shape[:-1], _blocks(n)), torch.float32, x.device, stream)
    _check(_lib.iqk_fp8_quantize(_dev(x, "x"), _DT[x.dtype], rows, n,
                                 _dev(codes, "codes", torch.float8_e4m3fn, rows * n),
                                 _dev(scales, "scales", torch.float32, rows * _blocks(n)), _stream(stream)))
    return codes, scales


def _fp8_x(x: torch.Tensor, x_scales: torch.Tensor | None, rows: int, n: int):
    if x.dtype not in _XDT:
        raise IqkValueError(_E_ARG, "x must be float32, float16, bfloat16 or float8_e4m3fn")
    return (_dev(x, "x", None, rows * n), _XDT[x.dtype],
            _dev(x_scales, "x_scales", torch.float32, rows * _blocks(n)))


@functools.lru_cache(maxsize=1024)
def _fp8_linear_bytes(experts: int, out: int, n: int, M: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.iqk_fp8_linear_workspace(ctypes.byref(_Fp8Weights(experts, out, n)), M, ctypes.byref(b)))
    return b.value


def fp8_linear_workspace_bytes(w: Fp8Weights, M: int) -> int:
    """Workspace fp8_linear needs for M rows (0: none, a few rows are quantized where they are used)."""
    return _fp8_linear_bytes(w.experts, w.out, w.in_features, M)


def fp8_path(experts: int, out: int, n: int, T: int, k: int = 0, out_dtype=torch.float32):
    """Which kernels fp8_linear (k 0, T rows) or moe_fp8 (T tokens of k pairs)
    run on for weights [experts, out, n], for tests and profiles: ("few",),
    ("rows",) or ("tiles", rows of x, weight rows, parts of the depth)."""
    path = (ctypes.c_int32 * 4)()
    _check(_lib.iqk_fp8_path(ctypes.byref(_Fp8Weights(experts, out, n)), T, k, _DT.get(out_dtype, -1), path))
    return ("few", "rows", "tiles")[path[0]], *(path[1:] if path[0] == 2 else ())


def _round256(nbytes: int) -> int:
    return -(-nbytes // 256) * 256


def _quantized_bytes(rows: int, n: int) -> int:
    """The share of a workspace that x in codes does without."""
    return _round256(rows * n) + _round256(rows * _blocks(n) * 4)


def _workspace(workspace: torch.Tensor | None, nbytes: int, device, stream):
    """(workspace, pointer, size): the caller's, or a new one where the call needs any."""
    if workspace is None:
        if nbytes == 0:
            return None, None, 0
        workspace = _empty(nbytes, torch.uint8, device, stream)
    return workspace, _dev(workspace, "workspace", torch.uint8), workspace.numel()


def fp8_linear(w: Fp8Weights, x: torch.Tensor, x_scales: torch.Tensor | None = None, out_dtype=torch.float32,
               workspace: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [..., out] = x [..., in] times one expert's 8-bit weights.  x in a
    float type is quantized on the way (as fp8_quantize does); codes come
    with their x_scales."""
    n = w.in_features
    if x.dim() == 0 or x.shape[-1] != n:
        raise IqkValueError(_E_SIZE, f"x must be [..., {n}]")
    M = x.numel() // n
    xp, xdt, sp = _fp8_x(x, x_scales, M, n)
    if y is None:
        y = _empty((*x.shape[:-1], w.out), out_dtype, x.device, stream)
    if y.dtype not in _DT:
        raise IqkValueError(_E_ARG, "y must be float32, float16 or bfloat16")
    need = fp8_linear_workspace_bytes(w, M)
    if xdt == _E4M3 and need:
        need -= _quantized_bytes(M, n)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream)
    cw = w._c()
    _check(_lib.iqk_fp8_linear(ctypes.byref(cw), xp, xdt, sp, M, wp, nbytes, _dev(y, "y", None, M * w.out),
                               _DT[y.dtype], _stream(stream)))
    return y


@functools.lru_cache(maxsize=1024)
def _moe_fp8_bytes(experts: int, out: int, n: int, T: int, k: int, x_slots: int) -> int:
    b = ctypes.c_size_t()
    _check(_lib.iqk_moe_fp8_workspace(ctypes.byref(_Fp8Weights(experts, out, n)), T, k, x_slots, ctypes.byref(b)))
    return b.value


def moe_fp8_workspace_bytes(w: Fp8Weights, T: int, k: int, x_slots: int = 1) -> int:
    """Workspace moe_fp8 needs for T tokens of k slots (0: none, few pairs are taken one by one)."""
    return _moe_fp8_bytes(w.experts, w.out, w.in_features, T, k, x_slots)


def moe_fp8(w: Fp8Weights, x: torch.Tensor, ids: torch.Tensor, x_slots: int = 1,
            x_scales: torch.Tensor | None = None, sorted: bool = False, out_dtype=torch.float32,
            workspace: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The routed projection over 8-bit experts: y [T, k, out].  x [T *
    x_slots, in] as in fp8_linear; pairs with an invalid id get NaN rows."""
    ip = _ids(ids)
    T, k = ids.shape
    xp, xdt, sp = _fp8_x(x, x_scales, T * x_slots, w.in_features)
    if y is None:
        y = _empty((T, k, w.out), out_dtype, x.device, stream)
    if y.dtype not in _DT:
        raise IqkValueError(_E_ARG, "y must be float32, float16 or bfloat16")
    need = moe_fp8_workspace_bytes(w, T, k, x_slots)
    if xdt == _E4M3 and need:
        need -= _quantized_bytes(T * x_slots, w.in_features)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream)
    cw = w._c()
    _check(_lib.iqk_moe_fp8(ctypes.byref(cw), xp, xdt, sp, x_slots, ip, T, k, int(bool(sorted)), wp, nbytes,
                            _dev(y, "y", None, T * k * w.out), _DT[y.dtype], _stream(stream)))
    return y


# ---------------------------------------------------------------------------
# rows sorted by expert, and back
# ---------------------------------------------------------------------------


def _float_dtype(t: torch.Tensor, what: str) -> int:
    if t.dtype not in _DT:
        raise IqkValueError(_E_ARG, f"{what} must be float32, float16 or bfloat16")
    return _DT[t.dtype]


# These calls take a few microseconds of the card, so the host's share counts: an address as a plain number
# (0.2 us less than the object _dev makes) and results made like an input (torch.empty_like 1.15 us, new_empty 1.9,
# torch.empty 2.4).


def _at(t: torch.Tensor | None, what: str, dtype=None, numel: int | None = None):
    """_dev's checks; the address as a number."""
    if t is None:
        return None
    if not t.is_cuda:
        raise IqkValueError(_E_ARG, f"{what} must be a device tensor")
    if not t.is_contiguous():
        raise IqkValueError(_E_ARG, f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise IqkValueError(_E_ARG, f"{what} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise IqkValueError(_E_SIZE, f"{what} has {t.numel()} elements, expected {numel}")
    return t.data_ptr()


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    return like.new_empty(shape, dtype=dtype) if stream is None else _empty(shape, dtype, like.device, stream)


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    return torch.empty_like(t) if stream is None else _empty(t.shape, t.dtype, t.device, stream)


def _one_device(*tensors: torch.Tensor | None):
    """All tensors of a call lie on the current device, whose memory its kernels reach."""
    here = None
    for t in tensors:
        if t is None:
            continue
        at = t.get_device()
        if at < 0:  # (a host tensor)
            continue
        if here is None:
            here = torch.cuda.current_device()
        if at != here:
            raise IqkValueError(_E_ARG, f"a tensor on cuda:{at} where cuda:{here} is current")


def _refuse_tangents(*tensors: torch.Tensor | None):
    """No call has a forward-mode derivative, and a result without one would pass for a constant."""
    if torch.is_inference_mode_enabled():
        return
    for t in tensors:
        if t is not None and _forward_ad.unpack_dual(t).tangent is not None:
            raise IqkValueError(_E_ARG, "a tensor carries a forward-mode tangent, which no call here hands on")


def _wants_grad(*tensors: torch.Tensor | None) -> bool:
    """Whether a result is to carry a gradient."""
    if getattr(_forward_ad, "_current_level", 0) >= 0:
        _refuse_tangents(*tensors)
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _refuse_grad(call: str):
    raise IqkValueError(_E_ARG, f"{call} has no gradient: detach what requires one, or call it under torch.no_grad()")


def _written(*given: torch.Tensor | None):
    """Caller's buffers that a call wrote: a gradient of an earlier call that still needs one can tell."""
    for t in given:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _on(stream):
    """The given stream as the current one (backward passes run on the stream of their forward call)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(_stream_object(stream))


@functools.lru_cache(maxsize=1024)
def moe_sort_workspace_bytes(T: int, k: int, E: int) -> int:
    """Workspace moe_sort needs for T tokens of k slots (0: none, few pairs are sorted in one launch)."""
    b = ctypes.c_size_t()
    _check(_lib.iqk_moe_sort_workspace(T, k, E, ctypes.byref(b)))
    return b.value


def _sort(x, ids, E, xs, offsets, place, workspace, stream):
    xp, dt, ip = _at(x, "x"), _float_dtype(x, "x"), _at(ids, "ids", torch.int32)
    T, k = ids.shape
    n = x.shape[1]
    need = moe_sort_workspace_bytes(T, k, E)
    if xs is None:
        xs = _new(x, (T * k, n), x.dtype, stream)
    if offsets is None:
        offsets = _new(x, (E + 1,), torch.int32, stream)
    if place is None:
        place = _like(ids, stream)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream)
    _check(_lib.iqk_moe_sort(xp, dt, ip, T, k, E, n, wp, nbytes, _at(xs, "xs", x.dtype, T * k * n), _at(offsets, "offsets", torch.int32, E + 1),
                             _at(place, "place", torch.int32, T * k), _stream(stream)))
    return xs, offsets, place


def moe_sort(x: torch.Tensor, ids: torch.Tensor, E: int, xs: torch.Tensor | None = None,
             offsets: torch.Tensor | None = None, place: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None):
    """Token rows x [T, n] in the order of their experts ids [T, k]: (xs
    [T * k, n], offsets int32 [E + 1], place int32 [T, k]).  Expert e's rows are
    offsets[e] .. offsets[e + 1] - 1 in the order of their pairs; place is each
    pair's row, or -1 - row (a row of zeros behind the experts') where its id is
    outside [0, E).  Where x requires a gradient xs carries it (through
    moe_unsort without weights)."""
    if x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise IqkValueError(_E_ARG, "x must be [T, n] and ids [T, k]")
    _one_device(x, ids, xs, offsets, place, workspace)
    if not _wants_grad(x):
        out = _sort(x, ids, E, xs, offsets, place, workspace, stream)
        _written(xs, offsets, place)
        return out
    if xs is not None:
        raise IqkValueError(_E_ARG, "xs given where x requires a gradient")
    with _on(stream):
        return _Sort.apply(x, ids, E, offsets, place, workspace)


class _Sort(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, ids, E, offsets, place, workspace):
        given = [t for t in (offsets, place) if t is not None]
        xs, offsets, place = _sort(x.detach(), ids, E, None, offsets, place, workspace, None)
        ctx.mark_dirty(*given)
        ctx.mark_non_differentiable(offsets, place)
        ctx.save_for_backward(place)
        return xs, offsets, place

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_xs, *_):
        (place,) = ctx.saved_tensors
        return moe_unsort(d_xs.contiguous(), place, out_dtype=d_xs.dtype), None, None, None, None, None


def _check_unsort(ys, place, weights):
    if ys.dim() != 2 or place.dim() != 2 or ys.shape[0] != place.numel():
        raise IqkValueError(_E_ARG, "ys must be [T * k, n] and place [T, k]")
    T, k = place.shape
    return (_at(ys, "ys"), _float_dtype(ys, "ys"), _at(place, "place", torch.int32),
            _at(weights, "weights", torch.float32, T * k), T, k, ys.shape[1])


def _unsort(ys, place, weights, out_dtype, y, stream):
    yp, dt, pp, wp, T, k, n = _check_unsort(ys, place, weights)
    if y is None:
        y = _new(ys, (T, n), out_dtype, stream)
    _check(_lib.iqk_moe_unsort(yp, dt, pp, wp, T, k, n, _at(y, "y", None, T * n), _float_dtype(y, "y"), _stream(stream)))
    return y


def moe_unsort(ys: torch.Tensor, place: torch.Tensor, weights: torch.Tensor | None = None, out_dtype=torch.float32,
               y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Expert rows ys [T * k, n] back to their tokens: y[t] = sum_j weights[t, j] *
    ys[place[t, j]] (float32 sums in slot order; weights None: ones), with place
    from moe_sort.  Pairs of no expert count as rows of zeros.  Where ys or weights
    require a gradient y carries it (through moe_unsort_grad)."""
    _one_device(ys, place, weights, y)
    if not _wants_grad(ys, weights):
        out = _unsort(ys, place, weights, out_dtype, y, stream)
        _written(y)
        return out
    if y is not None:
        raise IqkValueError(_E_ARG, "y given where ys or weights require a gradient")
    if out_dtype not in _DT:
        raise IqkValueError(_E_ARG, "y must be float32, float16 or bfloat16")
    with _on(stream):
        return _Unsort.apply(ys, place, weights, out_dtype)


class _Unsort(torch.autograd.Function):
    """Rows are kept for the weights' gradient only, and weights for the rows': a layer's largest tensor may go, or be
    written over, where the router is not trained."""

    @staticmethod
    def forward(ctx, ys, place, weights, out_dtype):
        want_ys, _, want_w = ctx.needs_input_grad[:3]
        ctx.save_for_backward(ys if want_w else None, place, weights if want_ys else None)
        ctx.rows, ctx.weights = (ys.shape, ys.dtype), None if weights is None else weights.shape
        return _unsort(ys.detach(), place, None if weights is None else weights.detach(), out_dtype, None, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        ys, place, weights = ctx.saved_tensors
        want_ys, _, want_w = ctx.needs_input_grad[:3]
        (rows, n), dtype = ctx.rows
        d_ys = dy.new_empty((rows, n), dtype=dtype) if want_ys else None
        d_w = dy.new_empty(ctx.weights, dtype=torch.float32) if want_w else None
        T, k = place.shape
        _unsort_grad(dy.contiguous(), None if ys is None else ys.data_ptr(), _DT[dtype], place.data_ptr(),
                     None if weights is None else weights.data_ptr(), T, k, n, dtype, d_ys, d_w, None)
        return d_ys, None, d_w, None


def _unsort_grad(dy, yp, dt, pp, wp, T, k, n, dtype, d_ys, d_weights, stream):
    _check(_lib.iqk_moe_unsort_grad(_at(dy, "dy", None, T * n), _float_dtype(dy, "dy"), yp, dt, pp, wp, T, k, n,
                                    _at(d_ys, "d_ys", dtype, T * k * n), _at(d_weights, "d_weights", torch.float32, T * k),
                                    _stream(stream)))


def moe_unsort_grad(dy: torch.Tensor, ys: torch.Tensor, place: torch.Tensor, weights: torch.Tensor | None = None,
                    d_ys: torch.Tensor | None = None, d_weights: torch.Tensor | None = None, want_ys: bool = True,
                    want_weights: bool = True, stream=None):
    """Gradient of moe_unsort from dy [T, n]: (d_ys [T * k, n] of ys' type,
    d_weights float32 [T, k]); None for one that is not wanted, and for d_weights
    where weights is None."""
    _one_device(dy, ys, place, weights, d_ys, d_weights)
    checked = _check_unsort(ys, place, weights)
    want_weights = want_weights and weights is not None
    if not want_ys and not want_weights:
        raise IqkValueError(_E_ARG, "neither gradient is wanted")
    d_ys, d_weights = given = d_ys if want_ys else None, d_weights if want_weights else None
    if want_ys and d_ys is None:
        d_ys = _like(ys, stream)
    if want_weights and d_weights is None:
        d_weights = _like(weights, stream)
    _unsort_grad(dy, *checked, ys.dtype, d_ys, d_weights, stream)
    _written(*given)
    return d_ys, d_weights


# ---------------------------------------------------------------------------
# products in 8-bit integers, a scale for each token and output channel
# ---------------------------------------------------------------------------

_IDT = {**_DT, torch.int8: _INT8}


@dataclass
class Int8Weights:
    """8-bit integer weights: codes int8 [experts, out, in] with scales float32
    [experts, out], one per output channel."""

    codes: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        if self.codes.dim() != 3 or self.codes.dtype != torch.int8:
            raise IqkValueError(_E_ARG, "codes must be int8 [experts, out, in]")
        if self.codes.numel() == 0:
            raise IqkValueError(_E_ARG, "codes hold no values")
        self.experts, self.out, self.in_features = self.codes.shape
        if self.scales.dtype != torch.float32 or self.scales.shape != (self.experts, self.out):
            raise IqkValueError(_E_SIZE, "scales must be float32 [experts, out]")

    def _c(self) -> _Int8Weights:
        cp, sp = _at(self.codes, "codes"), _at(self.scales, "scales")
        return _Int8Weights(self.experts, self.out, self.in_features, cp, self.codes.numel(), sp, self.scales.numel())


def int8_quantize(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """x [..., n] -> (codes int8 [..., n], scales float32 [...]), one scale per
    row.  It has no gradient: x that requires one is refused."""
    dt = _float_dtype(x, "x")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise IqkValueError(_E_ARG, "x must be [..., n] with n > 0")
    _one_device(x, codes, scales)
    if _wants_grad(x):
        _refuse_grad("int8_quantize")
    n = x.shape[-1]
    rows = x.numel() // n
    xp = _at(x, "x")
    given = codes, scales
    if codes is None:
        codes = _new(x, x.shape, torch.int8, stream)
    if scales is None:
        scales = _new(x, x.shape[:-1], torch.float32, stream)
    _check(_lib.iqk_int8_quantize(xp, dt, rows, n, _at(codes, "codes", torch.int8, rows * n),
                                  _at(scales, "scales", torch.float32, rows), _stream(stream)))
    if given[0] is not None or given[1] is not None:
        _written(*given)
    return codes, scales


def _int8_x(x: torch.Tensor, x_scales: torch.Tensor | None, rows: int, n: int):
    if x.dtype not in _IDT:
        raise IqkValueError(_E_ARG, "x must be float32, float16, bfloat16 or int8")
    return _at(x, "x", None, rows * n), _IDT[x.dtype], _at(x_scales, "x_scales", torch.float32, rows)


@functools.lru_cache(maxsize=1024)
def _int8_bytes(call: str, experts: int, out: int, n: int, rows: int, xdt: int) -> int:
    b = ctypes.c_size_t()
    _check(getattr(_lib, call)(ctypes.byref(_Int8Weights(experts, out, n)), rows, xdt, ctypes.byref(b)))
    return b.value


def int8_linear_workspace_bytes(w: Int8Weights, M: int, x_dtype=torch.bfloat16) -> int:
    """Workspace int8_linear needs for M rows (0: none, a few rows are quantized where they are used)."""
    return _int8_bytes("iqk_int8_linear_workspace", w.experts, w.out, w.in_features, M, _IDT.get(x_dtype, -1))


def int8_grouped_workspace_bytes(w: Int8Weights, rows: int, x_dtype=torch.bfloat16) -> int:
    """Workspace int8_grouped needs for so many rows (0: none)."""
    return _int8_bytes("iqk_int8_grouped_workspace", w.experts, w.out, w.in_features, rows, _IDT.get(x_dtype, -1))


def int8_path(experts: int, out: int, n: int, rows: int, grouped: bool = False):
    """Which kernel int8_linear or int8_grouped runs on for weights [experts, out,
    n], for tests and profiles: ("few",), ("rows",) or ("tiles", rows of x, weight rows)."""
    path = (ctypes.c_int32 * 3)()
    _check(_lib.iqk_int8_path(ctypes.byref(_Int8Weights(experts, out, n)), rows, int(bool(grouped)), path))
    return ("few", "rows", "tiles")[path[0]], *(path[1:] if path[0] == 2 else ())


def int8_linear(w: Int8Weights, x: torch.Tensor, x_scales: torch.Tensor | None = None, out_dtype=torch.float32,
                workspace: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [..., out] = x [..., in] times 8-bit integer weights.  x in a float type
    is quantized on the way (as int8_quantize does); codes come with their
    x_scales.  The product has no gradient: x and scales that require one are
    refused."""
    n = w.in_features
    if x.dim() == 0 or x.shape[-1] != n:
        raise IqkValueError(_E_SIZE, f"x must be [..., {n}]")
    _one_device(x, w.codes, w.scales, x_scales, workspace, y)
    if _wants_grad(x, w.scales, x_scales):
        _refuse_grad("int8_linear")
    M = x.numel() // n
    xp, xdt, sp = _int8_x(x, x_scales, M, n)
    cw = w._c()
    given = y
    if y is None:
        y = _new(x, (*x.shape[:-1], w.out), out_dtype, stream)
    need = _int8_bytes("iqk_int8_linear_workspace", w.experts, w.out, n, M, xdt)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream) if need or workspace is not None else (None, None, 0)
    _check(_lib.iqk_int8_linear(ctypes.byref(cw), xp, xdt, sp, M, wp, nbytes, _at(y, "y", None, M * w.out),
                                _float_dtype(y, "y"), _stream(stream)))
    if given is not None:
        _written(given)
    return y


def int8_grouped(w: Int8Weights, x: torch.Tensor, offsets: torch.Tensor, x_scales: torch.Tensor | None = None,
                 out_dtype=torch.float32, workspace: torch.Tensor | None = None, y: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """y [rows, out]: rows offsets[e] .. offsets[e + 1] - 1 of x [rows, in] times
    expert e's weights (x and offsets as moe_sort makes them); rows behind the last
    expert's are zeros.  x as in int8_linear."""
    if x.dim() != 2 or x.shape[1] != w.in_features:
        raise IqkValueError(_E_SIZE, f"x must be [rows, {w.in_features}]")
    _one_device(x, w.codes, w.scales, offsets, x_scales, workspace, y)
    if _wants_grad(x, w.scales, x_scales):
        _refuse_grad("int8_grouped")
    rows, n = x.shape
    xp, xdt, sp = _int8_x(x, x_scales, rows, n)
    op = _at(offsets, "offsets", torch.int32, w.experts + 1)
    cw = w._c()
    given = y
    if y is None:
        y = _new(x, (rows, w.out), out_dtype, stream)
    need = _int8_bytes("iqk_int8_grouped_workspace", w.experts, w.out, n, rows, xdt)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream) if need or workspace is not None else (None, None, 0)
    _check(_lib.iqk_int8_grouped(ctypes.byref(cw), xp, xdt, sp, op, rows, wp, nbytes,
                                 _at(y, "y", None, rows * w.out), _float_dtype(y, "y"), _stream(stream)))
    if given is not None:
        _written(given)
    return y


# ---------------------------------------------------------------------------
# the norms around a block
# ---------------------------------------------------------------------------


def _block(x, y, post_weight, gate, next_weight, alpha, beta, eps) -> _Block:
    """The call's descriptor, after checking every tensor's type and size."""
    dt = _float_dtype(x, "x")
    if x.dim() == 0 or x.shape[-1] == 0:
        raise IqkValueError(_E_ARG, "x must be [..., n] with n > 0")
    n = x.shape[-1]
    T = x.numel() // n
    ydt = dt
    if y is not None:
        ydt = _float_dtype(y, "y")
        if y.dim() == 0 or y.shape[-1] != n:
            raise IqkValueError(_E_SIZE, f"y must be [..., {n}]")
    weights = [t for t in (post_weight, next_weight) if t is not None]
    if len(weights) == 2 and weights[0].dtype != weights[1].dtype:
        raise IqkValueError(_E_ARG, "post_weight and next_weight must be of one type")
    kind, gdt, size = 0, _F32, None
    if gate is not None:
        gdt = _float_dtype(gate, "gate")
        shape = tuple(gate.shape)
        if shape == (n,):
            kind, size = 1, n
        elif shape == (*x.shape[:-1], 1):
            kind, size = 2, T
        elif shape == tuple(x.shape):
            kind, size = 3, T * n
        else:
            raise IqkValueError(_E_SIZE, f"gate must be [{n}], {[*x.shape[:-1], 1]} or {list(x.shape)}")
    return _Block(T, n, dt, ydt, _float_dtype(weights[0], "weights") if weights else _F32, gdt, kind, alpha, beta, eps,
                  _at(x, "x"), _at(y, "y", None, T * n), _at(post_weight, "post_weight", None, n),
                  _at(gate, "gate", None, size), _at(next_weight, "next_weight", None, n))


def _block_norm(x, y, post_weight, gate, next_weight, alpha, beta, eps, r, h, stream):
    b = _block(x, y, post_weight, gate, next_weight, alpha, beta, eps)
    numel = b.T * b.n
    if y is not None and r is None:
        r = _like(x, stream)
    if next_weight is not None and h is None:
        h = _like(x, stream)
    _check(_lib.iqk_block_norm(ctypes.byref(b), _at(r, "r", x.dtype, numel), _at(h, "h", x.dtype, numel), _stream(stream)))
    return r, h


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, post_weight: torch.Tensor | None = None,
               gate: torch.Tensor | None = None, next_weight: torch.Tensor | None = None, alpha: float = 1.0,
               beta: float = 1.0, eps: float = 1e-6, r: torch.Tensor | None = None, h: torch.Tensor | None = None,
               stream=None):
    """The norms around a block, its gate and the scaled residual, in one pass:
    (r, h) with

        u = y * s(y) * post_weight        (u = y without post_weight)
        r = alpha * x + beta * gate * u
        h = r * s(r) * next_weight        s(v) = 1 / sqrt(mean(v^2) + eps)

    x [..., n] is the residual stream, y [..., n] the block's output (of x's type
    or float32), gate [n], [..., 1] or [..., n]; r and h are of x's type, h from r
    before its rounding.  h is None without next_weight.  Without y it is the norm
    before the first block: (x, h).  Where an input requires a gradient the
    results carry it (through block_norm_grad)."""
    _one_device(x, y, post_weight, gate, next_weight, r, h)
    if not _wants_grad(x, y, post_weight, gate, next_weight):
        given = r, h
        r, h = _block_norm(x, y, post_weight, gate, next_weight, alpha, beta, eps, r, h, stream)
        _written(*given)
        return x if y is None else r, h
    if r is not None or h is not None:
        raise IqkValueError(_E_ARG, "r or h given where an input requires a gradient")
    with _on(stream):
        out = _BlockNorm.apply(x, y, post_weight, gate, next_weight, alpha, beta, eps)
    return (x, out[0]) if y is None else (out[0], out[1] if len(out) > 1 else None)


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, post_weight, gate, next_weight, alpha, beta, eps):
        ctx.save_for_backward(x, y, post_weight, gate, next_weight)
        ctx.args = alpha, beta, eps
        ctx.set_materialize_grads(False)
        plain = [None if t is None else t.detach() for t in (x, y, post_weight, gate, next_weight)]
        return tuple(t for t in _block_norm(*plain, alpha, beta, eps, None, None, None) if t is not None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        x, y, post_weight, gate, next_weight = ctx.saved_tensors
        grads = [None if g is None else g.contiguous() for g in grads]
        dr = grads[0] if y is not None else None
        dh = grads[-1] if next_weight is not None else None
        if dr is None and dh is None:
            return (None,) * 8
        alpha, beta, eps = ctx.args
        got = block_norm_grad(x, y, dr, dh, post_weight=post_weight, gate=gate, next_weight=next_weight, alpha=alpha,
                              beta=beta, eps=eps, want=ctx.needs_input_grad[:5])
        return (*got, None, None, None)


def block_norm_grad_workspace_bytes(T: int, n: int, post_weight: bool = True, next_weight: bool = True,
                                    channel_gate: bool = False) -> int:
    """Workspace block_norm_grad needs for the gradients of these parameters."""
    return _block_grad_bytes(T, n, bool(post_weight), bool(next_weight), bool(channel_gate))


@functools.lru_cache(maxsize=1024)
def _block_grad_bytes(T: int, n: int, post: bool, nxt: bool, channel: bool) -> int:
    b = ctypes.c_size_t()
    blk = _Block(T, n, gate_kind=int(channel), post_weight=1 if post else None, next_weight=1 if nxt else None)
    _check(_lib.iqk_block_norm_grad_workspace(ctypes.byref(blk), ctypes.byref(b)))
    return b.value


def block_norm_grad(x: torch.Tensor, y: torch.Tensor | None, dr: torch.Tensor | None, dh: torch.Tensor | None = None,
                    post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                    next_weight: torch.Tensor | None = None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
                    want=(True,) * 5, workspace: torch.Tensor | None = None, stream=None):
    """Gradient of block_norm from those of r and h (None: zero): (dx, dy,
    d_post_weight, d_gate, d_next_weight), each of its input's type and shape; None
    for inputs that are None and where want is false."""
    _one_device(x, y, dr, dh, post_weight, gate, next_weight, workspace)
    b = _block(x, y, post_weight, gate, next_weight, alpha, beta, eps)
    numel = b.T * b.n
    drp, dhp = _at(dr, "dr", x.dtype, numel), _at(dh, "dh", x.dtype, numel)
    out = [_like(t, stream) if t is not None and wanted else None
           for t, wanted in zip((x, y, post_weight, gate, next_weight), want)]
    channel = b.gate_kind == 1 and out[3] is not None
    need = _block_grad_bytes(b.T, b.n, out[2] is not None, out[4] is not None, channel)
    ws, wp, nbytes = _workspace(workspace, need, x.device, stream)
    _check(_lib.iqk_block_norm_grad(ctypes.byref(b), drp, dhp, *(None if t is None else t.data_ptr() for t in out), wp,
                                    nbytes, _stream(stream)))
    return tuple(out)
