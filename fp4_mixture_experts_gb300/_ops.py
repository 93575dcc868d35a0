"""The operators around the layer: MXFP4 quantisation, products of MXFP4
matrices (dense, and grouped by expert) and the end of a block.

The work of a call on the host (argument checks, results, workspaces, the
current CUDA stream) is native too (csrc/ops_binding.cpp): a single-token
operator takes a few microseconds on the GPU, less than its marshalling in
Python.  Wrong types, shapes or strides raise ValueError; a nonzero status of
the library becomes a MoeFp4Error.  `out`, `codes`, `scales` and `workspace` may
be given so that a call allocates nothing (a captured graph).
"""
from __future__ import annotations

import ctypes

from . import _binding
from ._binding import MoeFp4Error, load_library

_BF16 = None  # torch.bfloat16, once the binding is loaded


class MmDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "E", "swiglu", "y_type")]


class BlockNormArgs(ctypes.Structure):
    _fields_ = ([("T", ctypes.c_int64)] +
                [(n, ctypes.c_int32) for n in ("d", "post_norm", "gate_shape", "gate_sigmoid", "residual_type",
                                               "y_type", "y2_type", "gate_type", "post_weight_type",
                                               "next_weight_type")] +
                [(n, ctypes.c_int64) for n in ("residual_stride", "y_stride", "y2_stride", "gate_stride",
                                               "out_stride")] +
                [("scale", ctypes.c_float), ("eps", ctypes.c_float)] +
                [(n, ctypes.c_void_p) for n in ("residual", "y", "y2", "gate", "post_weight", "next_weight", "out",
                                                "normed")])


def _raise(status, entry):
    raise MoeFp4Error(status, entry)


class _Unloaded:
    """Stands for the native binding until the first call loads it."""

    def __getattr__(self, name):
        global _native, _BF16
        import torch
        lib = load_library()
        try:
            from . import _ops_native as native
        except ImportError as e:
            raise RuntimeError("the operators' native binding is missing: build it with `python -m "
                               "fp4_mixture_experts_gb300.build` (there is no fallback implementation)") from e
        native.bind(tuple(ctypes.cast(getattr(lib, "moe_fp4_" + n), ctypes.c_void_p).value for n in (
            "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_tile_scales", "mxfp4_matmul", "mxfp4_linear",
            "mxfp4_linear_workspace_bytes", "mxfp4_gathered_workspace_bytes", "block_norm")), _raise)
        _native, _BF16 = native, torch.bfloat16
        return getattr(native, name)


_native = _Unloaded()


def _handle(stream):
    return None if stream is None else stream.cuda_stream


def mxfp4_tiled_scale_bytes(rows: int, K: int, groups: int = 1) -> int:
    return int(load_library().moe_fp4_mxfp4_tiled_scale_bytes(rows, groups, K))


def mxfp4_quantize(x, row_index=None, index_div: int = 1, offsets=None, tiled: bool = False, codes=None, scales=None,
                   stream=None):
    """MXFP4 of rows x [R, K] (bf16 or fp32, K a multiple of 32; rows may be strided).

    Returns (codes uint8 [S, K/2], scales uint8): scales [S, K/32], or with tiled the layout of the products
    ([row tiles, ceil(K/128), 512]; by group with offsets, int32 [E + 1]).  row_index (int32 [S]) gathers: row r
    is row row_index[r] // index_div of x (sorted_slot and k of the layer's routing); without it S = R."""
    return _native.quantize(x, row_index, index_div, offsets, tiled, codes, scales, _handle(stream))


def mxfp4_dequantize(codes, scales, dtype=None, out=None, stream=None):
    """The values (bf16, or dtype=torch.float32, [.., K]) of MXFP4 codes uint8 [.., K/2] with row-major scales uint8
    [.., K/32]."""
    f = _native.dequantize
    return f(codes, scales, dtype or _BF16, out, _handle(stream))


def mxfp4_tile_scales(scales, swiglu: bool = False, out=None, stream=None):
    """Row-major weight scales uint8 [E, N, K/32] or [N, K/32] in the layout of the products, uint8
    [E, ceil(N/128), ceil(K/128), 512]: once, when weights are loaded.  swiglu: for products with SwiGLU."""
    return _native.tile_scales(scales, swiglu, out, _handle(stream))


def mxfp4_matmul(a, a_scale, w, w_scale, offsets=None, swiglu: bool = False, dtype=None, out=None, stream=None):
    """y = a w^T of MXFP4 matrices: a uint8 [M, K/2] with tiled scales (mxfp4_quantize), w uint8 [E, N, K/2] with
    tiled scales (mxfp4_tile_scales).  offsets (int32 [E + 1]): rows [off[e], off[e+1]) use w[e], and a_scale is in
    the grouped layout of the same offsets.  Returns [M, N], or with swiglu silu(first half) * second half [M, N/2]:
    bf16, or dtype=torch.float32."""
    f = _native.matmul
    return f(a, a_scale, w, w_scale, offsets, swiglu, dtype or _BF16, out, _handle(stream))


def mxfp4_linear_workspace_bytes(M: int, N: int, K: int, E: int = 1, x_rows: int | None = None) -> int:
    """Bytes of mxfp4_linear's workspace; x_rows: of a call that gathers its M rows from that many, enough to quantise
    rows that are used several times once (less, down to the size without x_rows, is fine too)."""
    dims = ctypes.byref(MmDims(M, N, K, E, 0, 0))
    if x_rows is None:
        return int(load_library().moe_fp4_mxfp4_linear_workspace_bytes(dims))
    return int(load_library().moe_fp4_mxfp4_gathered_workspace_bytes(dims, x_rows))


def mxfp4_linear(x, w, w_scale, offsets=None, row_index=None, index_div: int = 1, swiglu: bool = False, dtype=None,
                 out=None, workspace=None, stream=None):
    """The product from unquantised rows x [R, K] (bf16 or fp32): mxfp4_quantize (with row_index / index_div, and
    offsets) and mxfp4_matmul in one call, the same bits."""
    f = _native.linear
    return f(x, w, w_scale, offsets, row_index, index_div, swiglu, dtype or _BF16, out, workspace, _handle(stream))


def rms_norm(x, weight=None, eps: float = 1e-6, out=None, stream=None):
    """The norm before a block: bf16 [T, d] = x rsqrt(mean(x^2) + eps) * weight.  x bf16 or fp32 [T, d] (rows may
    be strided), weight bf16 or fp32 [d]."""
    return _native.rms_norm(x, weight, eps, out, _handle(stream))


def block_residual(residual, y, y2=None, post_norm: bool = True, post_weight=None, gate=None,
                   gate_sigmoid: bool = False, scale: float = 1.0, next_norm: bool = True, next_weight=None,
                   eps: float = 1e-6, out=None, normed=None, stream=None):
    """The end of a block and the norm before the next one, in one pass:

      b = y (+ y2); post_norm: b *= rsqrt(mean(b^2) + eps); b *= post_weight; b *= gate or sigmoid(gate)
      out = residual + scale * b;  normed = out rsqrt(mean(out^2) + eps) * next_weight

    residual, y, y2: bf16 or fp32 [T, d], rows may be strided.  gate: [T], [d] or [T, d] (T = d: give [T, 1],
    [1, d] or [T, d]).  Returns (out, normed): out of residual's type (out=residual adds in place), normed bf16,
    or None with next_norm=False."""
    return _native.block_residual(residual, y, y2, post_norm, post_weight, gate, gate_sigmoid, scale, next_norm,
                                  next_weight, eps, out, normed, _handle(stream))


def ops_check(stream=None) -> None:
    """Synchronise and raise if a kernel of an earlier operator call on this device, on any of its streams, reported an
    error (a row index out of range, or a pipeline wait that ran out); each error is reported by one check."""
    rc = load_library().moe_fp4_ops_check(_binding._stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_ops_check")
