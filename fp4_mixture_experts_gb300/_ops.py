"""Binding of the operators around the layer: MXFP4 quantisation, products of
MXFP4 matrices (dense, and grouped by expert) and the end of a block.

Like _binding: argument marshalling only, on the current CUDA stream unless
one is given.  Wrong types, shapes or strides raise ValueError; a nonzero
status of the library becomes a MoeFp4Error.  `out`, `codes`, `scales` and
`workspace` may be given so that a call allocates nothing (a captured graph).
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding
from ._binding import MoeFp4Error, load_library

_TYPES = {torch.bfloat16: 0, torch.float32: 1}


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


def _lib():
    return _binding._lib or load_library()


def _raw_stream(stream):
    return (stream or torch.cuda.current_stream()).cuda_stream


def _type(t, what):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16 or fp32, not {t.dtype}")
    return code


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _rows2d(t, what):
    """A GPU tensor of rows: 2-D, its last dimension contiguous (rows may be strided); its row stride"""
    _need(t.is_cuda and t.dim() == 2, f"{what} must be a 2-D GPU tensor")
    T, K = t.shape
    if T <= 1:
        _need(K <= 1 or t.stride(1) == 1, f"{what} must be contiguous along its rows")
        return K
    _need((K <= 1 or t.stride(1) == 1) and t.stride(0) >= K, f"{what} must have contiguous, separate rows")
    return t.stride(0)


def _bytes(t, what, numel):
    _need(t.is_cuda and t.dtype == torch.uint8 and t.is_contiguous() and t.numel() >= numel,
          f"{what} must be a contiguous uint8 GPU tensor of at least {numel} elements")


def _indices(row_index, index_div, offsets):
    if row_index is not None:
        _need(row_index.is_cuda and row_index.dtype == torch.int32 and row_index.is_contiguous() and
              row_index.dim() == 1, "row_index must be a contiguous 1-D int32 GPU tensor")
        _need(index_div >= 1, "index_div must be at least 1")
    if offsets is not None:
        _need(offsets.is_cuda and offsets.dtype == torch.int32 and offsets.is_contiguous() and offsets.dim() == 1 and
              offsets.numel() >= 2, "offsets must be a contiguous 1-D int32 GPU tensor of E + 1 elements")


def mxfp4_tiled_scale_bytes(rows: int, K: int, groups: int = 1) -> int:
    return int(_lib().moe_fp4_mxfp4_tiled_scale_bytes(rows, groups, K))


def mxfp4_quantize(x, row_index=None, index_div: int = 1, offsets=None, tiled: bool = False, codes=None, scales=None,
                   stream=None):
    """MXFP4 of rows x [R, K] (bf16 or fp32, K a multiple of 32; rows may be strided).

    Returns (codes uint8 [S, K/2], scales uint8): scales [S, K/32], or with tiled the layout of the products
    ([row tiles, ceil(K/128), 512]; by group with offsets, int32 [E + 1]).  row_index (int32 [S]) gathers: row r
    is row row_index[r] // index_div of x (sorted_slot and k of the layer's routing); without it S = R."""
    xt = _type(x, "x")
    stride = _rows2d(x, "x")
    _indices(row_index, index_div, offsets)
    _need(offsets is None or tiled, "offsets need tiled scales")
    R, K = x.shape
    _need(K > 0 and K % 32 == 0, "K must be a multiple of 32")
    S = R if row_index is None else row_index.numel()
    E = 1 if offsets is None else offsets.numel() - 1
    if codes is None:
        codes = torch.empty(S, K // 2, dtype=torch.uint8, device=x.device)
    else:
        _bytes(codes, "codes", S * (K // 2))
    kt = -(-K // 128)
    if scales is None:
        shape = (S // 128 + E, kt, 512) if tiled else (S, K // 32)
        scales = torch.empty(shape, dtype=torch.uint8, device=x.device)
    else:
        _bytes(scales, "scales", (S // 128 + E) * kt * 512 if tiled else S * (K // 32))
    rc = _lib().moe_fp4_mxfp4_quantize(
        x.data_ptr(), xt, R, stride, K, None if row_index is None else row_index.data_ptr(), index_div, S,
        None if offsets is None else offsets.data_ptr(), E, codes.data_ptr(), scales.data_ptr(), int(tiled),
        _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values (bf16 or fp32 [.., K]) of MXFP4 codes uint8 [.., K/2] with row-major scales uint8 [.., K/32]."""
    _need(dtype in _TYPES, "dtype must be bf16 or fp32")
    K = 2 * codes.shape[-1]
    _need(K > 0 and K % 32 == 0, "K must be a multiple of 32")
    rows = codes.numel() // (K // 2)
    _bytes(codes, "codes", codes.numel())
    _bytes(scales, "scales", rows * (K // 32))
    if out is None:
        out = torch.empty(*codes.shape[:-1], K, dtype=dtype, device=codes.device)
    else:
        _need(out.is_cuda and out.dtype == dtype and out.is_contiguous() and out.numel() == rows * K,
              "out must be a contiguous GPU tensor of dtype with a value for each code")
    rc = _lib().moe_fp4_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, K, _TYPES[dtype], out.data_ptr(),
                                         _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_dequantize")
    return out


def mxfp4_tile_scales(scales, swiglu: bool = False, out=None, stream=None):
    """Row-major weight scales uint8 [E, N, K/32] or [N, K/32] in the layout of the products, uint8
    [E, ceil(N/128), ceil(K/128), 512]: once, when weights are loaded.  swiglu: for products with SwiGLU."""
    _need(scales.dim() in (2, 3), "scales must be [E, N, K/32] or [N, K/32]")
    E = scales.shape[0] if scales.dim() == 3 else 1
    N, nb = scales.shape[-2:]
    _bytes(scales, "scales", E * N * nb)
    shape = (E, -(-N // 128), -(-nb // 4), 512)
    if out is None:
        out = torch.empty(shape, dtype=torch.uint8, device=scales.device)
    else:
        _bytes(out, "out", shape[0] * shape[1] * shape[2] * 512)
    rc = _lib().moe_fp4_mxfp4_tile_scales(scales.data_ptr(), E, N, 32 * nb, int(swiglu), out.data_ptr(),
                                          _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_tile_scales")
    return out


def _mm_dims(M, K, w, w_scale, offsets, swiglu, dtype):
    _need(w.dim() in (2, 3) and w.shape[-1] * 2 == K, "w must be uint8 [E, N, K/2] or [N, K/2]")
    E = w.shape[0] if w.dim() == 3 else 1
    N = w.shape[-2]
    _bytes(w, "w", w.numel())
    _bytes(w_scale, "w_scale (tiled: mxfp4_tile_scales)", E * -(-N // 128) * -(-K // 128) * 512)
    _need(dtype in _TYPES, "dtype must be bf16 or fp32")
    _need(not swiglu or N % 2 == 0, "swiglu needs an even number of features")
    if offsets is None:
        _need(E == 1, "several matrices need offsets")
    else:
        _need(offsets.numel() == E + 1, "offsets must have E + 1 elements")
    return MmDims(M, N, K, E, int(swiglu), _TYPES[dtype])


def _mm_out(out, M, n, dtype, device):
    if out is None:
        return torch.empty(M, n, dtype=dtype, device=device)
    _need(out.is_cuda and out.dtype == dtype and out.is_contiguous() and tuple(out.shape) == (M, n),
          f"out must be a contiguous {dtype} GPU tensor [{M}, {n}]")
    return out


def mxfp4_matmul(a, a_scale, w, w_scale, offsets=None, swiglu: bool = False, dtype=torch.bfloat16, out=None,
                 stream=None):
    """y = a w^T of MXFP4 matrices: a uint8 [M, K/2] with tiled scales (mxfp4_quantize), w uint8 [E, N, K/2] with
    tiled scales (mxfp4_tile_scales).  offsets (int32 [E + 1]): rows [off[e], off[e+1]) use w[e], and a_scale is in
    the grouped layout of the same offsets.  Returns [M, N], or with swiglu silu(first half) * second half [M, N/2]."""
    _need(a.dim() == 2, "a must be uint8 [M, K/2]")
    _indices(None, 1, offsets)
    M, K = a.shape[0], 2 * a.shape[1]
    _bytes(a, "a", a.numel())
    dims = _mm_dims(M, K, w, w_scale, offsets, swiglu, dtype)
    _bytes(a_scale, "a_scale", (M // 128 + dims.E) * -(-K // 128) * 512)
    out = _mm_out(out, M, dims.N // 2 if swiglu else dims.N, dtype, a.device)
    rc = _lib().moe_fp4_mxfp4_matmul(ctypes.byref(dims), a.data_ptr(), a_scale.data_ptr(),
                                     None if offsets is None else offsets.data_ptr(), w.data_ptr(),
                                     w_scale.data_ptr(), out.data_ptr(), _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_matmul")
    return out


def mxfp4_linear_workspace_bytes(M: int, N: int, K: int, E: int = 1) -> int:
    return int(_lib().moe_fp4_mxfp4_linear_workspace_bytes(ctypes.byref(MmDims(M, N, K, E, 0, 0))))


def mxfp4_linear(x, w, w_scale, offsets=None, row_index=None, index_div: int = 1, swiglu: bool = False,
                 dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """The product from unquantised rows x [R, K] (bf16 or fp32): mxfp4_quantize (with row_index / index_div, and
    offsets) and mxfp4_matmul in one call, the same bits."""
    xt = _type(x, "x")
    stride = _rows2d(x, "x")
    _indices(row_index, index_div, offsets)
    R, K = x.shape
    _need(K > 0 and K % 32 == 0, "K must be a multiple of 32")
    M = R if row_index is None else row_index.numel()
    dims = _mm_dims(M, K, w, w_scale, offsets, swiglu, dtype)
    lib = _lib()
    nbytes = lib.moe_fp4_mxfp4_linear_workspace_bytes(ctypes.byref(dims))
    if nbytes == 0:
        raise MoeFp4Error(-2, "moe_fp4_mxfp4_linear")
    ws = _binding._workspace(nbytes, x.device, workspace)
    out = _mm_out(out, M, dims.N // 2 if swiglu else dims.N, dtype, x.device)
    rc = lib.moe_fp4_mxfp4_linear(ctypes.byref(dims), x.data_ptr(), xt, R, stride,
                                  None if row_index is None else row_index.data_ptr(), index_div,
                                  None if offsets is None else offsets.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                                  out.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_linear")
    return out


def _block_norm(a, stream):
    rc = _lib().moe_fp4_block_norm(ctypes.byref(a), _raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_block_norm")


def _weight(a, name, w, d):
    if w is None:
        return
    _need(w.is_cuda and w.is_contiguous() and tuple(w.shape) == (d,), f"{name} must be a contiguous GPU tensor [{d}]")
    setattr(a, name + "_type", _type(w, name))
    setattr(a, name, w.data_ptr())


def rms_norm(x, weight=None, eps: float = 1e-6, out=None, stream=None):
    """The norm before a block: bf16 [T, d] = x rsqrt(mean(x^2) + eps) * weight.  x bf16 or fp32 [T, d] (rows may
    be strided), weight bf16 or fp32 [d]."""
    a = BlockNormArgs()
    a.residual_stride = _rows2d(x, "x")
    T, d = x.shape
    a.T, a.d, a.eps, a.scale = T, d, eps, 1.0
    a.residual, a.residual_type = x.data_ptr(), _type(x, "x")
    _weight(a, "next_weight", weight, d)
    out = _mm_out(out, T, d, torch.bfloat16, x.device)
    a.normed = out.data_ptr()
    _block_norm(a, stream)
    return out


def block_residual(residual, y, y2=None, post_norm: bool = True, post_weight=None, gate=None,
                   gate_sigmoid: bool = False, scale: float = 1.0, next_norm: bool = True, next_weight=None,
                   eps: float = 1e-6, out=None, normed=None, stream=None):
    """The end of a block and the norm before the next one, in one pass:

      b = y (+ y2); post_norm: b *= rsqrt(mean(b^2) + eps); b *= post_weight; b *= gate or sigmoid(gate)
      out = residual + scale * b;  normed = out rsqrt(mean(out^2) + eps) * next_weight

    residual, y, y2: bf16 or fp32 [T, d], rows may be strided.  gate: [T], [d] or [T, d] (T = d: give [T, 1],
    [1, d] or [T, d]).  Returns (out, normed): out of residual's type (out=residual adds in place), normed bf16,
    or None with next_norm=False."""
    a = BlockNormArgs()
    a.residual_stride = _rows2d(residual, "residual")
    T, d = residual.shape
    a.T, a.d, a.eps, a.scale, a.post_norm = T, d, eps, scale, int(post_norm)
    a.residual, a.residual_type = residual.data_ptr(), _type(residual, "residual")
    _need(tuple(y.shape) == (T, d), f"y must be [{T}, {d}]")
    a.y, a.y_type, a.y_stride = y.data_ptr(), _type(y, "y"), _rows2d(y, "y")
    if y2 is not None:
        _need(tuple(y2.shape) == (T, d), f"y2 must be [{T}, {d}]")
        a.y2, a.y2_type, a.y2_stride = y2.data_ptr(), _type(y2, "y2"), _rows2d(y2, "y2")
    _weight(a, "post_weight", post_weight, d)
    if gate is not None:
        _need(gate.is_cuda, "gate must be a GPU tensor")
        shape = tuple(gate.shape)
        _need(not (len(shape) == 1 and T == d), "gate is ambiguous for T = d: give [T, 1] or [1, d]")
        if shape == (T, d) and not (T > 1 and d == 1):
            a.gate_shape, a.gate_stride = 3, _rows2d(gate, "gate")
        elif shape in ((T,), (T, 1)):
            _need(gate.is_contiguous(), "gate must be contiguous")
            a.gate_shape, a.gate_stride = 1, d
        elif shape in ((d,), (1, d)):
            _need(gate.is_contiguous(), "gate must be contiguous")
            a.gate_shape, a.gate_stride = 2, d
        else:
            raise ValueError(f"gate must be [T], [d] or [T, d], not {list(shape)}")
        a.gate, a.gate_type, a.gate_sigmoid = gate.data_ptr(), _type(gate, "gate"), int(gate_sigmoid)
    if out is residual:
        a.out_stride = a.residual_stride
    else:
        out = _mm_out(out, T, d, residual.dtype, residual.device)
        a.out_stride = d
    a.out = out.data_ptr()
    if next_norm:
        _weight(a, "next_weight", next_weight, d)
        normed = _mm_out(normed, T, d, torch.bfloat16, residual.device)
        a.normed = normed.data_ptr()
    else:
        _need(next_weight is None and normed is None, "next_norm=False takes no next_weight and no normed")
    _block_norm(a, stream)
    return out, normed


def ops_check(stream=None) -> None:
    """Synchronise and raise if a kernel of an earlier operator call on this device reported an error (a row index
    out of range, or a pipeline wait that ran out); the error word is cleared."""
    rc = _lib().moe_fp4_ops_check(_raw_stream(stream))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_ops_check")
