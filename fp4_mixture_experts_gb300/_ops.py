"""Binding of the operators around the layer: MXFP4 quantisation, products of
MXFP4 matrices (dense, and grouped by expert) and the end of a block.

Like _binding: argument marshalling only, on the current CUDA stream unless
one is given.  Wrong types, shapes or strides raise ValueError; a nonzero
status of the library becomes a MoeFp4Error.  `out`, `codes`, `scales` and
`workspace` may be given so that a call allocates nothing (a captured graph).
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _binding
from ._binding import MoeFp4Error, load_library

_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_BF16, _U8, _I32 = torch.bfloat16, torch.uint8, torch.int32
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
# struct moe_fp4_block_norm_args of include/moe_fp4.h: T; 10 int32; 5 strides; scale, eps; 8 pointers
_BLOCK_NORM = struct.Struct("q10i5q2f8Q")


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


# The checks below run on every call: plain `if`s, messages built only when they are raised.

def _raw_stream(stream, t):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw_stream is not None:  # the handle alone, without the Stream object around it
        return _current_raw_stream(t.get_device())
    return torch.cuda.current_stream().cuda_stream


def _type(t, what):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be bf16 or fp32, not {t.dtype}")
    return code


def _rows(t, what):
    """(rows, K, row stride) of a GPU tensor of rows: 2-D, contiguous along its rows, rows may be strided"""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{what} must be a 2-D GPU tensor")
    R, K = t.shape
    s0, s1 = t.stride()
    if (s1 != 1 and K > 1) or (s0 < K and R > 1):
        raise ValueError(f"{what} must have contiguous, separate rows")
    return R, K, s0 if R > 1 else K


def _bytes(t, what, numel):
    if t.dtype is not _U8 or not t.is_cuda or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{what} must be a contiguous uint8 GPU tensor of at least {numel} elements")


def _index_ptr(t, what):
    if t is None:
        return None
    if t.dtype is not _I32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 1-D int32 GPU tensor")
    return t.data_ptr()


def _groups(offsets):
    E = offsets.numel() - 1
    if E < 1:
        raise ValueError("offsets must have E + 1 elements")
    return E


def mxfp4_tiled_scale_bytes(rows: int, K: int, groups: int = 1) -> int:
    return int(_lib().moe_fp4_mxfp4_tiled_scale_bytes(rows, groups, K))


def mxfp4_quantize(x, row_index=None, index_div: int = 1, offsets=None, tiled: bool = False, codes=None, scales=None,
                   stream=None):
    """MXFP4 of rows x [R, K] (bf16 or fp32, K a multiple of 32; rows may be strided).

    Returns (codes uint8 [S, K/2], scales uint8): scales [S, K/32], or with tiled the layout of the products
    ([row tiles, ceil(K/128), 512]; by group with offsets, int32 [E + 1]).  row_index (int32 [S]) gathers: row r
    is row row_index[r] // index_div of x (sorted_slot and k of the layer's routing); without it S = R."""
    xt = _type(x, "x")
    R, K, stride = _rows(x, "x")
    if K % 32 or K == 0:
        raise ValueError("K must be a multiple of 32")
    S = R if row_index is None else row_index.numel()
    E = 1
    if offsets is not None:
        if not tiled:
            raise ValueError("offsets need tiled scales")
        E = _groups(offsets)
    index, off = _index_ptr(row_index, "row_index"), _index_ptr(offsets, "offsets")
    if codes is None:
        codes = torch.empty((S, K // 2), dtype=_U8, device=x.device)
    else:
        _bytes(codes, "codes", S * (K // 2))
    shape = (S // 128 + E, -(-K // 128), 512) if tiled else (S, K // 32)
    if scales is None:
        scales = torch.empty(shape, dtype=_U8, device=x.device)
    else:
        _bytes(scales, "scales", shape[0] * shape[1] * (512 if tiled else 1))
    rc = _lib().moe_fp4_mxfp4_quantize(x.data_ptr(), xt, R, stride, K, index, index_div, S, off, E, codes.data_ptr(),
                                       scales.data_ptr(), 1 if tiled else 0, _raw_stream(stream, x))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_quantize")
    return codes, scales


def mxfp4_dequantize(codes, scales, dtype=torch.bfloat16, out=None, stream=None):
    """The values (bf16 or fp32 [.., K]) of MXFP4 codes uint8 [.., K/2] with row-major scales uint8 [.., K/32]."""
    ot = _TYPES.get(dtype)
    if ot is None:
        raise ValueError("dtype must be bf16 or fp32")
    *lead, half = codes.shape
    K = 2 * half
    if K % 32 or K == 0:
        raise ValueError("K must be a multiple of 32")
    n = codes.numel()
    rows = n // half
    _bytes(codes, "codes", n)
    _bytes(scales, "scales", rows * (K // 32))
    if out is None:
        out = torch.empty((*lead, K), dtype=dtype, device=codes.device)
    elif not out.is_cuda or out.dtype is not dtype or not out.is_contiguous() or out.numel() != 2 * n:
        raise ValueError("out must be a contiguous GPU tensor of dtype with a value for each code")
    rc = _lib().moe_fp4_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, K, ot, out.data_ptr(),
                                         _raw_stream(stream, codes))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_dequantize")
    return out


def mxfp4_tile_scales(scales, swiglu: bool = False, out=None, stream=None):
    """Row-major weight scales uint8 [E, N, K/32] or [N, K/32] in the layout of the products, uint8
    [E, ceil(N/128), ceil(K/128), 512]: once, when weights are loaded.  swiglu: for products with SwiGLU."""
    if scales.dim() not in (2, 3):
        raise ValueError("scales must be [E, N, K/32] or [N, K/32]")
    E = scales.shape[0] if scales.dim() == 3 else 1
    N, nb = scales.shape[-2:]
    _bytes(scales, "scales", E * N * nb)
    shape = (E, -(-N // 128), -(-nb // 4), 512)
    if out is None:
        out = torch.empty(shape, dtype=_U8, device=scales.device)
    else:
        _bytes(out, "out", shape[0] * shape[1] * shape[2] * 512)
    rc = _lib().moe_fp4_mxfp4_tile_scales(scales.data_ptr(), E, N, 32 * nb, int(swiglu), out.data_ptr(),
                                          _raw_stream(stream, scales))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_tile_scales")
    return out


@functools.lru_cache(maxsize=1024)
def _mm_plan(M, N, K, E, swiglu, dtype):
    """What a product's sizes alone give: its dims (kept alive beside their address), features of y, scale bytes of
    both operands, workspace bytes of the linear form"""
    yt = _TYPES.get(dtype)
    if yt is None:
        raise ValueError("dtype must be bf16 or fp32")
    if swiglu and N % 2:
        raise ValueError("swiglu needs an even number of features")
    dims = MmDims(M, N, K, E, int(swiglu), yt)
    kt = -(-K // 128)
    return (ctypes.addressof(dims), N // 2 if swiglu else N, E * -(-N // 128) * kt * 512, (M // 128 + E) * kt * 512,
            _lib().moe_fp4_mxfp4_linear_workspace_bytes(ctypes.byref(dims)), dims)


def _plan_of(M, K, w, w_scale, offsets, swiglu, dtype):
    shape = w.shape
    if len(shape) == 3:
        E, N, half = shape
    elif len(shape) == 2:
        E, (N, half) = 1, shape
    else:
        raise ValueError("w must be uint8 [E, N, K/2] or [N, K/2]")
    if 2 * half != K:
        raise ValueError(f"w must be uint8 [E, N, K/2] or [N, K/2] with K = {K}")
    if (offsets.numel() != E + 1) if offsets is not None else E != 1:
        raise ValueError("several matrices need offsets, of E + 1 elements")
    plan = _mm_plan(M, N, K, E, swiglu, dtype)
    _bytes(w, "w", 0)
    _bytes(w_scale, "w_scale (tiled, by mxfp4_tile_scales)", plan[2])
    return plan


def _result(out, M, n, dtype, device):
    if out is None:
        return torch.empty((M, n), dtype=dtype, device=device)
    if not out.is_cuda or out.dtype is not dtype or not out.is_contiguous() or out.shape != (M, n):
        raise ValueError(f"out must be a contiguous {dtype} GPU tensor [{M}, {n}]")
    return out


def mxfp4_matmul(a, a_scale, w, w_scale, offsets=None, swiglu: bool = False, dtype=torch.bfloat16, out=None,
                 stream=None):
    """y = a w^T of MXFP4 matrices: a uint8 [M, K/2] with tiled scales (mxfp4_quantize), w uint8 [E, N, K/2] with
    tiled scales (mxfp4_tile_scales).  offsets (int32 [E + 1]): rows [off[e], off[e+1]) use w[e], and a_scale is in
    the grouped layout of the same offsets.  Returns [M, N], or with swiglu silu(first half) * second half [M, N/2]."""
    if a.dim() != 2:
        raise ValueError("a must be uint8 [M, K/2]")
    M, K = a.shape[0], 2 * a.shape[1]
    off = _index_ptr(offsets, "offsets")
    dims, n, _, a_bytes, _, _ = _plan_of(M, K, w, w_scale, offsets, swiglu, dtype)
    _bytes(a, "a", 0)
    _bytes(a_scale, "a_scale (tiled)", a_bytes)
    out = _result(out, M, n, dtype, a.device)
    rc = _lib().moe_fp4_mxfp4_matmul(dims, a.data_ptr(), a_scale.data_ptr(), off, w.data_ptr(), w_scale.data_ptr(),
                                     out.data_ptr(), _raw_stream(stream, a))
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
    R, K, stride = _rows(x, "x")
    M = R if row_index is None else row_index.numel()
    index, off = _index_ptr(row_index, "row_index"), _index_ptr(offsets, "offsets")
    dims, n, _, _, nbytes, _ = _plan_of(M, K, w, w_scale, offsets, swiglu, dtype)
    if nbytes == 0:
        raise MoeFp4Error(-2, "moe_fp4_mxfp4_linear")
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=_U8, device=x.device)
    else:
        _bytes(workspace, "workspace", nbytes)
    out = _result(out, M, n, dtype, x.device)
    rc = _lib().moe_fp4_mxfp4_linear(dims, x.data_ptr(), xt, R, stride, index, index_div, off, w.data_ptr(),
                                     w_scale.data_ptr(), out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                     _raw_stream(stream, x))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_mxfp4_linear")
    return out


def _weight(w, what, d):
    """(pointer, type) of a weight [d], (0, 0) for none"""
    if w is None:
        return 0, 0
    if not w.is_cuda or not w.is_contiguous() or w.shape != (d,):
        raise ValueError(f"{what} must be a contiguous GPU tensor [{d}]")
    return w.data_ptr(), _type(w, what)


def rms_norm(x, weight=None, eps: float = 1e-6, out=None, stream=None):
    """The norm before a block: bf16 [T, d] = x rsqrt(mean(x^2) + eps) * weight.  x bf16 or fp32 [T, d] (rows may
    be strided), weight bf16 or fp32 [d]."""
    T, d, stride = _rows(x, "x")
    wp, wt = _weight(weight, "weight", d)
    out = _result(out, T, d, _BF16, x.device)
    rc = _lib().moe_fp4_block_norm(
        _BLOCK_NORM.pack(T, d, 0, 0, 0, _type(x, "x"), 0, 0, 0, 0, wt, stride, 0, 0, 0, 0, 1.0, eps, x.data_ptr(), 0, 0, 0,
                         0, wp, 0, out.data_ptr()), _raw_stream(stream, x))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_block_norm")
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
    T, d, r_stride = _rows(residual, "residual")
    rt = _type(residual, "residual")
    shape = residual.shape
    if y.shape != shape:
        raise ValueError(f"y must be [{T}, {d}]")
    y_stride, yt = _rows(y, "y")[2], _type(y, "y")
    y2p = y2t = y2_stride = gp = gt = g_shape = g_stride = 0
    if y2 is not None:
        if y2.shape != shape:
            raise ValueError(f"y2 must be [{T}, {d}]")
        y2p, y2t, y2_stride = y2.data_ptr(), _type(y2, "y2"), _rows(y2, "y2")[2]
    pp, pt = _weight(post_weight, "post_weight", d)
    if gate is not None:
        g = gate.shape
        if g == shape and not (T > 1 and d == 1):
            g_shape, g_stride = 3, _rows(gate, "gate")[2]
        else:
            if len(g) == 1 and T == d:
                raise ValueError("gate is ambiguous for T = d: give [T, 1] or [1, d]")
            g_shape, g_stride = (1 if g == (T,) or g == (T, 1) else 2 if g == (d,) or g == (1, d) else 0), d
            if g_shape == 0 or not gate.is_cuda or not gate.is_contiguous():
                raise ValueError(f"gate must be a GPU tensor [T], [d] or [T, d], not {list(g)}")
        gp, gt = gate.data_ptr(), _type(gate, "gate")
    if out is residual:
        o_stride = r_stride
    else:
        out = _result(out, T, d, residual.dtype, residual.device)
        o_stride = d
    npt = nwp = nwt = 0
    if next_norm:
        nwp, nwt = _weight(next_weight, "next_weight", d)
        normed = _result(normed, T, d, _BF16, residual.device)
        npt = normed.data_ptr()
    elif next_weight is not None or normed is not None:
        raise ValueError("next_norm=False takes no next_weight and no normed")
    rc = _lib().moe_fp4_block_norm(
        _BLOCK_NORM.pack(T, d, 1 if post_norm else 0, g_shape, 1 if gate_sigmoid else 0, rt, yt, y2t, gt, pt, nwt,
                         r_stride, y_stride, y2_stride, g_stride, o_stride, scale, eps, residual.data_ptr(),
                         y.data_ptr(), y2p, gp, pp, nwp, out.data_ptr(), npt), _raw_stream(stream, residual))
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_block_norm")
    return out, normed


def ops_check(stream=None) -> None:
    """Synchronise and raise if a kernel of an earlier operator call on this device reported an error (a row index
    out of range, or a pipeline wait that ran out); the error word is cleared."""
    rc = _lib().moe_fp4_ops_check((stream or torch.cuda.current_stream()).cuda_stream)
    if rc != 0:
        raise MoeFp4Error(rc, "moe_fp4_ops_check")
