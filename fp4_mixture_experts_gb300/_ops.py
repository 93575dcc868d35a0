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
from typing import NamedTuple

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


class PageSlotsArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "page", "width")] +
                [(n, ctypes.c_int64) for n in ("tokens", "free_count", "table_stride")] +
                [(n, ctypes.c_void_p) for n in ("lengths", "new_tokens", "free_pages", "table", "slots", "positions",
                                                "out_lengths", "q_offsets", "k_offsets", "taken")])


class LatentAttentionArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "H", "causal")] + [("scale", ctypes.c_float)] +
                [(n, ctypes.c_int64) for n in ("Tq", "Tk", "q_stride", "q_head_stride", "kv_stride", "kv_head_stride",
                                               "rope_stride")] +
                [(n, ctypes.c_void_p) for n in ("q", "kv", "k_rope", "q_offsets", "k_offsets", "out")])


class LatentDecodeArgs(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("B", "H", "page", "pages", "width")] + [("scale", ctypes.c_float)] +
                [(n, ctypes.c_int64) for n in ("q_stride", "q_head_stride", "table_stride")] +
                [(n, ctypes.c_void_p) for n in ("q", "cache", "table", "lengths", "out")])


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
            "mxfp4_linear_workspace_bytes", "mxfp4_gathered_workspace_bytes", "block_norm", "fp8_tile_scales",
            "fp8_linear_workspace_bytes", "fp8_linear", "latent_decode_workspace_bytes", "latent_decode",
            "latent_attention_workspace_bytes", "latent_attention", "page_slots")), _raise)
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


def fp8_tile_scales(scales, N: int, K: int, swiglu: bool = False, out=None, stream=None):
    """E8M0 weight scales uint8 [E, ceil(N/128), ceil(K/128)] (or without E), one for each 128 x 128 of w [E, N, K], in
    the layout of fp8_linear, uint8 [E, ceil(N/128), ceil(K/128), 512]: once, when weights are loaded.  swiglu: for
    products with SwiGLU."""
    return _native.fp8_tile_scales(scales, N, K, swiglu, out, _handle(stream))


def fp8_linear_workspace_bytes(M: int, N: int, K: int, E: int = 1) -> int:
    """Bytes of fp8_linear's workspace."""
    return int(load_library().moe_fp4_fp8_linear_workspace_bytes(ctypes.byref(MmDims(M, N, K, E, 0, 0))))


def fp8_linear(x, w, w_scale, offsets=None, swiglu: bool = False, dtype=None, out=None, workspace=None, stream=None):
    """y = x_q w^T of rows x [M, K] (bf16 or fp32, K a multiple of 32; rows may be strided), quantised in the call to
    E4M3 with a power-of-two scale for each 128 elements, and weights w float8_e4m3fn [E, N, K] or [N, K] with scales
    of fp8_tile_scales.  offsets (int32 [E + 1]): rows [off[e], off[e+1]) use w[e]; rows in no group are left as they
    were.  Returns [M, N], or with swiglu silu(first half) * second half [M, N/2]: bf16, or dtype=torch.float32."""
    f = _native.fp8_linear
    return f(x, w, w_scale, offsets, swiglu, dtype or _BF16, out, workspace, _handle(stream))


def latent_decode_workspace_bytes(H: int) -> int:
    """Bytes of latent_decode's workspace on the current device."""
    return int(load_library().moe_fp4_latent_decode_workspace_bytes(H))


def latent_decode(q, cache, block_table, lengths, scale, out=None, workspace=None, stream=None):
    """Latent attention of one new token a sequence in its absorbed form, over a paged cache: bf16 [B, H, 512],

      out[b, h] = sum_j softmax(scale q[b, h] . c_j) c_j[:512],   j < lengths[b]

    q bf16 [B, H, 576] (latent part, rotary part; heads that start on 16 bytes), cache bf16 [pages, page, 576] (page a
    multiple of 16), block_table int32 [B, width]: the pages of each sequence, lengths int32 [B].  What the cache holds
    behind a sequence's end is not used; a sequence of no tokens gets zeros.  Lengths that the table does not hold and
    pages outside the cache are reported by ops_check."""
    return _native.latent_decode(q, cache, block_table, lengths, scale, out, workspace, _handle(stream))


def latent_attention_workspace_bytes() -> int:
    """Bytes of latent_attention's workspace on the current device."""
    return int(load_library().moe_fp4_latent_attention_workspace_bytes())


def latent_attention(q, kv, k_rope, q_offsets, k_offsets, scale, causal: bool = True, out=None, workspace=None, stream=None):
    """Latent attention in its expanded form for the new tokens of a ragged batch: bf16 [Tq, H, 128],

      out[i, h] = sum_j softmax(scale (q[i, h, :128] . kv[j, h, :128] + q[i, h, 128:] . k_rope[j])) kv[j, h, 128:]

    q bf16 [Tq, H, 192], kv bf16 [Tk, H, 256] (keys and values of a head side by side, as the latent vectors' up
    projection writes them), k_rope bf16 [Tk, 64]; heads and rows start on 16 bytes.  Sequence b has queries
    [q_offsets[b], q_offsets[b+1]) and keys [k_offsets[b], k_offsets[b+1]) (int32 [B + 1]); causal: its last query sees
    all keys, each one before it one less.  A query that sees no key gets zeros, queries of no sequence are left as
    they were.  Offsets that decrease or lie behind the rows (but for 2^31 - 1, their end) are reported by ops_check.
    Values are to be finite; scale is positive."""
    return _native.latent_attention(q, kv, k_rope, q_offsets, k_offsets, scale, causal, out, workspace, _handle(stream))


class PageSlots(NamedTuple):
    """What page_slots returns (GPU tensors)."""
    slots: object      # int64 [tokens]: page * page_size + place in it; -1: none (block.write_rows leaves such tokens out)
    positions: object  # int32 [tokens]
    lengths: object    # int32 [B], with the new tokens that have a place
    q_offsets: object  # int32 [B + 1], of the new tokens
    k_offsets: object  # int32 [B + 1], of all tokens of lengths
    taken: object      # int32 []: pages taken from the front of free_pages


def page_slots(lengths, new_tokens, block_table, free_pages, page_size: int, tokens: int, out: PageSlots | None = None,
               stream=None) -> PageSlots:
    """Places of a batch's new tokens in a paged cache.  Request b has lengths[b] tokens and gets new_tokens[b] more (int32
    [B], B up to 8192); the pages that they need are taken from the front of free_pages (int32), request after request,
    and entered in block_table (int32 [B, width], in place).  tokens: the size of slots and positions, at least the
    number of new tokens; behind the last one slots are -1.  out: an earlier result of the same sizes, to be
    overwritten.  Requests that their rows do not hold, too few free pages or too many tokens are reported by
    ops_check; the tokens without a place have slot -1 and are not in lengths and k_offsets."""
    f = _native.page_slots
    return PageSlots(*f(lengths, new_tokens, block_table, free_pages, page_size, tokens, *(out or (None,) * 6),
                        _handle(stream)))


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
