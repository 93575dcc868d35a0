"""Refusals of the operators around the layer, without a GPU: every bad
argument is caught on the host, before anything is enqueued."""
import ctypes
import os

import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import BlockNormArgs, MmDims

P = ctypes.c_void_p
FAKE = 0x100000  # never dereferenced: every call below fails its host-side checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


def test_quantize(lib):
    good = dict(x=FAKE, x_type=0, x_rows=8, stride=64, K=64, index=None, div=1, rows=8, off=None, groups=1, codes=FAKE,
                scales=FAKE, tiled=0)

    def call(**kw):
        a = {**good, **kw}
        return lib.moe_fp4_mxfp4_quantize(*[a[k] for k in good], None)

    for bad in (dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, x_type=1), dict(x_type=2), dict(x_rows=-1), dict(x_rows=7),
                dict(stride=63), dict(K=0), dict(K=48), dict(K=-32), dict(K=32800, stride=32800), dict(rows=-1),
                dict(rows=1 << 31, x_rows=1 << 31), dict(index=FAKE, div=0), dict(index=FAKE + 2), dict(codes=None),
                dict(codes=FAKE + 8), dict(scales=None), dict(tiled=1, scales=FAKE + 8), dict(off=FAKE),
                dict(off=FAKE, tiled=1, groups=0), dict(off=FAKE, tiled=1, groups=1025),
                dict(off=FAKE + 2, tiled=1, groups=2)):
        assert call(**bad) == -1, bad
    assert call(rows=0, x=None, codes=None, scales=None) == 0
    assert call(rows=0, K=48) == -1


def test_dequantize_and_scale_layout(lib):
    d = lib.moe_fp4_mxfp4_dequantize
    for bad in ((None, FAKE, 4, 64, 0, FAKE), (FAKE, None, 4, 64, 0, FAKE), (FAKE, FAKE, 4, 64, 0, None),
                (FAKE, FAKE, -1, 64, 0, FAKE), (FAKE, FAKE, 4, 40, 0, FAKE), (FAKE, FAKE, 4, 64, 5, FAKE),
                (FAKE + 4, FAKE, 4, 64, 0, FAKE), (FAKE, FAKE, 4, 64, 0, FAKE + 8)):
        assert d(*bad, None) == -1, bad
    assert d(None, None, 0, 64, 0, None, None) == 0
    t = lib.moe_fp4_mxfp4_tile_scales
    for bad in ((None, 1, 8, 64, 0, FAKE), (FAKE, 0, 8, 64, 0, FAKE), (FAKE, 1025, 8, 64, 0, FAKE),
                (FAKE, 1, 0, 64, 0, FAKE), (FAKE, 1, 8, 65, 0, FAKE), (FAKE, 1, 7, 64, 1, FAKE),
                (FAKE, 1, 8, 64, 0, FAKE + 8), (FAKE, 1, 8, 64, 0, None)):
        assert t(*bad, None) == -1, bad
    b = moe.mxfp4_tiled_scale_bytes
    assert b(1, 32) == 512 and b(128, 128) == 1024 and b(127, 160, 3) == 3 * 2 * 512
    assert b(-1, 32) == 0 and b(1, 33) == 0 and b(1, 32, 0) == 0 and b(1, 32, 1025) == 0


def test_products(lib):
    dims = dict(M=40, N=8, K=64, E=1, swiglu=0, y_type=0)

    def matmul(a=FAKE, s=FAKE, off=None, w=FAKE, ws=FAKE, y=FAKE, null_dims=False, **kw):
        d = MmDims(*{**dims, **kw}.values())
        return lib.moe_fp4_mxfp4_matmul(None if null_dims else ctypes.byref(d), a, s, off, w, ws, y, None)

    for bad in (dict(null_dims=True), dict(M=-1), dict(N=0), dict(K=0), dict(K=40), dict(K=32800), dict(E=0), dict(E=1025, off=FAKE),
                dict(swiglu=2), dict(swiglu=1, N=7), dict(y_type=2), dict(a=None), dict(s=None), dict(w=None), dict(ws=None),
                dict(y=None), dict(E=2), dict(a=FAKE + 8), dict(s=FAKE + 8), dict(w=FAKE + 8), dict(ws=FAKE + 8), dict(y=FAKE + 1),
                dict(y=FAKE + 2, y_type=1), dict(E=2, off=FAKE + 2)):
        assert matmul(**bad) == -1, bad
    assert matmul(M=0, a=None, w=None, y=None) == 0
    assert matmul(M=1 << 30, K=64, N=1 << 20) == -2

    def linear(x=FAKE, xt=0, x_rows=40, stride=64, index=None, div=1, off=None, w=FAKE, ws=FAKE, y=FAKE, work=FAKE, size=1 << 30,
               **kw):
        d = MmDims(*{**dims, **kw}.values())
        return lib.moe_fp4_mxfp4_linear(ctypes.byref(d), x, xt, x_rows, stride, index, div, off, w, ws, y, work, size, None)

    need = moe.mxfp4_linear_workspace_bytes(40, 8, 64)
    assert need > 0 and moe.mxfp4_linear_workspace_bytes(40, 8, 65) == 0
    for bad in (dict(x=None), dict(xt=3), dict(x_rows=39), dict(stride=32), dict(index=FAKE, div=0), dict(w=None), dict(y=None),
                dict(work=None), dict(work=FAKE + 16), dict(E=2), dict(K=33)):
        assert linear(**bad) == -1, bad
    assert linear(size=need - 1) == -3
    assert linear(M=0, x=None, work=None) == 0
    assert linear(M=16, x_rows=16, E=2, off=FAKE, work=None) == -1  # few rows need none, but not with offsets


def test_block_norm(lib):
    base = dict(T=4, d=64, residual=FAKE, residual_stride=64, y=FAKE, y_stride=64, out=FAKE, out_stride=64, normed=FAKE,
                scale=1.0, eps=1e-6)

    def call(**kw):
        a = BlockNormArgs()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return lib.moe_fp4_block_norm(ctypes.byref(a), None)

    assert lib.moe_fp4_block_norm(None, None) == -1
    for bad in (dict(T=-1), dict(d=0), dict(d=16385), dict(eps=-1.0), dict(eps=float("nan")), dict(residual=None),
                dict(out=None), dict(out=None, normed=None, y=None), dict(residual_type=2), dict(residual_stride=63),
                dict(y_stride=63), dict(y_type=7), dict(y=FAKE + 1), dict(y=FAKE + 2, y_type=1), dict(gate_shape=4),
                dict(gate_shape=1), dict(gate=FAKE), dict(gate=FAKE, gate_shape=3, gate_stride=63), dict(y=None, post_norm=1),
                dict(y=None, y2=FAKE, y2_stride=64), dict(y=None, post_weight=FAKE), dict(y=None, gate=FAKE, gate_shape=1),
                dict(y2=FAKE, y2_stride=3), dict(out_stride=63), dict(normed=None, next_weight=FAKE),
                dict(normed=FAKE + 1), dict(post_weight=FAKE + 1), dict(next_weight=FAKE, next_weight_type=9)):
        assert call(**bad) == -1, bad
    assert call(T=0, residual=None) == 0


def test_the_binding_checks_shapes_and_types(lib):
    """CPU tensors: the binding refuses them, and every wrong shape, before it calls the library"""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w, ws = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 1, 1, 512, dtype=torch.uint8)
    for call in (lambda: moe.mxfp4_quantize(x), lambda: moe.mxfp4_quantize(x.half()),
                 lambda: moe.mxfp4_linear(x, w, ws), lambda: moe.mxfp4_matmul(w, ws, w, ws),
                 lambda: moe.mxfp4_dequantize(w, w), lambda: moe.mxfp4_dequantize(w, w, dtype=torch.float16),
                 lambda: moe.mxfp4_tile_scales(w), lambda: moe.rms_norm(x), lambda: moe.block_residual(x, x)):
        with pytest.raises(ValueError):
            call()
