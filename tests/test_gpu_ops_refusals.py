"""Wrong operands of the operators' Python calls, GPU tensors all: each is
refused before anything is enqueued, with the exception that the interface
names and no other left behind."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def scales(N, K, E=1):
    return z(E, -(-N // 128), -(-K // 128), 512, dtype=U8)


def quantize(x=(40, 64), x_type=BF, **kw):
    return moe.mxfp4_quantize(x if isinstance(x, torch.Tensor) else z(*x, dtype=x_type), **kw)


def dequantize(codes=(8, 32), s=(8, 2), codes_type=U8, **kw):
    return moe.mxfp4_dequantize(codes if isinstance(codes, torch.Tensor) else z(*codes, dtype=codes_type), z(*s, dtype=U8), **kw)


def linear(x=(40, 64), w=(8, 32), ws=None, x_type=BF, w_type=U8, **kw):
    return moe.mxfp4_linear(x if isinstance(x, torch.Tensor) else z(*x, dtype=x_type), z(*w, dtype=w_type),
                            scales(w[-2], 2 * w[-1], w[0] if len(w) == 3 else 1) if ws is None else ws, **kw)


def matmul(a=(40, 32), s=None, w=(8, 32), **kw):
    return moe.mxfp4_matmul(z(*a, dtype=U8), scales(40, 64) if s is None else s, z(*w, dtype=U8), scales(8, 64), **kw)


def end(r=(6, 64), y=(6, 64), **kw):
    return moe.block_residual(r if isinstance(r, torch.Tensor) else z(*r), y if isinstance(y, torch.Tensor) else z(*y), **kw)


BOTH = np.ones(2)  # neither true nor false

REFUSED = {
    "quantize: half": lambda: quantize(x_type=torch.float16),
    "quantize: one dimension": lambda: quantize((64,)),
    "quantize: K of 48": lambda: quantize((4, 48)),
    "quantize: no K": lambda: quantize((4, 0)),
    "quantize: columns apart": lambda: quantize(z(64, 40).t()),
    "quantize: rows over one another": lambda: quantize(z(1, 64).expand(4, 64)),
    "quantize: not a tensor": lambda: moe.mxfp4_quantize([[1.0] * 32]),
    "quantize: int64 index": lambda: quantize(row_index=z(4, dtype=torch.int64)),
    "quantize: 2-D index": lambda: quantize(row_index=z(4, 1, dtype=I32)),
    "quantize: strided index": lambda: quantize(row_index=z(8, dtype=I32)[::2]),
    "quantize: division by 0": lambda: quantize(row_index=z(4, dtype=I32), index_div=0),
    "quantize: division by a fraction": lambda: quantize(row_index=z(4, dtype=I32), index_div=1.5),
    "quantize: groups without tiles": lambda: quantize(offsets=z(2, dtype=I32)),
    "quantize: one offset": lambda: quantize(offsets=z(1, dtype=I32), tiled=True),
    "quantize: small codes": lambda: quantize(codes=z(39, 32, dtype=U8)),
    "quantize: int8 codes": lambda: quantize(codes=z(40, 32, dtype=torch.int8)),
    "quantize: small scales": lambda: quantize(tiled=True, scales=z(511, dtype=U8)),
    "quantize: tiled neither": lambda: quantize(tiled=BOTH),
    "dequantize: fp16": lambda: dequantize(dtype=torch.float16),
    "dequantize: half a block": lambda: dequantize((8, 8)),
    "dequantize: int8": lambda: dequantize(codes_type=torch.int8),
    "dequantize: small scales": lambda: dequantize(s=(8, 1)),
    "dequantize: codes apart": lambda: dequantize(z(8, 64, dtype=U8)[:, ::2]),
    "dequantize: out's type": lambda: dequantize(out=z(8, 64, dtype=F32)),
    "dequantize: out's size": lambda: dequantize(out=z(8, 32)),
    "tile scales: one dimension": lambda: moe.mxfp4_tile_scales(z(8, dtype=U8)),
    "tile scales: small out": lambda: moe.mxfp4_tile_scales(z(129, 2, dtype=U8), out=z(512, dtype=U8)),
    "tile scales: swiglu neither": lambda: moe.mxfp4_tile_scales(z(8, 2, dtype=U8), BOTH),
    "linear: another K": lambda: linear(w=(8, 48)),
    "linear: w of bf16": lambda: linear(w_type=BF),
    "linear: w of one dimension": lambda: linear(w=(1, 1, 1, 32), ws=scales(8, 64)),
    "linear: several matrices without offsets": lambda: linear(w=(2, 8, 32)),
    "linear: offsets of another number": lambda: linear(w=(2, 8, 32), offsets=z(2, dtype=I32)),
    "linear: int64 offsets": lambda: linear(w=(2, 8, 32), offsets=z(3, dtype=torch.int64)),
    "linear: small scales": lambda: linear(w=(129, 32), ws=scales(128, 64)),
    "linear: odd features": lambda: linear(w=(7, 32), swiglu=True),
    "linear: fp16 result": lambda: linear(dtype=torch.float16),
    "linear: not a type": lambda: linear(dtype="bf16"),
    "linear: out's width": lambda: linear(out=z(40, 7)),
    "linear: out's rows": lambda: linear(out=z(39, 8)),
    "linear: out's width with swiglu": lambda: linear(swiglu=True, out=z(40, 8)),
    "linear: out's type": lambda: linear(out=z(40, 8, dtype=F32)),
    "linear: out's strides": lambda: linear(out=z(40, 16)[:, :8]),
    "linear: small workspace": lambda: linear(workspace=z(moe.mxfp4_linear_workspace_bytes(40, 8, 64) - 1, dtype=U8)),
    "linear: workspace's type": lambda: linear(workspace=z(1 << 16)),
    "linear: swiglu neither": lambda: linear(swiglu=BOTH),
    "linear: columns apart": lambda: linear(z(64, 40).t()),
    "matmul: small a_scale": lambda: matmul(s=z(511, dtype=U8)),
    "matmul: a of one dimension": lambda: matmul(a=(32,)),
    "matmul: offsets of another number": lambda: matmul(offsets=z(3, dtype=I32)),
    "rms_norm: half": lambda: moe.rms_norm(z(4, 64, dtype=torch.float16)),
    "rms_norm: weight's width": lambda: moe.rms_norm(z(4, 64), z(63)),
    "rms_norm: weight of two dimensions": lambda: moe.rms_norm(z(4, 64), z(1, 64)),
    "rms_norm: weight's strides": lambda: moe.rms_norm(z(4, 64), z(128)[::2]),
    "rms_norm: eps": lambda: moe.rms_norm(z(4, 64), eps="small"),
    "rms_norm: fp32 out": lambda: moe.rms_norm(z(4, 64), out=z(4, 64, dtype=F32)),
    "end: y's rows": lambda: end(y=(5, 64)),
    "end: y's width": lambda: end(y=(6, 32)),
    "end: y2's rows": lambda: end(y2=z(5, 64)),
    "end: one row for all": lambda: end(y=z(1, 64).expand(6, 64)),
    "end: post_weight's width": lambda: end(post_weight=z(63)),
    "end: gate's width": lambda: end(gate=z(5)),
    "end: gate's shape": lambda: end(gate=z(64, 6)),
    "end: gate of three dimensions": lambda: end(gate=z(1, 6, 64)),
    "end: gate of none": lambda: end(gate=torch.zeros((), device=DEV)),
    "end: gate's type": lambda: end(gate=z(6, dtype=torch.int32)),
    "end: gate's strides": lambda: end(gate=z(12)[::2]),
    "end: one gate for T = d": lambda: end((64, 64), (64, 64), gate=z(64)),
    "end: gate_sigmoid neither": lambda: end(gate=z(6), gate_sigmoid=BOTH),
    "end: post_norm neither": lambda: end(post_norm=BOTH),
    "end: next_norm neither": lambda: end(next_norm=BOTH),
    "end: scale": lambda: end(scale="half"),
    "end: weight of no next norm": lambda: end(next_norm=False, next_weight=z(64)),
    "end: result of no next norm": lambda: end(next_norm=False, normed=z(6, 64)),
    "end: out's type": lambda: end(out=z(6, 64, dtype=F32)),
    "end: out's strides": lambda: end(out=z(6, 128)[:, :64]),
    "end: normed's type": lambda: end(normed=z(6, 64, dtype=F32)),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()


@pytest.mark.parametrize("call", [lambda: linear((40, 48), (8, 24), ws=scales(8, 64)),       # K no multiple of 32
                                  lambda: linear((20, 32800), (8, 16400)),                    # beyond 32768
                                  lambda: quantize((4, 32800)),
                                  lambda: moe.rms_norm(z(2, 16385)),
                                  lambda: moe.rms_norm(z(2, 64), eps=-1.0),
                                  lambda: linear(workspace=z(1 << 16, dtype=U8)[8:])])        # not on 256 bytes
def test_refused_by_the_library(call):
    with pytest.raises(moe.MoeFp4Error):
        call()


def test_a_gate_for_T_equal_d_by_its_shape():
    r, y = z(64, 64, dtype=F32), torch.ones(64, 64, device=DEV)
    g = torch.arange(64.0, device=DEV)
    for gate in (g[:, None], g[None], g.expand(64, 64).contiguous()):
        out, _ = moe.block_residual(r, y, post_norm=False, gate=gate)
        assert torch.equal(out, gate.expand(64, 64))


def test_the_device_is_as_it_was():
    torch.cuda.synchronize()
    moe.ops_check()
