"""The operators' calls with tensors on different GPUs, or beside the GPU, are
refused before CUDA is asked for anything.  Fake tensors stand for two GPUs; no
memory is behind them and none is touched."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp4_mixture_experts_gb300 as moe

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


def on(device, *shape, dtype=BF):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def calls(other):
    """one operand of each call on `other`, all the rest on the first GPU"""
    x, y, d = on("cuda:0", 4, 64), on(other, 4, 64), on(other, 64)
    w, ws = on("cuda:0", 8, 32, dtype=U8), on("cuda:0", 1, 1, 1, 512, dtype=U8)
    w_o, ws_o = on(other, 8, 32, dtype=U8), on(other, 1, 1, 1, 512, dtype=U8)
    i = on(other, 4, dtype=I32)
    return {
        "quantize index": lambda: moe.mxfp4_quantize(x, row_index=i),
        "quantize offsets": lambda: moe.mxfp4_quantize(x, offsets=i, tiled=True),
        "quantize codes": lambda: moe.mxfp4_quantize(x, codes=on(other, 4, 32, dtype=U8)),
        "dequantize scales": lambda: moe.mxfp4_dequantize(w, on(other, 8, 2, dtype=U8)),
        "dequantize out": lambda: moe.mxfp4_dequantize(w, on("cuda:0", 8, 2, dtype=U8), out=on(other, 8, 64)),
        "tile scales out": lambda: moe.mxfp4_tile_scales(on("cuda:0", 8, 2, dtype=U8), out=ws_o),
        "matmul a_scale": lambda: moe.mxfp4_matmul(w, ws_o, w, ws),
        "matmul w": lambda: moe.mxfp4_matmul(w, ws, w_o, ws),
        "linear w": lambda: moe.mxfp4_linear(x, w_o, ws),
        "linear w_scale": lambda: moe.mxfp4_linear(x, w, ws_o),
        "linear index": lambda: moe.mxfp4_linear(x, w, ws, row_index=i),
        "linear out": lambda: moe.mxfp4_linear(x, w, ws, out=on(other, 4, 8)),
        "linear workspace": lambda: moe.mxfp4_linear(x, w, ws, workspace=on(other, 4096, dtype=U8)),
        "rms_norm weight": lambda: moe.rms_norm(x, d),
        "rms_norm out": lambda: moe.rms_norm(x, out=y),
        "block_residual y": lambda: moe.block_residual(x, y),
        "block_residual y2": lambda: moe.block_residual(x, x, y2=y),
        "block_residual gate": lambda: moe.block_residual(x, x, gate=d),
        "block_residual weight": lambda: moe.block_residual(x, x, post_weight=d),
        "block_residual next": lambda: moe.block_residual(x, x, next_weight=d),
        "block_residual out": lambda: moe.block_residual(x, x, out=y),
        "block_residual normed": lambda: moe.block_residual(x, x, normed=y),
    }


@pytest.mark.parametrize("other,message", [("cuda:1", "same GPU"), ("cpu", "GPU tensors")])
@pytest.mark.parametrize("name", list(calls("cpu")))
def test_operands_elsewhere_are_refused(name, other, message):
    with pytest.raises(ValueError, match=message):
        calls(other)[name]()
