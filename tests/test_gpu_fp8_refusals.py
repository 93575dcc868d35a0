"""Wrong operands of the FP8 products' Python calls, GPU tensors all: each is
refused before anything is enqueued."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests.test_gpu_ops_refusals import BF, BOTH, F32, I32, U8, scales, z

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def linear(x=(40, 64), w=(8, 64), ws=None, x_type=BF, w_type=F8, **kw):
    w = w if isinstance(w, torch.Tensor) else z(*w, dtype=w_type)
    return moe.fp8_linear(x if isinstance(x, torch.Tensor) else z(*x, dtype=x_type), w,
                          scales(w.shape[-2], w.shape[-1], w.shape[0] if w.dim() == 3 else 1) if ws is None else ws, **kw)


REFUSED = {
    "half": lambda: linear(x_type=torch.float16),
    "not a tensor": lambda: moe.fp8_linear([[1.0] * 64], z(8, 64, dtype=F8), scales(8, 64)),
    "one dimension": lambda: linear(z(64)),
    "columns apart": lambda: linear(z(64, 40).t()),
    "rows over one another": lambda: linear(z(1, 64).expand(4, 64)),
    "another K": lambda: linear(w=(8, 96)),
    "w of bytes": lambda: linear(w_type=U8),
    "w of e5m2": lambda: linear(w_type=torch.float8_e5m2),
    "w of four dimensions": lambda: linear(w=(1, 1, 1, 64), ws=scales(8, 64)),
    "w's strides": lambda: linear(w=z(8, 128, dtype=F8)[:, :64]),
    "several matrices without offsets": lambda: linear(w=(2, 8, 64)),
    "offsets of another number": lambda: linear(w=(2, 8, 64), offsets=z(2, dtype=I32)),
    "int64 offsets": lambda: linear(w=(2, 8, 64), offsets=z(3, dtype=torch.int64)),
    "small scales": lambda: linear(w=(129, 64), ws=scales(128, 64)),
    "scales' type": lambda: linear(ws=z(1, 1, 1, 512)),
    "odd features": lambda: linear(w=(7, 64), swiglu=True),
    "swiglu neither": lambda: linear(swiglu=BOTH),
    "fp16 result": lambda: linear(dtype=torch.float16),
    "out's width": lambda: linear(out=z(40, 7)),
    "out's type": lambda: linear(out=z(40, 8, dtype=F32)),
    "out's strides": lambda: linear(out=z(40, 16)[:, :8]),
    "small workspace": lambda: linear(workspace=z(moe.fp8_linear_workspace_bytes(40, 8, 64) - 1, dtype=U8)),
    "tiles: another N": lambda: moe.fp8_tile_scales(z(2, 1, dtype=U8), 128, 128),
    "tiles: another K": lambda: moe.fp8_tile_scales(z(1, 1, dtype=U8), 128, 160),
    "tiles: type": lambda: moe.fp8_tile_scales(z(1, 1), 128, 128),
    "tiles: one dimension": lambda: moe.fp8_tile_scales(z(1, dtype=U8), 128, 128),
    "tiles: no features": lambda: moe.fp8_tile_scales(z(1, 1, dtype=U8), 0, 128),
    "tiles: small out": lambda: moe.fp8_tile_scales(z(2, 1, dtype=U8), 129, 128, out=z(512, dtype=U8)),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()
    moe.ops_check()


def test_sizes_that_the_library_refuses():
    for call in (lambda: linear((40, 48), (8, 48), ws=scales(8, 64)),                   # K not a multiple of 32
                 lambda: linear((2, 32800), (8, 32800)),
                 lambda: moe.fp8_tile_scales(z(1, 1, dtype=U8), 7, 64, True)):
        with pytest.raises(moe.MoeFp4Error):
            call()
    moe.ops_check()
