"""Refusals of the FP8 products, without a GPU: every bad argument is caught on
the host, before anything is enqueued; and no read-only loads in their sources
(test_early_launch_loads.py says why)."""
import ctypes
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import MmDims
from tests.test_early_launch_loads import CSRC, code

FAKE = 0x100000  # never dereferenced
F8, U8, BF = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


def test_scale_layout(lib):
    t = lib.moe_fp4_fp8_tile_scales
    for bad in ((None, 1, 8, 64, 0, FAKE), (FAKE, 0, 8, 64, 0, FAKE), (FAKE, 1025, 8, 64, 0, FAKE), (FAKE, 1, 0, 64, 0, FAKE),
                (FAKE, 1, 2**31 - 1, 64, 0, FAKE), (FAKE, 1, 8, 65, 0, FAKE), (FAKE, 1, 8, 32800, 0, FAKE),
                (FAKE, 1, 7, 64, 1, FAKE), (FAKE, 1, 8, 64, 0, FAKE + 8), (FAKE, 1, 8, 64, 0, None)):
        assert t(*bad, None) == -1, bad


def test_products(lib):
    dims = dict(M=40, N=8, K=64, E=1, swiglu=0, y_type=0)

    def linear(x=FAKE, xt=0, x_rows=40, stride=64, off=None, w=FAKE, ws=FAKE, y=FAKE, work=FAKE, size=1 << 30, **kw):
        d = MmDims(*{**dims, **kw}.values())
        return lib.moe_fp4_fp8_linear(ctypes.byref(d), x, xt, x_rows, stride, off, w, ws, y, work, size, None)

    need = moe.fp8_linear_workspace_bytes(40, 8, 64)
    assert need == 40 * 64 + 512 and moe.fp8_linear_workspace_bytes(40, 8, 65) == 0
    assert lib.moe_fp4_fp8_linear(None, FAKE, 0, 40, 64, None, FAKE, FAKE, FAKE, FAKE, 1 << 30, None) == -1
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=40), dict(K=32800, stride=32800), dict(E=0), dict(E=1025, off=FAKE),
                dict(swiglu=2), dict(swiglu=1, N=7), dict(y_type=2), dict(x=None), dict(x=FAKE + 1), dict(x=FAKE + 2, xt=1),
                dict(xt=3), dict(x_rows=39), dict(stride=32), dict(w=None), dict(w=FAKE + 8), dict(ws=None), dict(ws=FAKE + 8),
                dict(y=None), dict(y=FAKE + 1), dict(y=FAKE + 2, y_type=1), dict(E=2), dict(E=2, off=FAKE + 2), dict(work=None),
                dict(work=FAKE + 16)):
        assert linear(**bad) == -1, bad
    assert linear(size=need - 1) == -3
    assert linear(M=1 << 30, x_rows=1 << 30, K=32, stride=32, N=1 << 20) == -2
    assert linear(M=0, x=None, work=None) == 0
    assert linear(M=16, x_rows=16, E=2, off=FAKE, work=None) == -1  # few rows need none, but not with offsets


def on(device, *shape, dtype=BF):
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def calls(o):
    x, w, ws = on("cuda:0", 4, 64), on("cuda:0", 8, 64, dtype=F8), on("cuda:0", 1, 1, 1, 512, dtype=U8)
    return {
        "w": lambda: moe.fp8_linear(x, on(o, 8, 64, dtype=F8), ws),
        "w_scale": lambda: moe.fp8_linear(x, w, on(o, 1, 1, 1, 512, dtype=U8)),
        "offsets": lambda: moe.fp8_linear(x, w, ws, offsets=on(o, 2, dtype=torch.int32)),
        "out": lambda: moe.fp8_linear(x, w, ws, out=on(o, 4, 8)),
        "workspace": lambda: moe.fp8_linear(x, w, ws, workspace=on(o, 1 << 16, dtype=U8)),
        "tiles' out": lambda: moe.fp8_tile_scales(on("cuda:0", 1, 1, dtype=U8), 8, 64, out=on(o, 512, dtype=U8)),
    }


@pytest.mark.parametrize("other,message", [("cuda:1", "same GPU"), ("cpu", "GPU tensors")])
@pytest.mark.parametrize("name", list(calls("cpu")))
def test_operands_elsewhere_are_refused(name, other, message):
    with pytest.raises(ValueError, match=message):
        calls(other)[name]()


@pytest.mark.parametrize("what", [r"__ldg", r"\.nc", r"__restrict__"])
def test_no_read_only_loads(what):
    import re
    assert not re.search(what + r"\b", code(os.path.join(CSRC, "fp8_quant.cu")))
