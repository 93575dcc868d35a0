"""Sizes whose tiles cannot be counted in 32 bits are refused on the host
(no GPU: nothing is enqueued)."""
import ctypes
import os

import pytest

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import MmDims

FAKE = 0x100000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


@pytest.mark.parametrize("N", [2**31 - 1, 2**31 - 2, 2**31 - 127, 2**31 - 128, 2**31 - 255])
@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("swiglu", [0, 1])
def test_features(lib, N, M, swiglu):
    if swiglu:
        N -= N % 2
    d = MmDims(M, N, 64, 1, swiglu, 0)
    if N > 2**31 - 256:
        assert lib.moe_fp4_mxfp4_matmul(ctypes.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == -2
        assert lib.moe_fp4_mxfp4_linear_workspace_bytes(ctypes.byref(d)) == 0
        assert lib.moe_fp4_mxfp4_linear(ctypes.byref(d), FAKE, 0, M, 64, None, 1, None, FAKE, FAKE, FAKE, FAKE, 1 << 40,
                                        None) == -2
        assert lib.moe_fp4_mxfp4_tile_scales(FAKE, 1, N, 64, swiglu, FAKE, None) == -1
    assert moe.mxfp4_linear_workspace_bytes(M, 2**31 - 256, 64) > 0


def test_rows_times_features(lib):
    for M, N in ((2**20, 2**24), (2**16, 2**28), (2**29, 2**22)):
        d = MmDims(M, N, 32, 1, 0, 0)
        assert lib.moe_fp4_mxfp4_matmul(ctypes.byref(d), FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == -2
