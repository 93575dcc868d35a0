"""Gates of the operators far from 0, in fp32: SwiGLU of the products and the
sigmoid of the block end, where everything else in the result is exact.

Error bound: exp within 2 ulp (2^-22 relative), 1 + exp, the quotient and the
products by one rounding each (2^-24), at most four of them: 2^-22 + 4 2^-24 =
2^-21 relative.  exp's own argument is exact.  Beyond |g| = 87 a factor leaves
fp32's normal range: not compared.  bf16 results add half an ulp, 2^-9, with
2^-8 used as for the products."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from oracle import mxfp4 as O
from tests.test_gpu_mxfp4_ops import gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def within(got, want, dtype, what):
    bound = (2.0 ** -21 + (2.0 ** -8 if dtype == BF else 0)) * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    bad = err > bound
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, by up to {(err / np.maximum(bound, 1e-300)).max():.1f} bounds"


# every form of the product: few rows, K split over a cluster, one SM a tile, SM pairs
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("M", [1, 20, 333, 4096])
def test_swiglu(M, dtype):
    """rows of ones against a feature's 32 multiples of 2^-1: gate and up are exact"""
    I = 2048
    rng = np.random.default_rng(M)
    w = rng.integers(0, 256, (2 * I, 16), dtype=np.uint8)
    s = np.full((2 * I, 1), 127, np.uint8)
    x = torch.ones(M, 32, dtype=BF, device=DEV)
    y = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(s), True), swiglu=True, dtype=dtype)
    sums = O.values(w, s).sum(axis=1)
    g = sums[:I]
    assert np.abs(sums).max() < 87 and g.min() < -40 and g.max() > 40
    assert torch.equal(y, y[:1].expand_as(y))
    within(y[0], O.swiglu(sums), dtype, f"M={M}")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", ["token", "channel", "element"])
@pytest.mark.parametrize("T,d", [(3, 4096), (7, 1001), (3000, 4096), (620, 7167)])
def test_sigmoid(T, d, shape, dtype):
    """a residual of zeros and a branch of ones: out is the sigmoid itself"""
    n = {"token": (T, 1), "channel": (1, d), "element": (T, d)}[shape]
    g = torch.linspace(-80, 80, n[0] * n[1], device=DEV).view(n)
    z, one = torch.zeros(T, d, dtype=dtype, device=DEV), torch.ones(T, d, device=DEV)
    out, _ = moe.block_residual(z, one, post_norm=False, gate=g, gate_sigmoid=True)
    want = 1.0 / (1.0 + np.exp(-g.double().cpu().numpy()))
    within(out, np.broadcast_to(want, (T, d)), dtype, shape)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shape", ["token", "channel", "element"])
@pytest.mark.parametrize("T,d", [(5, 64), (5, 333), (3000, 4096), (700, 7167)])
def test_infinite_and_nan_gates(T, d, shape, dtype):
    """sigmoid(inf) = 1, sigmoid(-inf) = 0; a NaN stays in its token, channel or element"""
    n = {"token": (T, 1), "channel": (1, d), "element": (T, d)}[shape]
    g = torch.zeros(n[0] * n[1], device=DEV)
    g[0], g[1], g[2], g[3] = float("inf"), -float("inf"), float("nan"), 1e30
    g = g.view(n)
    z, one = torch.zeros(T, d, dtype=dtype, device=DEV), torch.ones(T, d, device=DEV)
    out, normed = moe.block_residual(z, one, post_norm=False, gate=g, gate_sigmoid=True)
    want = torch.sigmoid(g.double()).expand(T, d)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out.double(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert torch.equal(torch.isnan(normed).any(dim=1), torch.isnan(want).any(dim=1))  # the next norm's row alone
