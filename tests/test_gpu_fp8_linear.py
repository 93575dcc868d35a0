"""Products with E4M3 weights (a scale for 128 x 128) from quantised rows,
against the fp64 definition of oracle/fp8.py.

Error bound: codes and scales are exact, and so is every product of two values
(8 significant bits), so only the fp32 accumulation and the last rounding err.
An instruction adds 32 aligned products to the accumulator, K / 32 instructions
follow one another: with each of these additions off by at most 2^-23 of S = sum
|a w|, an fp32 result is within (K / 32 + 32) 2^-23 S of the definition, and the
sum over a cluster of up to 8 CTAs adds 8 roundings; bf16 adds half a step, 2^-8
of the value with its fp32 error.  SwiGLU: as for the MXFP4 products.
"""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from oracle import fp8 as O
from oracle import mxfp4
from tests.test_gpu_mxfp4_ops import f64, gpu, rows
from tests.test_gpu_ops_waits import planted, right_or_untouched

pytestmark = pytest.mark.gpu
DEV = "cuda"


def weights(rng, E, N, K):
    codes = rng.integers(0, 256, (E, N, K), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0                            # no NaN
    return codes, rng.integers(110, 120, (E, -(-N // 128), -(-K // 128)), dtype=np.uint8)


def on_gpu(w, s, N, K, swiglu):
    return gpu(w).view(torch.float8_e4m3fn), moe.fp8_tile_scales(gpu(s), N, K, swiglu)


def check_product(y, a, w, swiglu, what):
    K = a.shape[1]
    ref, S = mxfp4.matmul(a, w)
    err = (K / 32 + 32 + 8) * 2.0 ** -23 * S
    if swiglu:
        g, u = np.split(ref, 2, axis=-1)
        eg, eu = np.split(err, 2, axis=-1)
        h = mxfp4.swiglu(ref)
        err = 1.1 * eg * (np.abs(u) + eu) + np.minimum(np.abs(g), 1e30) * eu + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(h)
        ref = h
    err = err + (2.0 ** -8 * (np.abs(ref) + err) if y.dtype == torch.bfloat16 else 2.0 ** -23 * np.abs(ref))
    got = f64(y)
    bad = ~(np.abs(got - ref) <= err + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, bound {err[bad][0]}"


def wide(rng, R, K, f32):
    """rows whose blocks of 128 differ in scale"""
    x = rng.standard_normal((R, K)) * np.repeat(np.exp2(rng.integers(-20, 20, (R, -(-K // 128)))), 128, axis=1)[:, :K]
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    return t if f32 else t.to(torch.bfloat16)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("E,N,K", [(1, 2, 32), (3, 130, 160), (2, 300, 512), (1, 512, 128)])
def test_tile_scales(E, N, K, swiglu):
    s = np.random.default_rng(N).integers(0, 255, (E, -(-N // 128), -(-K // 128)), dtype=np.uint8)
    np.testing.assert_array_equal(moe.fp8_tile_scales(gpu(s), N, K, swiglu).cpu().numpy(), O.tile_scales(s, N, swiglu))


# few rows (one kernel), tiles of 64 and 128 rows, K split over a cluster, SM pairs
@pytest.mark.parametrize("f32,dtype", [(False, torch.bfloat16), (True, torch.float32)])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 2, 32), (1, 4096, 512), (2, 130, 160), (3, 1000, 1056), (7, 258, 96),
                                   (8, 64, 4096), (16, 514, 1536), (17, 130, 160), (33, 300, 1056), (64, 256, 4096),
                                   (100, 2050, 544), (300, 1030, 256), (700, 1536, 384)])
def test_dense(M, N, K, swiglu, f32, dtype):
    rng = np.random.default_rng(M * N + K)
    x = wide(rng, M, K, f32)
    w, s = weights(rng, 1, N, K)
    y = moe.fp8_linear(x, *on_gpu(w, s, N, K, swiglu), swiglu=swiglu, dtype=dtype)
    check_product(y, O.row_values(*O.quantize(f64(x))), O.weight_values(w[0], s[0]), swiglu, f"{M} {N} {K}")
    moe.ops_check()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(2049, 2560, 256), (1300, 4096, 160)])
def test_many_rows_on_sm_pairs(M, N, K, swiglu):
    rng = np.random.default_rng(M)
    x = wide(rng, M, K, False)
    w, s = weights(rng, 1, N, K)
    y = moe.fp8_linear(x, *on_gpu(w, s, N, K, swiglu), swiglu=swiglu)
    check_product(y, O.row_values(*O.quantize(f64(x))), O.weight_values(w[0], s[0]), swiglu, f"{M} {N} {K}")
    moe.ops_check()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K", [([0, 1, 0], 64, 32), ([1, 0, 5, 33, 128, 0], 130, 160), ([300, 1, 129, 17], 1000, 96),
                                        ([5] * 40, 256, 128), ([0, 0], 64, 128), ([600, 513, 0, 257], 514, 288)])
def test_groups(counts, N, K, swiglu):
    rng = np.random.default_rng(len(counts) + N)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + 3                                       # three rows in no group
    x = wide(rng, M, K, False)
    w, s = weights(rng, len(counts), N, K)
    out = torch.full((M, N // 2 if swiglu else N), 7.0, dtype=torch.float32, device=DEV)
    y = moe.fp8_linear(x, *on_gpu(w, s, N, K, swiglu), offsets=gpu(off), swiglu=swiglu, dtype=torch.float32, out=out)
    assert y.data_ptr() == out.data_ptr()
    a = O.row_values(*O.quantize(f64(x)))
    for e, n in enumerate(counts):
        if n:
            check_product(y[off[e]:off[e + 1]], a[off[e]:off[e + 1]], O.weight_values(w[e], s[e]), swiglu, f"group {e}")
    assert (y[off[-1]:] == 7.0).all()
    moe.ops_check()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M", [8, 60])
def test_special_values_and_scale_boundaries(M, f32):
    """an identity of weights returns the quantised rows themselves"""
    K = 256
    x = np.zeros((M, K), dtype=np.float32)
    x[0, :6] = [448, -448, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10]
    x[1, :2] = [450, -449]                                     # above the largest code: the next scale
    x[1, 128] = 3.5
    x[1, 129] = -3.515625
    x[2, 5] = np.inf
    x[2, 200] = 1.0
    x[3, 130] = np.nan
    x[3, 1] = -2.0
    x[4, 0] = 2.0 ** -133                                      # subnormals, and the least scale
    x[4, 1] = 2.0 ** -126
    x[4, 128] = 448 * 2.0 ** -127
    x[5, 0] = 3.3895314e38                                     # the largest bf16
    x[5, 1] = 1e30
    x[6, :] = -0.0
    x[7, :] = np.linspace(-500, 500, K)
    t = torch.from_numpy(x).to(DEV)
    t = t if f32 else t.to(torch.bfloat16)
    w = np.zeros((1, K, K), dtype=np.uint8)
    w[0, np.arange(K), np.arange(K)] = 0x38                    # 1
    s = np.full((1, 2, 2), 127, dtype=np.uint8)
    y = f64(moe.fp8_linear(t, *on_gpu(w, s, K, K, False), dtype=torch.float32))
    # In fp32, as the result is: the largest bf16, (2 - 2^-7) 2^127, becomes 256 x 2^120 = 2^128, and fp32's largest value is
    # (2 - 2^-23) 2^127: whatever reaches 2^128 - 2^103 rounds to an infinity.  (The tensor core may flush results below
    # the smallest normal.)
    with np.errstate(over="ignore"):
        want = O.row_values(*O.quantize(f64(t))).astype(np.float32)
    nan = np.isnan(want).reshape(M, 2, 128).any(axis=2)
    assert nan[2, 0] and nan[3, 1] and not nan[3, 0]
    for r in range(M):
        if nan[r].any():                                       # NaN times the identity's zeros too
            assert np.isnan(y[r]).all()
        else:
            np.testing.assert_allclose(y[r], want[r], rtol=0, atol=2.0 ** -126)
    moe.ops_check()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M", [5, 70, 1300])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (4, 0), (1, 1)])
def test_strided_and_unaligned_rows(M, pad, shift, f32):
    rng = np.random.default_rng(M + pad)
    N, K = 130, 416
    x = rows(rng, M, 448, f32)[:, :K + pad + shift].contiguous()[:, shift:shift + K]
    w, s = weights(rng, 1, N, K)
    wg = on_gpu(w, s, N, K, False)
    assert torch.equal(moe.fp8_linear(x, *wg), moe.fp8_linear(x.contiguous(), *wg))
    check_product(moe.fp8_linear(x, *wg), O.row_values(*O.quantize(f64(x))), O.weight_values(w[0], s[0]), False, "strided")


@pytest.mark.parametrize("M", [4, 200])
def test_no_rows_other_streams_workspaces_and_graphs(M):
    rng = np.random.default_rng(M)
    N, K = 256, 384
    w, s = weights(rng, 1, N, K)
    wg = on_gpu(w, s, N, K, False)
    assert moe.fp8_linear(rows(rng, 0, K), *wg).shape == (0, N)
    x = rows(rng, M, K)
    want = moe.fp8_linear(x, *wg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.fp8_linear(x, *wg, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.empty(moe.fp8_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.fp8_linear(x, *wg, out=out, workspace=ws)
    x2 = rows(rng, M, K)
    x.copy_(x2)
    graph.replay()
    assert torch.equal(out, moe.fp8_linear(x2, *wg))
    moe.ops_check()


@pytest.mark.parametrize("counts,N,K", [(None, 1000, 4096), (None, 4096, 1024), ([5, 40, 1, 64, 33, 17, 2, 50, 0, 32, 9, 70] * 2, 4002, 512),
                                        ([257, 0, 1, 513, 255, 31, 130, 96, 17, 600, 3], 2002, 1504)])
def test_waits_that_run_out_store_nothing_wrong(counts, N, K):
    rng = np.random.default_rng(N)
    M = 12 if counts is None else sum(counts)
    off = None if counts is None else gpu(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    x = rows(rng, M, K)
    w, s = weights(rng, 1 if counts is None else len(counts), N, K)
    wg = on_gpu(w, s, N, K, False)
    want = moe.fp8_linear(x, *wg, offsets=off)
    before = torch.full_like(want, 7.0)
    out = before.clone()
    planted(lambda: moe.fp8_linear(x, *wg, offsets=off, out=out))
    right_or_untouched(out, want, before)
    assert torch.equal(moe.fp8_linear(x, *wg, offsets=off), want)
