"""MXFP4 quantisation and the products of MXFP4 matrices on the GPU against
the fp64 definitions of oracle/mxfp4.py.

Quantisation is compared bit for bit.  Error bound of a product: codes and
scales are exact, and so is every product of two values, so only the fp32
accumulation and the last rounding err.  An instruction adds 64 aligned
products to the accumulator, K / 64 instructions follow one another: with each
of these additions off by at most 2^-23 of S = sum |a w|, an fp32 result is
within (K / 64 + 64) 2^-23 S of the definition; bf16 adds half an ulp, 2^-8
|y| / 2 (2^-8 |y| is used: the fp32 error may move a value to the other side of
a rounding boundary).  With SwiGLU the error of gate and up passes through
h = silu(g) u with |silu'| <= 1.1 and |silu(g)| <= |g|, and the fast exponential and division add
at most 2^-20 (1 + |g|) |h|.
"""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from oracle import mxfp4 as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rows(rng, R, K, f32=False, wide=False):
    x = rng.standard_normal((R, K)).astype(np.float32)
    if wide:
        x *= np.exp2(rng.integers(-30, 30, size=(R, K // 32))).astype(np.float32).repeat(32, axis=1)
    t = torch.from_numpy(x).to(DEV)
    return t if f32 else t.to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


def weights(rng, E, N, K, lo=118, hi=124):
    return (rng.integers(0, 256, (E, N, K // 2), dtype=np.uint8), rng.integers(lo, hi, (E, N, K // 32), dtype=np.uint8))


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_product(y, a, w, swiglu, what):
    """y (GPU) against a [M, K] w [N, K]^T (fp64 values)"""
    K = a.shape[1]
    ref, S = O.matmul(a, w)
    err = (K / 64 + 64) * 2.0 ** -23 * S
    if swiglu:
        g, u = np.split(ref, 2, axis=-1)
        eg, eu = np.split(err, 2, axis=-1)
        h = O.swiglu(ref)
        err = 1.1 * eg * (np.abs(u) + eu) + np.minimum(np.abs(g), 1e30) * eu + 2.0 ** -20 * (1 + np.abs(g)) * np.abs(h)
        ref = h
    if y.dtype == torch.bfloat16:
        err = err + 2.0 ** -8 * (np.abs(ref) + err)
    else:
        err = err + 2.0 ** -23 * np.abs(ref)
    got = f64(y)
    bad = ~(np.abs(got - ref) <= err + 1e-37)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} for {ref[bad][0]}, bound {err[bad][0]}"


# ---- quantisation -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (1, 4096), (33, 96), (130, 1056), (257, 2048)])
def test_quantize_matches_the_definition(R, K, f32):
    x = rows(np.random.default_rng(R * K), R, K, f32, wide=True)
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = O.quantize(f64(x))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    for dtype in (torch.bfloat16, torch.float32):
        np.testing.assert_array_equal(f64(moe.mxfp4_dequantize(codes, scales, dtype)), O.values(want_c, want_s))


@pytest.mark.parametrize("f32", [False, True])
def test_quantize_special_values(f32):
    x = np.zeros((12, 64), dtype=np.float32)
    x[0] = 0.0
    x[1, :32] = -0.0
    x[2, :8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0]       # ties, and saturation: amax 7 -> scale 1
    x[3, :8] = [-0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -7.0]
    x[4, 3] = np.inf
    x[5, 40] = np.nan
    x[6, 0] = 3.3895314e38                                         # the largest bf16
    x[6, 1] = -1e30
    x[7, 0] = 2.0 ** -126                                          # the smallest normal
    x[8, 0] = 2.0 ** -133                                          # a subnormal: the scale stays at 2^-127
    x[8, 1] = 2.0 ** -128
    x[9, 0] = 2.0 ** -124                                          # scale byte 1, then 0 below
    x[9, 32] = 2.0 ** -125
    x[10, :] = -np.inf
    x[11, :32] = np.linspace(-8, 8, 32)
    t = torch.from_numpy(x).to(DEV)
    t = t if f32 else t.to(torch.bfloat16)
    codes, scales = moe.mxfp4_quantize(t)
    want_c, want_s = O.quantize(f64(t))
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    back = f64(moe.mxfp4_dequantize(codes, scales))
    assert np.isnan(back[4, :32]).all() and np.isnan(back[5, 32:]).all() and np.isnan(back[10]).all()
    assert np.isfinite(back[4, 32:]).all()


def test_every_scale_reads_back():
    scales = np.arange(256, dtype=np.uint8).reshape(8, 32)
    codes = np.random.default_rng(0).integers(0, 256, (8, 512), dtype=np.uint8)
    want = O.values(codes, scales)
    for dtype, top in ((torch.float32, 3.4028234663852886e38), (torch.bfloat16, 3.3895313892515355e38)):
        got = f64(moe.mxfp4_dequantize(gpu(codes), gpu(scales), dtype))
        expect = np.where(np.abs(want) > top, np.copysign(np.inf, want), want)
        np.testing.assert_array_equal(got, expect)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K,pad,shift", [(96, 8, 0), (1056, 3, 0), (64, 1, 1), (128, 0, 3)])
def test_quantize_strided_and_unaligned_rows(K, pad, shift, f32):
    R = 37
    buf = rows(np.random.default_rng(K + pad), R, K + 32 * ((pad + shift + 31) // 32), f32)
    buf = buf[:, :K + pad + shift].contiguous()
    x = buf[:, shift:shift + K]
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = O.quantize(f64(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (4, 0), (8, 8), (1, 1)])
def test_quantize_many_rows_at_every_alignment(pad, shift, f32):
    R, K = 1300, 544
    x = rows(np.random.default_rng(pad), R, K + 32, f32)[:, :K + pad + shift].contiguous()[:, shift:shift + K]
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = O.quantize(f64(x))
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    tiled_c, tiled_s = moe.mxfp4_quantize(x, tiled=True)
    assert torch.equal(tiled_c, codes)
    t = tiled_s.cpu().numpy().reshape(-1, (K + 127) // 128, 32, 4, 4)      # [tile, K / 128, row % 32, row / 32, block]
    back = t.transpose(0, 3, 2, 1, 4).reshape(-1, (K + 127) // 128 * 4)[:R, :K // 32]
    np.testing.assert_array_equal(back, want_s)


@pytest.mark.parametrize("K", [32, 160, 512])
def test_quantize_gathers_and_tiles_by_group(K):
    rng = np.random.default_rng(K)
    T, k = 70, 3
    counts = [0, 1, 128, 0, 5, 70, 6, 0]
    S = sum(counts)
    assert S == T * k
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    slot = rng.permutation(S).astype(np.int32)
    x = rows(rng, T, K)
    codes, tiled = moe.mxfp4_quantize(x, row_index=gpu(slot), index_div=k, offsets=gpu(off), tiled=True)
    want_c, want_s = O.quantize(f64(x)[slot // k])
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    tiled = tiled.cpu().numpy()
    assert tiled.shape[0] == S // 128 + len(counts)
    for e, c in enumerate(counts):
        for i in range(c):
            for b in range(-(-K // 128) * 4):
                want = want_s[off[e] + i, b] if b < K // 32 else 0
                assert O.tiled_scale(tiled[off[e] // 128 + e:], i, b) == want, (e, i, b)
    moe.ops_check()


def test_a_row_index_out_of_range_gives_a_zero_row_and_an_error():
    x = rows(np.random.default_rng(1), 4, 64)
    codes, scales = moe.mxfp4_quantize(x, row_index=gpu(np.array([0, 4, -1, 3], dtype=np.int32)))
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    moe.ops_check()  # cleared
    want_c, want_s = O.quantize(f64(x)[[0, 0, 0, 3]])
    got = codes.cpu().numpy()
    np.testing.assert_array_equal(got[[0, 3]], want_c[[0, 3]])
    assert not got[[1, 2]].any() and not scales.cpu().numpy()[[1, 2]].any()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("E,N,K", [(1, 2, 32), (3, 130, 160), (2, 256, 512)])
def test_tile_scales(E, N, K, swiglu):
    s = np.random.default_rng(N).integers(0, 255, (E, N, K // 32), dtype=np.uint8)
    np.testing.assert_array_equal(moe.mxfp4_tile_scales(gpu(s), swiglu).cpu().numpy(), O.tile_scales(s, swiglu))


# ---- dense products -----------------------------------------------------------------------------------------

def dense(M, N, K, swiglu, dtype, seed, f32=False):
    rng = np.random.default_rng(seed)
    x = rows(rng, M, K, f32)
    w, ws = weights(rng, 1, N, K)
    y = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws), swiglu), swiglu=swiglu, dtype=dtype)
    a = O.values(*O.quantize(f64(x)))
    check_product(y, a, O.values(w[0], ws[0]), swiglu, f"M={M} N={N} K={K}")
    moe.ops_check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [32, 64, 96, 128, 256, 288, 544, 1056])
def test_linear_k(K, dtype):
    dense(19, 136, K, False, dtype, K)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 127, 128, 129, 191, 256, 257, 385, 700])
def test_linear_rows(M, dtype):
    dense(M, 200, 320, False, dtype, M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("N", [1, 2, 7, 31, 127, 128, 129, 255, 386, 1001])
def test_linear_features(N, M, dtype):
    dense(M, N, 192, False, dtype, N)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 2, 32), (1, 4096, 4096), (5, 130, 96), (64, 254, 512), (130, 256, 1024),
                                   (300, 514, 288)])
def test_linear_swiglu(M, N, K, dtype):
    dense(M, N, K, True, dtype, M + N)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (8, 4096, 2048), (100, 1000, 8192), (3, 16, 32768)])
def test_linear_long_k(M, N, K):
    dense(M, N, K, False, torch.float32, 5, f32=True)


# odd sizes for which tiles of 128 token rows are chosen, and for which SM pairs are
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K,swiglu", [(290, 4095, 1056, False), (640, 2050, 96, True), (777, 4095, 2016, False),
                                          (1999, 4096, 1056, False), (900, 2562, 2080, True), (2700, 1004, 2080, True)])
def test_linear_larger_tiles(M, N, K, swiglu, dtype):
    dense(M, N, K, swiglu, dtype, M)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N,K,swiglu", [([100, 120, 0, 130, 97, 1, 128, 129, 90], 2001, 544, False),
                                               ([100, 120, 0, 130, 97, 1, 128, 129, 90], 2002, 544, True),
                                               ([257, 0, 1, 513, 255, 31, 130, 96, 17], 1501, 1504, False),
                                               ([257, 0, 1, 513, 255, 31, 130, 96, 17], 1498, 2080, True),
                                               ([0, 256, 0, 512, 224, 33, 192, 64, 19], 4002, 544, False)])
def test_grouped_larger_tiles(counts, N, K, swiglu, dtype):
    grouped(counts, N, K, swiglu, dtype, N, before=3, after=2)


def test_linear_equals_quantize_then_matmul():
    rng = np.random.default_rng(3)
    for M in (1, 9, 100, 600):
        x = rows(rng, M, 544)
        w, ws = weights(rng, 1, 272, 544)
        wt = moe.mxfp4_tile_scales(gpu(ws))
        y = moe.mxfp4_linear(x, gpu(w), wt)
        a, s = moe.mxfp4_quantize(x, tiled=True)
        assert torch.equal(y, moe.mxfp4_matmul(a, s, gpu(w), wt))
        assert torch.equal(y, moe.mxfp4_linear(x, gpu(w), wt))  # the same bits again


def test_nan_blocks_stay_in_their_row_and_column():
    rng = np.random.default_rng(4)
    x = rows(rng, 40, 256)
    x[7, 100] = float("nan")
    w, ws = weights(rng, 1, 200, 256)
    ws[0, 33, 2] = 255
    y = f64(moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws))))
    nan = np.isnan(y)
    want = np.zeros_like(nan)
    want[7] = True
    want[:, 33] = True
    np.testing.assert_array_equal(nan, want)


# ---- grouped products ---------------------------------------------------------------------------------------

def grouped(counts, N, K, swiglu, dtype, seed, before=0, after=0):
    rng = np.random.default_rng(seed)
    E = len(counts)
    off = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
    S = int(off[-1]) + after
    x = rows(rng, max(S, 1), K)[:S]
    w, ws = weights(rng, E, N, K)
    n = N // 2 if swiglu else N
    out = torch.full((S, n), 7.0, dtype=dtype, device=DEV)
    y = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws), swiglu), offsets=gpu(off), swiglu=swiglu,
                         dtype=dtype, out=out)
    a = O.values(*O.quantize(f64(x))) if S else np.zeros((0, K))
    for e in range(E):
        if counts[e]:
            check_product(y[off[e]:off[e + 1]], a[off[e]:off[e + 1]], O.values(w[e], ws[e]), swiglu, f"group {e}")
    # rows in no group are not written
    assert (y[:before] == 7).all() and (y[int(off[-1]):] == 7).all()
    moe.ops_check()


COUNTS = [[5], [0, 3], [1, 0, 0, 1], [64, 65, 63, 0, 128, 129], [300, 0, 1, 17], [1] * 40, [0, 0, 0], [16] * 9,
          [200, 7, 0, 513], [2, 90, 3, 70, 66, 130, 1]]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped(counts, swiglu):
    grouped(counts, 140, 288, swiglu, torch.bfloat16, len(counts))


@pytest.mark.parametrize("N,K", [(1, 32), (129, 64), (256, 1056), (1001, 128)])
@pytest.mark.parametrize("counts", [[3, 0, 130], [70, 1, 2]])
def test_grouped_fp32(counts, N, K):
    grouped(counts, N, K, False, torch.float32, N)


def test_grouped_rows_in_no_group():
    grouped([3, 0, 70], 64, 128, False, torch.bfloat16, 1, before=5, after=200)
    grouped([0, 0], 64, 128, False, torch.float32, 1, before=0, after=9)


def test_grouped_many_experts():
    rng = np.random.default_rng(11)
    counts = rng.integers(0, 3, 1024).tolist()
    grouped(counts, 16, 32, False, torch.bfloat16, 2)


def test_grouped_with_the_layers_routing():
    """the layer's own sort feeds the grouped product: gather by sorted_slot, groups by expert_offsets"""
    rng = np.random.default_rng(6)
    T, E, k, d, I = 50, 16, 4, 256, 128
    logits = gpu(rng.standard_normal((T, E)).astype(np.float32))
    ids, _, off, slot = moe.route(logits, k)
    x = rows(rng, T, d)
    w, ws = weights(rng, E, 2 * I, d)
    h = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws), True), offsets=off, row_index=slot, index_div=k,
                         swiglu=True)
    a = O.values(*O.quantize(f64(x)))[slot.cpu().numpy() // k]
    o = off.cpu().numpy()
    for e in range(E):
        if o[e + 1] > o[e]:
            check_product(h[o[e]:o[e + 1]], a[o[e]:o[e + 1]], O.values(w[e], ws[e]), True, f"expert {e}")


def test_another_stream_and_a_captured_graph():
    rng = np.random.default_rng(8)
    x = rows(rng, 24, 512)
    w, ws = weights(rng, 1, 256, 512)
    wt = moe.mxfp4_tile_scales(gpu(ws))
    w = gpu(w)
    want = moe.mxfp4_linear(x, w, wt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    ws_buf = torch.empty(moe.mxfp4_linear_workspace_bytes(24, 256, 512), dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(s):
        moe.mxfp4_linear(x, w, wt, out=out, workspace=ws_buf)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.mxfp4_linear(x, w, wt, out=out, workspace=ws_buf)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_rows():
    w, ws = weights(np.random.default_rng(0), 2, 64, 64)
    wt = moe.mxfp4_tile_scales(gpu(ws))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert moe.mxfp4_linear(x, gpu(w), wt, offsets=off).shape == (0, 64)
    c, s = moe.mxfp4_quantize(x)
    assert c.shape == (0, 32) and s.shape == (0, 2)
    assert moe.mxfp4_dequantize(c, s).shape == (0, 64)


def test_rows_used_several_times_are_quantised_once_with_the_same_bits():
    """a workspace that lets the call quantise each source row once and gather its codes"""
    rng = np.random.default_rng(21)
    T, k, E, N, K = 2100, 8, 16, 96, 1056
    S = T * k
    counts = rng.multinomial(S, np.ones(E) / E)
    counts[3] += counts[4]
    counts[4] = 0
    off = gpu(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    slot = rng.permutation(S).astype(np.int32)
    slot[5] = S + 3                                     # out of range: a zero row, and an error
    slot = gpu(slot)
    x = rows(rng, T, K)
    w, ws = weights(rng, E, N, K)
    wt, w = moe.mxfp4_tile_scales(gpu(ws)), gpu(w)
    small = moe.mxfp4_linear_workspace_bytes(S, N, K, E)
    large = moe.mxfp4_linear_workspace_bytes(S, N, K, E, x_rows=T)
    assert large > small
    got = []
    for size in (small, large):
        buf = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        got.append(moe.mxfp4_linear(x, w, wt, offsets=off, row_index=slot, index_div=k, workspace=buf))
        with pytest.raises(moe.MoeFp4Error):
            moe.ops_check()
    assert torch.equal(got[0], got[1])
    assert not got[0][5].any()
    a = O.values(*O.quantize(f64(x)))[np.minimum(slot.cpu().numpy(), S - 1) // k]
    a[5] = 0
    o = off.cpu().numpy()
    for e in range(E):
        if counts[e]:
            check_product(got[1][o[e]:o[e + 1]], a[o[e]:o[e + 1]], O.values(w[e].cpu().numpy(), ws[e]), False, f"expert {e}")


def test_a_given_stream_owns_what_a_call_allocates():
    """results and workspaces of a call with stream= are not handed to the current stream's work while it runs"""
    rng = np.random.default_rng(33)
    M, N, K = 300, 512, 2048
    x = rows(rng, M, K)
    w, ws = weights(rng, 1, N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws))
    want = moe.mxfp4_linear(x, w, wt)
    size = moe.mxfp4_linear_workspace_bytes(M, N, K)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(50):
        got = [moe.mxfp4_linear(x, w, wt, stream=s) for _ in range(4)]
        junk = [torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]  # on the current stream
        s.synchronize()
        for y in got:
            assert torch.equal(y, want)
        del got, junk


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("M", [1, 5, 16, 17, 90])
@pytest.mark.parametrize("K,pad,shift", [(544, 24, 8), (1056, 3, 1)])
def test_linear_strided_and_unaligned_rows(M, K, pad, shift, f32):
    rng = np.random.default_rng(M + K)
    buf = rows(rng, M, K + 32, f32)[:, :K + pad].contiguous()
    x = buf[:, shift:shift + K - 32]
    K -= 32
    w, ws = weights(rng, 1, 130, K)
    y = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws)), dtype=torch.float32)
    check_product(y, O.values(*O.quantize(f64(x))), O.values(w[0], ws[0]), False, "strided")


@pytest.mark.parametrize("M", [3, 16, 40])
def test_linear_gathers_without_groups(M):
    rng = np.random.default_rng(M)
    x = rows(rng, 9, 288)
    index = rng.integers(0, 18, M).astype(np.int32)
    index[1] = 18                                       # out of range: a zero row, and an error
    w, ws = weights(rng, 1, 66, 288)
    y = moe.mxfp4_linear(x, gpu(w), moe.mxfp4_tile_scales(gpu(ws)), row_index=gpu(index), index_div=2, dtype=torch.float32)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    a = O.values(*O.quantize(f64(x)))[np.minimum(index, 17) // 2]
    a[1] = 0
    check_product(y, a, O.values(w[0], ws[0]), False, "gathered")
    assert not y[1].any()


@pytest.mark.parametrize("M", [4, 60, 120, 2000])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(M):
    """host-planted: the first CTA never loads its first stage (no fault on the GPU); every waiting role gives up"""
    rng = np.random.default_rng(M)
    N, K = (256, 1024) if M < 2000 else (4096, 1024)
    x = rows(rng, M, K)
    w, ws = weights(rng, 1, N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws))
    want = moe.mxfp4_linear(x, w, wt)
    moe.ops_check()
    moe.set_fault_injection(moe.FAULT_TC_TOKEN_TILE, 2000)
    try:
        moe.mxfp4_linear(x, w, wt)
        torch.cuda.synchronize()
    finally:
        moe.set_fault_injection(moe.FAULT_NONE)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    assert torch.equal(moe.mxfp4_linear(x, w, wt), want)
    moe.ops_check()


def test_offsets_beyond_32_bits():
    """more than 2^31 elements of rows, codes and results: the last rows are right"""
    rng = np.random.default_rng(5)
    last = 5
    x = torch.zeros(70016, 32768, dtype=torch.bfloat16, device=DEV)
    x[-last:] = rows(rng, last, 32768)
    codes, scales = moe.mxfp4_quantize(x)
    want_c, want_s = O.quantize(f64(x[-last:]))
    np.testing.assert_array_equal(codes[-last:].cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales[-last:].cpu().numpy(), want_s)
    back = moe.mxfp4_dequantize(codes, scales)
    np.testing.assert_array_equal(f64(back[-last:]), O.values(want_c, want_s))
    del back, codes, scales
    w, ws = weights(rng, 1, 32768, 64)
    y = moe.mxfp4_linear(x[:, -64:], gpu(w), moe.mxfp4_tile_scales(gpu(ws)))
    check_product(y[-last:], O.values(*O.quantize(f64(x[-last:, -64:]))), O.values(w[0], ws[0]), False, "last rows")
    assert not y[:64].any()
    moe.ops_check()
