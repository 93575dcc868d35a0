"""Waits of the operators that run out, without a GPU fault: the host plants a
first stage that is never loaded and a short limit.  The call has to end, the
error has to be reported, every element of a result has to be either right or
left as it was, and the next call has to be right."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests.test_gpu_mxfp4_ops import gpu, rows, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def planted(call, limit_us=2000):
    """call() with the planted wait; the error it has to leave is taken"""
    moe.ops_check()
    moe.set_fault_injection(moe.FAULT_TC_TOKEN_TILE, limit_us)
    try:
        call()
        torch.cuda.synchronize()
    finally:
        moe.set_fault_injection(moe.FAULT_NONE)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    moe.ops_check()


def right_or_untouched(got, want, before):
    bits = {torch.bfloat16: torch.int16, torch.float32: torch.int32}[got.dtype]
    got, want, before = got.view(bits), want.view(bits), before.view(bits)
    left = got != want
    assert left.any(), "the planted wait left nothing undone"
    assert torch.equal(got[left], before[left]), "a wrong value was stored"


# groups of one chunk of 32 rows and of several beside one another, on tiles of 64, of 128 rows and on SM pairs;
# several items for each CTA
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,N,K", [([5, 40, 1, 64, 33, 17, 2, 50, 0, 32, 9, 70] * 2, 4002, 512),
                                        ([100, 120, 0, 130, 7, 1, 128, 129, 90, 20, 31, 95], 4002, 544),
                                        ([257, 0, 1, 513, 255, 31, 130, 96, 17, 600, 3], 2002, 1504)])
def test_ragged_groups(counts, N, K, swiglu):
    rng = np.random.default_rng(N + K)
    off = gpu(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    S = sum(counts)
    x = rows(rng, S, K)
    w, ws = weights(rng, len(counts), N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws), swiglu)
    want = moe.mxfp4_linear(x, w, wt, offsets=off, swiglu=swiglu)
    for _ in range(3):
        before = torch.full_like(want, 7.0)
        out = before.clone()
        planted(lambda: moe.mxfp4_linear(x, w, wt, offsets=off, swiglu=swiglu, out=out))
        right_or_untouched(out, want, before)
        assert torch.equal(moe.mxfp4_linear(x, w, wt, offsets=off, swiglu=swiglu), want)
    moe.ops_check()


# few rows, and rows whose K is split over a cluster: nothing is stored for a tile whose sums are incomplete
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (3, 130, 96), (4, 256, 1024), (16, 1000, 8192), (40, 512, 2048),
                                   (100, 1000, 4096)])
def test_sums_over_a_cluster(M, N, K, swiglu):
    rng = np.random.default_rng(M + N)
    x = rows(rng, M, K)
    w, ws = weights(rng, 1, N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws), swiglu)
    want = moe.mxfp4_linear(x, w, wt, swiglu=swiglu)
    before = torch.full_like(want, 7.0)
    out = before.clone()
    planted(lambda: moe.mxfp4_linear(x, w, wt, swiglu=swiglu, out=out))
    right_or_untouched(out, want, before)
    assert torch.equal(moe.mxfp4_linear(x, w, wt, swiglu=swiglu), want)
    moe.ops_check()


# the block end's form for many rows (with a norm after the row's sum and without, one warp and several a CTA)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T,d,post,following", [(3000, 4096, True, True), (7000, 520, False, True), (700, 7167, True, True),
                                                (20000, 200, True, False), (13000, 64, True, True), (650, 16384, False, False)])
def test_block_end(T, d, post, following, in_place):
    rng = np.random.default_rng(T)
    r, y = rows(rng, T, d), rows(rng, T, d, f32=True)
    kw = dict(post_norm=post, next_norm=following)
    want, want_n = moe.block_residual(r, y, **kw)
    out = r.clone() if in_place else torch.full_like(r, 7.0)
    before = out.clone()
    normed = torch.full_like(r, 7.0) if following else None
    planted(lambda: moe.block_residual(out if in_place else r, y, out=out, normed=normed, **kw))
    right_or_untouched(out, want, before)
    assert torch.equal(out[0], before[0])  # the withheld row itself
    if following:
        right_or_untouched(normed, want_n, torch.full_like(normed, 7.0))
    again = moe.block_residual(r, y, **kw)
    assert torch.equal(again[0], want) and (not following or torch.equal(again[1], want_n))
    moe.ops_check()
