"""Gathered rows whose source rows are used unevenly (padding places that all
name one row, places out of range), with a workspace that lets the call quantise
source rows once and without: the same bits, and those of the rows gathered first.
A wrong or slow list shows on no even sort."""
import time

import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests.test_gpu_mxfp4_ops import gpu, rows, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"
S, T, K, N, E = 36864, 4608, 544, 64, 4


def indices(kind, rng):
    even = rng.permutation(S) % T
    odd = np.arange(S) % 2 == 1
    return {"half one row": np.where(odd, 17, even), "all one row": np.full(S, T - 1), "all out of range": np.full(S, T),
            "half no row": np.where(odd, -1, even), "runs of one row": np.sort(rng.zipf(1.3, S) % T),
            "three rows": rng.integers(0, 3, S), "random": rng.integers(0, T, S)}[kind]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["half one row", "all one row", "all out of range", "half no row", "runs of one row",
                                  "three rows", "random"])
def test_uneven_uses(kind, f32):
    rng = np.random.default_rng(len(kind))
    x = rows(rng, T, K, f32)
    index = indices(kind, rng).astype(np.int32)
    bad = (index < 0) | (index >= T)
    w, ws = weights(rng, E, N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws))
    off = gpu(np.array([0, 9000, 9000, 30001, S], dtype=np.int32))
    source = x[gpu(np.where(bad, 0, index)).long()]
    source[gpu(bad)] = 0
    want = moe.mxfp4_linear(source, w, wt, offsets=off)
    sizes = [moe.mxfp4_linear_workspace_bytes(S, N, K, E), moe.mxfp4_linear_workspace_bytes(S, N, K, E, x_rows=T)]
    assert sizes[1] > sizes[0]
    moe.ops_check()
    for size in sizes:
        buf = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
        got = moe.mxfp4_linear(x, w, wt, offsets=off, row_index=gpu(index), workspace=buf)
        assert torch.equal(got, want)
        if bad.any():
            with pytest.raises(moe.MoeFp4Error):
                moe.ops_check()
        else:
            moe.ops_check()


def test_one_row_used_by_half_of_the_places_costs_no_more_than_a_few_times_an_even_sort():
    """(with all of a row's places left to one warp: two hundred times)"""
    rng = np.random.default_rng(1)
    x = rows(rng, T, K)
    w, ws = weights(rng, E, N, K)
    w, wt = gpu(w), moe.mxfp4_tile_scales(gpu(ws))
    off = gpu(np.array([0, 9000, 9000, 30001, S], dtype=np.int32))
    buf = torch.empty(moe.mxfp4_linear_workspace_bytes(S, N, K, E, x_rows=T), dtype=torch.uint8, device=DEV)
    took = {}
    for kind in ("random", "half one row"):
        index = gpu(indices(kind, rng).astype(np.int32))
        best = float("inf")
        for _ in range(5):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            for _ in range(10):
                moe.mxfp4_linear(x, w, wt, offsets=off, row_index=index, workspace=buf)
            torch.cuda.synchronize()
            best = min(best, time.perf_counter() - t0)
        took[kind] = best
    assert took["half one row"] < 20 * took["random"]
