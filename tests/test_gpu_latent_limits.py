"""Latent attention at the ends of what its calls allow: as many heads as there may be,
pages of any multiple of 16, batches of nothing, several captured calls that share one
workspace in one stream's order."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check
from tests.test_gpu_latent_attention import SCALE, check_all, make
from tests.test_gpu_latent_decode import check_all as check_decoded
from tests.test_gpu_latent_decode import make as make_cache
from tests.test_gpu_latent_decode import tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("H", [1000, 1024])
@pytest.mark.parametrize("lens,page", [([1], 64), ([700, 0, 65], 16), ([5000, 3], 64)])
def test_absorbed_with_many_heads(lens, page, H):
    q, cache, table, lengths = make_cache(lens, H, page, seed=H)
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    for b, n in enumerate(lens):
        c = tokens(cache, table, b, n)
        for h in (0, 63, 64, 511, H - 1) if n else ():
            check(out[b, h:h + 1], *attend(q[b, h:h + 1], c, c[:, :512], SCALE), f"sequence {b}, head {h}")
        assert n or not out[b].any()
    moe.ops_check()


@pytest.mark.parametrize("H", [1000, 1024])
@pytest.mark.parametrize("q_lens,k_lens", [([1], [1]), ([7, 0, 300], [20, 5, 300]), ([30, 9], [1500, 9])])
def test_expanded_with_many_heads(q_lens, k_lens, H):
    t = make(q_lens, k_lens, H, seed=H)
    check_all(moe.latent_attention(*t, SCALE), *t, True, heads=(0, 1, 500, H - 1))
    moe.ops_check()


@pytest.mark.parametrize("page", [80, 112, 256, 1024, 4096, 4112])
def test_pages_of_any_multiple_of_16(page):
    lens = [5000, 1, 4096, 0, 4097, 63]
    q, cache, table, lengths = make_cache(lens, 20, page, seed=page)
    check_decoded(moe.latent_decode(q, cache, table, lengths, SCALE), q, cache, table, lens)
    moe.ops_check()


@pytest.mark.parametrize("B", [1, 40, 700])
def test_batches_of_nothing(B):
    q, cache, table, lengths = make_cache([0] * B, 16, 64)
    assert not moe.latent_decode(q, cache, table, lengths, SCALE).any()
    t = make([0] * B, [5] * B, 4)
    assert moe.latent_attention(*t, SCALE).shape == (0, 4, 128)
    t = make([3] * B, [0] * B, 4)
    for causal in (False, True):
        assert not moe.latent_attention(*t, SCALE, causal=causal).any()
    moe.ops_check()


def test_captured_calls_that_share_a_workspace():
    """one after the other, in a graph and in two that are replayed in turn"""
    a, b = make_cache([3000, 70], 24, 64, seed=1), make_cache([900] * 9, 24, 64, seed=2)
    wa, wb = moe.latent_decode(*a, SCALE), moe.latent_decode(*b, SCALE)
    x, y = make([300, 40], [5000, 40], 3, seed=3), make([64], [9000], 2, seed=4)
    wx, wy = moe.latent_attention(*x, SCALE), moe.latent_attention(*y, SCALE)
    ws = torch.full((max(moe.latent_decode_workspace_bytes(24), moe.latent_attention_workspace_bytes()),), 255, dtype=torch.uint8, device=DEV)
    ga, gb, gx, gy = (torch.empty_like(w) for w in (wa, wb, wx, wy))
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        moe.latent_decode(*a, SCALE, out=ga, workspace=ws)
        moe.latent_attention(*x, SCALE, out=gx, workspace=ws)
        moe.latent_decode(*b, SCALE, out=gb, workspace=ws)
    with torch.cuda.graph(two):
        moe.latent_attention(*y, SCALE, out=gy, workspace=ws)
        moe.latent_decode(*a, SCALE, out=ga, workspace=ws)
    for _ in range(10):
        for g in (ga, gb, gx, gy):
            g.fill_(7)
        one.replay()
        assert torch.equal(ga, wa) and torch.equal(gx, wx) and torch.equal(gb, wb)
        ga.fill_(7)
        two.replay()
        assert torch.equal(ga, wa) and torch.equal(gy, wy)
        one.replay()
        two.replay()
        one.replay()
        assert torch.equal(ga, wa) and torch.equal(gx, wx) and torch.equal(gb, wb) and torch.equal(gy, wy)
    moe.ops_check()
