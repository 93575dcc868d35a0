"""Every tile of keys counted once, in both forms of latent attention.  With queries of zero
all keys weigh the same; values that are 1 in the column of their tile (or of their place
in it) and 0 elsewhere make each result a count of keys, which one lost or repeated tile
(or key) changes by many times its bound.  Random values do not: their mean over a long
sequence is as small as the bound."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check
from tests.test_gpu_latent_attention import SCALE, make
from tests.test_gpu_latent_decode import make as make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


def signature(n, width, tile, by_tile):
    """[n, width]: key j's column is its tile or its place in the tile, modulo the width"""
    j = torch.arange(n, device=DEV)
    column = (j // tile if by_tile else j % tile) % width
    return torch.nn.functional.one_hot(column, width).to(torch.bfloat16)


def test_a_lost_tile_is_seen():
    """in the definition itself: without a tile, or with one twice, the result is outside the bound (one query, 20000 keys)"""
    for n, width, tile in ((20000, 128, 128), (20000, 512, 64)):
        v = signature(n, width, tile, True)
        q, k = torch.zeros(1, 64, device=DEV), torch.zeros(n, 64, device=DEV)
        want, bound = attend(q, k, v, 1.0)
        for t in range(0, n // tile, 13):
            other = torch.cat([v[:t * tile], v[(t + 1) * tile:]])
            for rows in (other, torch.cat([other, v[t * tile:(t + 1) * tile], v[t * tile:(t + 1) * tile]])):
                off = (attend(q, k[:1].expand(len(rows), -1), rows, 1.0)[0] - want).abs()
                assert (off > 4 * bound).any()


@pytest.mark.parametrize("by_tile", [True, False])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([1], [20000], 1), ([64], [30000], 2), ([130], [9000], 3), ([2500], [2500], 5),
                                             ([255] * 7, [1100] * 7, 24), ([3, 200, 1], [7000, 300, 12000], 2), ([500], [20000], 1),
                                             ([1] * 30, [1024 + i for i in range(30)], 1), ([300], [2047], 40)])
def test_expanded(q_lens, k_lens, H, causal, by_tile):
    q, kv, rope, qo, ko = make(q_lens, k_lens, H)
    q.zero_()
    at = 0
    for n in k_lens:
        kv[at:at + n, :, 128:] = signature(n, 128, 128, by_tile)[:, None]
        at += n
    out = moe.latent_attention(q, kv, rope, qo, ko, SCALE, causal=causal)
    q0 = k0 = 0
    for nq, nk in zip(q_lens, k_lens):
        seen = torch.arange(nq, device=DEV)[:, None] + (nk - nq) >= torch.arange(nk, device=DEV)[None] if causal else None
        zero = torch.zeros(nk, 1, device=DEV)
        want, bound = attend(zero[:1].expand(nq, 1), zero, kv[k0:k0 + nk, 0, 128:], SCALE, seen)
        for h in {0, H // 2, H - 1}:
            check(out[q0:q0 + nq, h], want, bound, f"{nq} of {nk}, head {h}")
        q0, k0 = q0 + nq, k0 + nk
    moe.ops_check()


@pytest.mark.parametrize("by_tile", [True, False])
@pytest.mark.parametrize("lens,H,page", [([20000], 64, 64), ([9999, 1, 30000, 64], 17, 32), ([12000, 0, 5000], 65, 16), ([4608], 64, 64),
                                         ([4000] * 16, 64, 64), ([32768], 16, 64), ([8000] + [500] * 7, 128, 64), ([700] * 12, 33, 48),
                                         ([4608, 3000, 1200] * 11, 20, 16)])
def test_absorbed(lens, H, page, by_tile):
    q, cache, table, lengths = make_cache(lens, H, page)
    q.zero_()
    for b, n in enumerate(lens):
        t = torch.arange(n, device=DEV)
        cache[table[b, t // page].long(), t % page, :512] = signature(n, 512, 64, by_tile)
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    for b, n in enumerate(lens):
        zero = torch.zeros(n, 1, device=DEV)
        if n:
            want, bound = attend(zero[:1], zero, signature(n, 512, 64, by_tile), SCALE)
            check(out[b], want.expand(H, -1), bound.expand(H, -1), f"sequence {b} of {n} tokens")
        else:
            assert not out[b].any()
    moe.ops_check()
