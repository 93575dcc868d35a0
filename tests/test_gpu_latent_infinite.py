"""Scores of -infinity in both forms of latent attention: some of a query's are weights of
zero, all of them leave 0 / 0, NaN, as in the formula; a query that sees nothing gets
zeros."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check
from tests.test_gpu_latent_attention import SCALE, make
from tests.test_gpu_latent_decode import make as make_cache

pytestmark = pytest.mark.gpu
DEV = "cuda"


# whole and cut items, few queries and keys, a tile and several; more queries than keys
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([70, 30], [100, 30], 3), ([4, 8], [20, 32], 5), ([64, 9], [9000, 40], 2), ([600], [3000], 2),
                                             ([300, 6], [200, 3], 2)])
def test_expanded(q_lens, k_lens, H, causal):
    q, kv, rope, qo, ko = make(q_lens, k_lens, H, seed=3)
    n, m = k_lens[0], q_lens[0]
    rope[:n, 0] = -torch.inf                                # the first sequence's keys, all of them, where a query's element is positive
    q[:, :, 128] = 0.5
    out = moe.latent_attention(q, kv, rope, qo, ko, SCALE, causal=causal)
    sees = torch.arange(m, device=DEV) + (n - m) >= 0 if causal else torch.ones(m, dtype=torch.bool, device=DEV)
    assert torch.isnan(out[:m][sees]).all() and not out[:m][~sees].any()
    rope[n // 2:n, 0] = 0.25                                # half of them: the others are weights of zero
    out = moe.latent_attention(q, kv, rope, qo, ko, SCALE, causal=causal)
    seen = torch.arange(m, device=DEV)[:, None] + (n - m) >= torch.arange(n, device=DEV)[None]
    keys = torch.arange(n, device=DEV) >= n // 2
    use = (seen if causal else torch.ones_like(seen)) & keys[None]
    some = use.any(1)
    for h in range(H):
        k = torch.cat([kv[:n, h, :128], rope[:n]], 1).clone()
        k[:n // 2] = 0
        want, bound = attend(q[:m, h], k, kv[:n, h, 128:], SCALE, use)
        check(out[:m, h][some], want[some], bound[some], f"head {h}")
    assert torch.isnan(out[:m][~some & sees]).all() and not out[:m][~sees].any()
    for h in range(H) if len(q_lens) > 1 else ():            # the neighbour
        s = torch.arange(q_lens[1], device=DEV)[:, None] + (k_lens[1] - q_lens[1]) >= torch.arange(k_lens[1], device=DEV)[None]
        k = torch.cat([kv[n:, h, :128], rope[n:]], 1)
        near = (s.any(1) if causal else torch.ones_like(s[:, 0]))
        want, bound = attend(q[m:, h], k, kv[n:, h, 128:], SCALE, s if causal else None)
        check(out[m:, h][near], want[near], bound[near], "neighbour")
    moe.ops_check()


@pytest.mark.parametrize("lens,H,page", [([100, 30], 16, 64), ([9000, 5], 20, 16), ([1, 64], 3, 32)])
def test_absorbed(lens, H, page):
    q, cache, table, lengths = make_cache(lens, H, page)
    q[:, :, 512] = 0.5
    q[0, 1, 512] = -0.5                                     # this head's scores are +infinity: NaN too
    t = torch.arange(lens[0], device=DEV)
    at = (table[0, t // page].long(), t % page)
    cache[at[0], at[1], 512] = -torch.inf
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    if lens[0] > 1:
        half = lens[0] // 2
        cache[at[0][half:], at[1][half:], 512] = 0.25
        q[0, 1, 512] = 0.5
        out = moe.latent_decode(q, cache, table, lengths, SCALE)
        c = cache[at][half:]
        check(out[0], *attend(q[0], c, c[:, :512], SCALE), "half of the tokens")
    moe.ops_check()
