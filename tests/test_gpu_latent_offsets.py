"""Latent attention's offsets: those that are no sequences' are reported, and the other
sequences' results do not change."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests.test_gpu_latent_attention import SCALE, check_all, make

pytestmark = pytest.mark.gpu
END = 2 ** 31 - 1


def reported():
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    moe.ops_check()


# a block's search, a warp's, few queries and keys alone, beside others; items cut and whole
SIZES = [([100, 100], [150, 150], 2), ([60] * 40, [300] * 40, 3), ([4, 8], [4, 30], 5), ([2] * 500, [9] * 500, 6), ([300, 20], [3000, 1500], 2)]


@pytest.mark.parametrize("q_lens,k_lens,H", SIZES)
def test_offsets_behind_the_rows(q_lens, k_lens, H):
    t = make(q_lens, k_lens, H)
    want = moe.latent_attention(*t, SCALE)
    moe.ops_check()
    for which, rows in ((3, sum(q_lens)), (4, sum(k_lens))):
        for value in (rows + 1, END - 1):
            o = list(t)
            o[which] = t[which].clone()
            o[which][-1] = value
            out = moe.latent_attention(*o, SCALE)
            reported()
            assert torch.equal(out, want)                   # taken as the rows' end
        o[which][-1] = END                                  # which stands for it
        assert torch.equal(moe.latent_attention(*o, SCALE), want)
        o[which][0] = -3
        assert torch.equal(moe.latent_attention(*o, SCALE), want)
        moe.ops_check()


@pytest.mark.parametrize("which", [3, 4])
@pytest.mark.parametrize("q_lens,k_lens,H", SIZES)
def test_offsets_that_decrease(q_lens, k_lens, H, which):
    """the sequence before the smaller one is empty; those before it are as they were"""
    q_lens, k_lens = q_lens + [6, 5], k_lens + [11, 7]
    t = list(make(q_lens, k_lens, H))
    want = moe.latent_attention(*t, SCALE)
    moe.ops_check()
    t[which] = t[which].clone()
    t[which][-2] = t[which][-3] - 1                         # the last sequence then begins in the one before
    out = moe.latent_attention(*t, SCALE)
    reported()
    before = sum(q_lens[:-3])
    assert torch.equal(out[:before], want[:before])


@pytest.mark.parametrize("causal", [False, True])
def test_fewer_rows_of_keys_than_the_offsets_say(causal):
    """as where only the new tokens' keys are given for sequences that have cached ones"""
    t = make([40, 30], [140, 230], 3)
    short = (t[0], t[1][:200].clone(), t[2][:200].clone(), t[3], t[4])
    out = moe.latent_attention(*short, SCALE, causal=causal)
    reported()
    check_all(out[:40], t[0][:40], t[1], t[2], t[3][:2], t[4][:2], causal)
