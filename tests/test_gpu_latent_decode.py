"""Latent attention of one new token over a paged cache against its definition in
64 bits (tests/_latent_util.py says how far off a result may be)."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check
from tests.test_gpu_ops_waits import planted, right_or_untouched

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 192 ** -0.5


def make(lens, H, page, seed=0, spare=3, width=2):
    """queries, cache, table and lengths; unused places of the cache are NaN or infinite"""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B = len(lens)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    q = torch.randn(B, H, 576, generator=g, device=DEV, dtype=torch.bfloat16)
    cache = torch.full((pages, page, 576), float("nan"), device=DEV, dtype=torch.bfloat16)
    cache[:, ::2] = float("inf")
    ids = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max(counts + [0]) + width), -7, dtype=torch.int32, device=DEV)  # unused entries are no pages
    at = 0
    for b, n in enumerate(lens):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
        t = torch.arange(n, device=DEV)
        cache[table[b, t // page].long(), t % page] = torch.randn(n, 576, generator=g, device=DEV, dtype=torch.bfloat16)
    return q, cache, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def tokens(cache, table, b, n):
    t = torch.arange(n, device=DEV)
    return cache[table[b, t // cache.shape[1]].long(), t % cache.shape[1]]


def check_all(out, q, cache, table, lens, scale=SCALE):
    assert out.shape == (q.shape[0], q.shape[1], 512) and out.dtype == torch.bfloat16
    for b, n in enumerate(lens):
        if n == 0:
            assert not out[b].any(), f"sequence {b}"
            continue
        c = tokens(cache, table, b, n)
        check(out[b], *attend(q[b], c, c[:, :512], scale), f"sequence {b} of {n} tokens")


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 192])
@pytest.mark.parametrize("lens,H", [([1], 1), ([63, 64, 65], 16), ([0, 5, 0, 0, 130, 1, 0], 20), ([700], 64), ([257, 1025], 128)])
def test_lengths_heads_and_pages(lens, H, page):
    q, cache, table, lengths = make(lens, H, page, seed=page)
    check_all(moe.latent_decode(q, cache, table, lengths, SCALE), q, cache, table, lens)
    moe.ops_check()


# cut sequences: a long one, several, a boundary at a sequence's start, short ones beside them
@pytest.mark.parametrize("lens,H,page", [([20000], 64, 64), ([9999, 1, 30000, 64], 17, 32), ([4096 * k + 7 for k in (1, 3, 2)], 128, 64),
                                         ([12000, 0, 5000], 65, 16), ([256] * 40, 48, 64), ([1 + 37 * i for i in range(70)], 8, 16),
                                         ([50000], 200, 64), ([64] * 700, 5, 64), ([3] * 1500 + [0] * 300 + [2000], 2, 16)])
def test_split_over_the_sms(lens, H, page):
    q, cache, table, lengths = make(lens, H, page, seed=H)
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    check_all(out, q, cache, table, lens)
    assert torch.equal(out, moe.latent_decode(q, cache, table, lengths, SCALE))
    moe.ops_check()


def test_scores_that_grow_and_that_are_far_apart():
    """the running maximum moves in every tile, by more and by less than what it is let fall behind"""
    for step in (0.02, 0.3, 3.0, -0.3):
        q, cache, table, lengths = make([3000], 33, 64, seed=3)
        t = torch.arange(3000, device=DEV)
        cache[table[0, t // 64].long(), t % 64, 0] = (t * step / 8).to(torch.bfloat16)
        q[:, :, 0] = 8.0
        q[:, 3, 0] = -8.0
        q[:, 4] = 0
        check_all(moe.latent_decode(q, cache, table, lengths, SCALE), q, cache, table, [3000])


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 4.0])
def test_scales(scale):
    q, cache, table, lengths = make([100, 5], 16, 64)
    check_all(moe.latent_decode(q, cache, table, lengths, scale), q, cache, table, [100, 5], scale)


def test_strides_streams_workspaces_and_graphs():
    lens = [500, 0, 77, 1300]
    q, cache, table, lengths = make(lens, 24, 64)
    want = moe.latent_decode(q, cache, table, lengths, SCALE)
    wide = torch.zeros(4, 30, 600, dtype=torch.bfloat16, device=DEV)
    wide[:, 3:27, 8:584] = q
    wide_table = torch.full((4, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    wide_table[:, :table.shape[1]] = table
    assert torch.equal(moe.latent_decode(wide[:, 3:27, 8:584], cache, wide_table[:, :table.shape[1]], lengths, SCALE), want)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(moe.latent_decode(heads_first, cache, table, lengths, SCALE), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.latent_decode(q, cache, table, lengths, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((moe.latent_decode_workspace_bytes(24),), 255, dtype=torch.uint8, device=DEV)
    out = torch.full_like(want, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.latent_decode(q, cache, table, lengths, SCALE, out=out, workspace=ws)
    graph.replay()
    assert torch.equal(out, want)
    lengths.copy_(torch.tensor([1, 300, 77, 0], dtype=torch.int32))     # other lengths, the same graph
    table[1, :5] = table[3, :5]
    graph.replay()
    check_all(out, q, cache, table, [1, 300, 77, 0])
    empty = moe.latent_decode(q[:0], cache, table[:0], lengths[:0], SCALE)
    assert empty.shape == (0, 24, 512)
    moe.ops_check()


def test_bad_pages_and_lengths_are_reported():
    lens = [200, 64, 640]
    q, cache, table, lengths = make(lens, 16, 64, width=0)
    want = moe.latent_decode(q, cache, table, lengths, SCALE)
    for bad in (-1, cache.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[0, 1] = bad
        out = moe.latent_decode(q, cache, t, lengths, SCALE)
        with pytest.raises(moe.MoeFp4Error):
            moe.ops_check()
        assert torch.equal(out[1:], want[1:])
        c = tokens(cache, table, 0, 200)
        c[64:128] = 0
        check(out[0], *attend(q[0], c, c[:, :512], SCALE), "a page outside reads as zeros")
    for length, taken in ((-5, 0), (64 * table.shape[1] + 1, 64 * table.shape[1])):
        n = lengths.clone()
        n[2] = length
        out = moe.latent_decode(q, cache, table, n, SCALE)
        with pytest.raises(moe.MoeFp4Error):
            moe.ops_check()
        check_all(out, q, cache, table, lens[:2] + [taken])
    moe.ops_check()


@pytest.mark.parametrize("lens,H,page", [([20000], 64, 64), ([500] * 60, 20, 16), ([300, 9000, 20], 128, 32)])
def test_a_wait_that_runs_out_stores_nothing_wrong(lens, H, page):
    q, cache, table, lengths = make(lens, H, page)
    want = moe.latent_decode(q, cache, table, lengths, SCALE)
    out = torch.full_like(want, 7.0)
    ws = torch.full((moe.latent_decode_workspace_bytes(H),), 1, dtype=torch.uint8, device=DEV)
    planted(lambda: moe.latent_decode(q, cache, table, lengths, SCALE, out=out, workspace=ws))
    right_or_untouched(out, want, torch.full_like(want, 7.0))
    assert torch.equal(moe.latent_decode(q, cache, table, lengths, SCALE, workspace=ws), want)


def test_places_beyond_32_bits():
    """pages whose elements and bytes lie beyond 2^32"""
    page, lens, H = 64, [300, 129], 16
    q, small, table, lengths = make(lens, H, page)
    cache = torch.empty(2 ** 32 // (576 * page) + 200, page, 576, dtype=torch.bfloat16, device=DEV)
    at = cache.shape[0] - small.shape[0]
    cache[at:] = small
    used = table >= 0
    far = torch.where(used, table + at, table).to(torch.int32)
    want = moe.latent_decode(q, small, table, lengths, SCALE)
    assert torch.equal(moe.latent_decode(q, cache, far, lengths, SCALE), want)
    moe.ops_check()


def test_two_streams_at_once():
    a, b = make([5000, 70], 64, 64, seed=1), make([900] * 20, 24, 16, seed=2)
    wa, wb = moe.latent_decode(*a, SCALE), moe.latent_decode(*b, SCALE)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        ga, gb = moe.latent_decode(*a, SCALE, stream=one), moe.latent_decode(*b, SCALE, stream=two)
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    moe.ops_check()


# pieces of a sequence joined by one part or four, in one round of 32 and in several, with few and with many heads
@pytest.mark.parametrize("lens,H,page", [([9000] + [64] * 7, 64, 64), ([9000, 64, 64, 64], 64, 64), ([32768], 16, 64), ([5000] * 6, 16, 32),
                                         ([4000] * 16, 64, 64), ([8000] + [500] * 7, 128, 64), ([700] * 12, 33, 16)])
def test_pieces_joined(lens, H, page):
    q, cache, table, lengths = make(lens, H, page, seed=len(lens))
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    check_all(out, q, cache, table, lens)
    assert torch.equal(out, moe.latent_decode(q, cache, table, lengths, SCALE))
    moe.ops_check()


@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_among_many_tiles(page):
    """as zeros, wherever they are in a range of tiles; the other sequences are as without them"""
    lens = [3000] * 60
    q, cache, table, lengths = make(lens, 16, page, seed=5)
    whole = moe.latent_decode(q, cache, table, lengths, SCALE)
    moe.ops_check()
    last = (3000 - 1) // page
    for i, bad in zip((0, 7, last // 2, last - 1, last), (-1, cache.shape[0], 2 ** 31 - 1, -2 ** 31, cache.shape[0] + 5)):
        table[3, i] = bad
    out = moe.latent_decode(q, cache, table, lengths, SCALE)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    t = torch.arange(3000, device=DEV)
    pages = table[3, t // page].long()
    c = torch.where(((pages >= 0) & (pages < cache.shape[0]))[:, None], cache[pages.clamp(0, cache.shape[0] - 1), t % page], 0)
    check(out[3], *attend(q[3], c, c[:, :512], SCALE), "pages outside read as zeros")
    others = [b for b in range(60) if b != 3]
    assert torch.equal(out[others], whole[others])
    moe.ops_check()
