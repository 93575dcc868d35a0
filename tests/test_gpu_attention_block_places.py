"""The attention block with batches that are filled up to a fixed size, and with requests
that the free pages do not hold: nothing faults, the other requests are as without them,
and what has no place is not written."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import block
from tests.test_gpu_attention_block import D, PAGE, attention_weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def inputs(T, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(T, D, generator=g, device=DEV, dtype=torch.bfloat16)


def bits(x):
    return x.view(torch.int16)


def filled(W, lens, pages=40, width=5, rows=None):
    """cache and table of requests that a prompt each has brought in; the free pages"""
    rows = len(lens) if rows is None else rows
    cache = torch.full((pages, PAGE, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)
    x = inputs(sum(lens), seed=9)
    p = moe.page_slots(i32([0] * rows), i32(lens + [0] * (rows - len(lens))), table, free, PAGE, sum(lens))
    block.attention_forward(x, moe.rms_norm(x, W.next_norm), W, cache, table, p, True)
    moe.ops_check()
    return cache, table, free[int(p.taken):].clone()


# (sequences of one tile each stay whole in any batch: the same bits)
@pytest.mark.parametrize("real", [0, 1, 3])
def test_a_captured_step_of_fixed_size(real):
    W, lens = attention_weights(), [20, 3, 16, 9]
    cache, table, free = filled(W, lens)
    n, new = i32(lens), i32([1] * 4)
    residual = inputs(4)
    normed = moe.rms_norm(residual, W.next_norm)
    whole, t = cache.clone(), table.clone()
    p = moe.page_slots(n, new, t, free, PAGE, 4)
    want = block.attention_forward(residual, normed, W, whole, t, p, False)
    n[real:], new[real:] = 0, 0
    t = table.clone()
    out = moe.page_slots(n, new, t, free, PAGE, 4)
    block.attention_forward(residual, normed, W, cache.clone(), t, out, False)
    captured, t = cache.clone(), table.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = moe.page_slots(n, new, t, free, PAGE, 4, out=out)
        got = block.attention_forward(residual, normed, W, captured, t, out, False)
    for step in range(20):
        graph.replay()
        moe.ops_check()
        if step == 0:
            assert out.slots.tolist() == p.slots.tolist()[:real] + [-1] * (4 - real)
            for a, b in zip(got, want):
                assert torch.equal(bits(a[:real]), bits(b[:real]))
            other = torch.ones(whole.shape[0] * PAGE, dtype=torch.bool, device=DEV)
            other[p.slots] = False
            flat, before, after = (bits(c.view(-1, 576)) for c in (captured, cache, whole))
            assert torch.equal(flat[other], before[other])
            assert torch.equal(flat[p.slots[:real]], after[p.slots[:real]]) and torch.equal(flat[p.slots[real:]], before[p.slots[real:]])
        n.copy_(out.lengths)                                # the next step's
        free.copy_(free.roll(-int(out.taken)))
    assert out.lengths.tolist() == [a + 20 for a in lens[:real]] + [0] * (4 - real)


@pytest.mark.parametrize("prompt", [False, True])
def test_too_few_free_pages(prompt):
    """the second request's token has no place: reported, not written, and the others do not notice"""
    W, lens = attention_weights(), [20, 16, 9, 32]
    cache, table, free = filled(W, lens)
    residual = inputs(4)
    normed = moe.rms_norm(residual, W.next_norm)
    n, new = i32(lens), i32([1] * 4)
    kw = dict(cached_tokens=sum(lens) + 4) if prompt else {}
    whole, t = cache.clone(), table.clone()
    p = moe.page_slots(n, new, t, free, PAGE, 4)
    want = block.attention_forward(residual, normed, W, whole, t, p, prompt, **kw)
    moe.ops_check()
    few, t = cache.clone(), table.clone()
    q = moe.page_slots(n, new, t, free[:1], PAGE, 4)
    assert q.slots.tolist() == p.slots.tolist()[:3] + [-1]  # (requests 1 and 3 need a page each)
    got = block.attention_forward(residual, normed, W, few, t, q, prompt, **kw)
    torch.cuda.synchronize()
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    for a, b in zip(got, want):
        assert torch.equal(bits(a[:3]), bits(b[:3]))
    changed = (bits(few) != bits(cache)).view(-1, 576).any(1).nonzero().flatten().tolist()
    assert changed == sorted(p.slots.tolist()[:3])


@pytest.mark.parametrize("room", [0, 1, 200])
def test_more_of_prompts_with_room_for_further_tokens(room):
    """cached tokens and new ones behind them, rows for more than there are: the same bits"""
    W, lens, new = attention_weights(), [20, 3, 16, 9], [7, 0, 30, 1]
    cache, table, free = filled(W, lens)
    T, n = sum(new), sum(lens) + sum(new)
    x = inputs(T)
    normed = moe.rms_norm(x, W.next_norm)
    p = moe.page_slots(i32(lens), i32(new), table, free, PAGE, T)
    one, two = cache.clone(), cache.clone()
    want = block.attention_forward(x, normed, W, one, table, p, True, cached_tokens=n)
    rows = block.cached_rows(one, table, p, n + room)
    b = torch.repeat_interleave(torch.arange(4, device=DEV), p.lengths)
    at = torch.cat([torch.arange(k, device=DEV) for k in p.lengths.tolist()])
    assert torch.equal(rows[:n], one[table[b, at // PAGE].long(), at % PAGE])
    got = block.attention_forward(x, normed, W, two, table, p, True, cached_tokens=n + room)
    moe.ops_check()
    assert torch.equal(bits(one), bits(two))
    for a, c in zip(got, want):
        assert torch.equal(bits(a), bits(c))


@pytest.mark.parametrize("bad", [-1, 40, 2 ** 31 - 1])
def test_cached_pages_outside_the_cache(bad):
    W, lens, new = attention_weights(), [20, 3, 16, 9], [7, 2, 3, 1]
    cache, table, free = filled(W, lens)
    p = moe.page_slots(i32(lens), i32(new), table, free, PAGE, sum(new))
    moe.ops_check()
    n = int(p.k_offsets[-1])
    want = block.cached_rows(cache, table, p, n)
    table[2, 0] = bad                                       # the third sequence's first 16 tokens
    want[27 + 5:27 + 5 + 16] = 0
    assert torch.equal(bits(block.cached_rows(cache, table, p, n)), bits(want))


def test_cached_tokens_that_are_left_out_are_reported():
    W, lens, new = attention_weights(), [20, 0, 16, 9], [7, 2, 3, 1]
    cache, table, free = filled(W, lens)
    for pad in (0, 100):
        T = sum(new) + pad
        x, n = inputs(T), sum(lens) + sum(new)
        normed = moe.rms_norm(x, W.next_norm)
        t = table.clone()
        p = moe.page_slots(i32(lens), i32(new), t, free, PAGE, T)
        moe.ops_check()
        for kw in ({}, dict(cached_tokens=n - 1)):
            block.attention_forward(x, normed, W, cache.clone(), t, p, True, **kw)
            with pytest.raises(moe.MoeFp4Error):
                moe.ops_check()
        block.attention_forward(x, normed, W, cache.clone(), t, p, True, cached_tokens=n)
        moe.ops_check()


def test_a_request_without_a_token_ahead_of_others_is_reported():
    W, lens = attention_weights(), [20, 3, 16]
    cache, table, free = filled(W, lens)
    x = inputs(3)
    normed = moe.rms_norm(x, W.next_norm)
    for new, right in (([1, 1, 1], True), ([1, 1, 0], True), ([1, 0, 1], False), ([0, 1, 1], False), ([0, 0, 0], True)):
        t = table.clone()
        p = moe.page_slots(i32(lens), i32(new), t, free, PAGE, 3)
        moe.ops_check()
        block.attention_forward(x, normed, W, cache.clone(), t, p, False)
        if right:
            moe.ops_check()
        else:
            with pytest.raises(moe.MoeFp4Error):
                moe.ops_check()


def test_a_prompt_that_the_free_pages_do_not_hold():
    """the second of three: the others' results are as without it missing any"""
    W, new = attention_weights(), [20, 40, 9]
    T, x = sum(new), inputs(sum(new))
    normed = moe.rms_norm(x, W.next_norm)
    cache = torch.full((12, PAGE, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    free, results = i32(list(range(12))), []
    for n in (12, 4):                                       # the second request's third page, and the third one's, are missing
        table = torch.full((3, 4), 5, dtype=torch.int32, device=DEV)
        p = moe.page_slots(i32([0] * 3), i32(new), table, free[:n], PAGE, T)
        results.append(block.attention_forward(x, normed, W, cache.clone(), table, p, True))
        if n < 12:
            assert p.lengths.tolist() == [20, 32, 0] and int(p.taken) == 4
            with pytest.raises(moe.MoeFp4Error):
                moe.ops_check()
    moe.ops_check()
    for a, b in zip(*results):                              # (keys and queries are the new tokens', with a place or without)
        assert torch.equal(bits(a), bits(b))
