"""Requests whose new tokens do not all get a place: what page_slots returns is what has
one, whatever the table's rows held before, and the next step goes on from there."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def account(lens, new, table, free, page, tokens):
    """token by token: table, slots, positions, lengths, pages taken, tokens lost"""
    table, slots, positions, after, taken, lost = table.copy(), [], [], [], 0, 0
    for b, (n, t) in enumerate(zip(lens, new)):
        owned, held, placed = -(-n // page), -(-n // page), 0
        for i in range(n, n + t):
            if len(slots) == tokens:
                lost += 1
                continue
            slot = -1
            if i < table.shape[1] * page:
                if i // page >= held and taken < len(free):
                    table[b, i // page] = free[taken]
                    taken, held = taken + 1, held + 1
                if i // page < held:
                    slot = int(table[b, i // page]) * page + i % page
            slots.append(slot)
            positions.append(i if i < table.shape[1] * page else 0)
            placed += slot >= 0
            lost += slot < 0
        after.append(n + placed)
        assert held >= owned
    pad = tokens - len(slots)
    return table, slots + [-1] * pad, positions + [0] * pad, after, taken, lost


def check_call(lens, new, table, free, page, tokens):
    want, slots, positions, after, taken, lost = account(lens, new, table, free, page, tokens)
    t = i32(table)
    p = moe.page_slots(i32(lens), i32(new), t, i32(free), page, tokens)
    if lost:
        with pytest.raises(moe.MoeFp4Error):
            moe.ops_check()
    moe.ops_check()
    np.testing.assert_array_equal(t.cpu().numpy(), want)
    assert p.slots.tolist() == slots and p.positions.tolist() == positions
    assert p.lengths.tolist() == after
    assert p.k_offsets.tolist() == np.cumsum([0] + after).tolist()
    assert p.q_offsets.tolist() == np.minimum(np.cumsum([0] + list(new)), tokens).tolist()
    assert int(p.taken) == taken
    return t, p, lost


def case(rng, B, page, width):
    lens = [int(n) for n in rng.integers(0, page * width + 1, B) * rng.integers(0, 2, B)]
    new = [int(t) for t in rng.integers(0, 3 * page, B) * rng.integers(0, 2, B)]
    ids = rng.permutation(B * width + 8)
    table = ids[:B * width].reshape(B, width).astype(np.int32)  # pages everywhere, the owned ones and old entries behind them
    return lens, new, table, ids[B * width:].astype(np.int32)


@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("B,width", [(1, 3), (5, 4), (40, 6), (300, 3)])
def test_free_pages_and_places_that_run_out(B, width, page):
    rng = np.random.default_rng(1000 * B + page)
    lost = 0
    for _ in range(12):
        lens, new, table, free = case(rng, B, page, width)
        free = free[:int(rng.integers(0, len(free) + 1))]
        tokens = int(rng.integers(0, sum(new) + 4)) if rng.integers(2) else sum(new) + int(rng.integers(0, 5))
        lost += check_call(lens, new, table, free, page, tokens)[2]
    assert lost > 0 or page == 1


def test_old_entries_behind_a_request_are_not_read():
    """the second request's row still names another one's page where its new one is missing"""
    g = torch.Generator(device=DEV)
    g.manual_seed(0)
    page, lens = 16, [20, 16]
    table = np.array([[3, 1, 9], [4, 1, 5]], dtype=np.int32)
    cache = torch.randn(12, page, 576, generator=g, device=DEV, dtype=torch.bfloat16)
    t, p, lost = check_call(lens, [1, 1], table, [], page, 2)
    assert lost == 1 and p.lengths.tolist() == [21, 16]
    q = torch.randn(2, 8, 576, generator=g, device=DEV, dtype=torch.bfloat16)
    out = moe.latent_decode(q, cache, t, p.lengths, 0.1)
    moe.ops_check()
    for b, n in enumerate(p.lengths.tolist()):
        i = torch.arange(n, device=DEV)
        c = cache[t[b, i // page].long(), i % page]
        check(out[b], *attend(q[b], c, c[:, :512], 0.1), f"sequence {b}")


def test_the_next_step_goes_on_where_places_ran_out():
    rng = np.random.default_rng(5)
    page, lens, new = 16, [30, 0, 16, 5], [40, 33, 1, 9]
    ids = rng.permutation(40)
    table = np.full((4, 6), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k], ids = ids[:k], ids[k:]
    whole = account(lens, new, table, ids.tolist(), page, sum(new))
    t, p, lost = check_call(lens, new, table, ids[:3].tolist(), page, sum(new) - 4)
    assert lost > 4 and int(p.taken) == 3
    after = p.lengths.tolist()
    rest = [n + k - a for n, k, a in zip(lens, new, after)]
    t, p, lost = check_call(after, rest, t.cpu().numpy(), ids[3:].tolist(), page, sum(rest))
    assert lost == 0 and p.lengths.tolist() == whole[3]
    np.testing.assert_array_equal(t.cpu().numpy(), whole[0])


def test_pages_are_taken_for_tokens_with_a_place_only():
    """pages of tokens beyond `tokens` stay free"""
    t, p, lost = check_call([0, 0], [20, 40], np.full((2, 4), -1, dtype=np.int32), [7, 8, 9, 10, 11], 16, 30)
    assert lost == 30 and int(p.taken) == 3 and p.lengths.tolist() == [20, 10]
    assert t.tolist() == [[7, 8, -1, -1], [9, -1, -1, -1]]


@pytest.mark.parametrize("bad", [-1, -7, -2 ** 31])
def test_an_owned_page_that_the_table_does_not_name_is_reported(bad):
    for row, lens in ((0, [10, 20, 5]), (1, [16, 30, 0]), (2, [1, 1, 3])):
        table = np.array([[3, 1, 9], [4, 0, 5], [7, 8, 2]], dtype=np.int32)
        at = lens[row] // 16
        table[row, at] = bad
        p = moe.page_slots(i32(lens), i32([1, 1, 1]), i32(table), i32([20, 21, 22]), 16, 3)
        if lens[row] % 16:                                  # else that page is a new one
            assert p.slots[row] == -1
            with pytest.raises(moe.MoeFp4Error):
                moe.ops_check()
        else:
            assert p.slots[row] >= 0
        moe.ops_check()
        assert (p.slots >= 0).sum() == (2 if lens[row] % 16 else 3)


def test_a_negative_free_page_is_reported():
    p = moe.page_slots(i32([0, 3]), i32([20, 1]), i32([[-1, -1], [4, -1]]), i32([6, -2]), 16, 21)
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    assert p.slots.tolist() == [6 * 16 + i for i in range(16)] + [-1] * 4 + [4 * 16 + 3]
    moe.ops_check()
