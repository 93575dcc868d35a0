"""The attention block's own indexing, without a GPU: its operators are replaced by
plain ones, so that an index out of range is an exception here and not a fault there.
Tokens without a place (slot -1, or beyond the cache) are what page_slots gives padded
batches and batches that the free pages do not hold."""
import pytest
import torch

from fp4_mixture_experts_gb300 import block
from fp4_mixture_experts_gb300._ops import PageSlots

BF = torch.bfloat16
D, R, H, PAGE, PAGES = 32, 16, 3, 4, 6


def plain(monkeypatch):
    """the operators in their plain form; what attention got, by name"""
    got = {}

    def fp8_linear(x, w, w_scale, offsets=None, **kw):
        if offsets is None:
            return (x.float() @ w.float().t()).to(BF)
        o = offsets.tolist()
        return torch.cat([x[o[e]:o[e + 1]].float() @ w[e].float().t() for e in range(len(w))]).to(BF)

    def rms_norm(x, weight=None, eps=1e-6):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + eps)).to(BF)

    def latent_decode(q, cache, block_table, lengths, scale, workspace=None):
        got["decode"] = (q, cache, block_table, lengths)
        return torch.zeros(q.shape[0], q.shape[1], 512, dtype=BF)

    def latent_attention(q, kv, k_rope, q_offsets, k_offsets, scale):
        got["attention"] = (q, kv, k_rope, q_offsets, k_offsets)
        return torch.zeros(*q.shape[:2], 128, dtype=BF)

    for f in (fp8_linear, rms_norm, latent_decode, latent_attention):
        monkeypatch.setattr(block, f.__name__, f)
    monkeypatch.setattr(block, "block_residual", lambda residual, y, **kw: (residual + y, y))
    return got


def weights():
    g = torch.Generator().manual_seed(1)
    m = lambda *shape: (0.1 * torch.randn(*shape, generator=g)).to(BF)  # noqa: E731
    kw = {n + "_scale": None for n in ("w_down", "w_q", "w_kv", "w_k", "w_v", "w_o")}
    return block.AttentionWeights(w_down=m(R + 576, D), q_norm=None, kv_norm=None, w_q=m(192 * H, R), w_kv=m(256 * H, 512), w_k=m(H, 512, 128),
                                  w_v=m(H, 128, 512), w_o=m(D, 128 * H), next_norm=None, **kw)


def i32(a):
    return torch.tensor(a, dtype=torch.int32)


def slots(lens, new, table, T, out=None):
    """what page_slots gives, and `out` in place of some slots: {token: slot}"""
    s, positions, q, k = [], [], [0], [0]
    for b, (n, t) in enumerate(zip(lens, new)):
        for i in range(n, n + t):
            s.append(int(table[b, i // PAGE]) * PAGE + i % PAGE)
            positions.append(i)
        q.append(q[-1] + t)
        k.append(k[-1] + n + t)
    s, positions = s + [-1] * (T - len(s)), positions + [0] * (T - len(positions))
    for i, v in (out or {}).items():
        s[i] = v
    return PageSlots(torch.tensor(s, dtype=torch.int64), i32(positions), i32([n + t for n, t in zip(lens, new)]), i32(q), i32(k), i32(0))


def run(W, cache, table, p, T, prompt, **kw):
    residual = torch.randn(T, D, generator=torch.Generator().manual_seed(T)).to(BF)
    return block.attention_forward(residual, residual, W, cache, table, p, prompt, **kw)


def bits(x):
    return x.view(torch.int16)


TABLE = i32([[3, 1], [0, 5], [4, 2]])


@pytest.mark.parametrize("prompt", [False, True])
@pytest.mark.parametrize("out", [{1: -1}, {0: -1}, {2: -1}, {0: -1, 2: -1}, {0: -1, 1: -1, 2: -1}, {1: PAGES * PAGE}, {0: 2 ** 40, 2: -1},
                                 {0: 2 ** 40, 1: 2 ** 33, 2: -7}, {}])
def test_tokens_without_a_place_are_not_written(prompt, out, monkeypatch):
    plain(monkeypatch)
    W, lens, new = weights(), [0, 4, 6], [1, 1, 1]
    want = torch.full((PAGES, PAGE, 576), float("nan"), dtype=BF)
    want[0, 0] = -0.0
    cache = want.clone()
    all_placed = want.clone()
    full = slots(lens, new, TABLE, 3)
    run(W, all_placed, TABLE, full, 3, prompt)
    for i in set(range(3)) - set(out):
        s = int(full.slots[i])
        want.view(-1, 576)[s] = all_placed.view(-1, 576)[s]
    run(W, cache, TABLE, slots(lens, new, TABLE, 3, out), 3, prompt)
    assert torch.equal(bits(cache), bits(want))
    assert not torch.isnan(want.view(-1, 576)[full.slots[[i for i in range(3) if i not in out]]]).any()


def test_a_token_at_the_first_place_beside_ones_without(monkeypatch):
    plain(monkeypatch)
    W, cache = weights(), torch.full((PAGES, PAGE, 576), 7.0, dtype=BF)
    other = cache.clone()
    table = i32([[0], [3]])
    run(W, other, table, slots([0, 0], [2, 1], table, 3), 3, True)
    run(W, cache, table, slots([0, 0], [2, 1], table, 3, {1: -1, 2: -1}), 3, True)
    assert torch.equal(cache.view(-1, 576)[0], other.view(-1, 576)[0]) and (cache.view(-1, 576)[1:] == 7).all()


def test_a_padded_step(monkeypatch):
    """requests without a token behind the others: their rows are there, nothing of theirs is written"""
    got = plain(monkeypatch)
    W, cache = weights(), torch.full((PAGES, PAGE, 576), 7.0, dtype=BF)
    table = i32([[3, 1], [0, 5], [9, 9], [-1, -1]])
    p = slots([5, 2, 0, 0], [1, 1, 0, 0], table, 4)
    out, _ = run(W, cache, table, p, 4, False)
    assert out.shape == (4, D)
    changed = (cache.view(-1, 576) != 7).any(1).nonzero().flatten().tolist()
    assert changed == sorted(p.slots[:2].tolist())
    assert got["decode"][3].tolist() == [6, 3, 0, 0]


def test_no_tokens_at_all(monkeypatch):
    plain(monkeypatch)
    W, cache = weights(), torch.full((PAGES, PAGE, 576), 7.0, dtype=BF)
    out, _ = run(W, cache, TABLE, slots([3, 4, 6], [0, 0, 0], TABLE, 0), 0, True)
    assert out.shape == (0, D) and (cache == 7).all()


def rows_of(cache, table, lens):
    """the sequences' vectors side by side; pages outside the cache are zeros"""
    out = []
    for b, n in enumerate(lens):
        for i in range(n):
            page = int(table[b, i // PAGE])
            out.append(cache[page, i % PAGE] if 0 <= page < len(cache) else torch.zeros(576, dtype=BF))
    return torch.stack(out)


@pytest.mark.parametrize("more", [0, 1, 5, 40])
@pytest.mark.parametrize("lens,new", [([3, 0, 5], [2, 4, 1]), ([0, 0, 0], [1, 1, 1]), ([3, 4, 6], [0, 2, 2]), ([0, 7, 0], [0, 1, 0])])
def test_rows_of_cached_tokens_behind_the_last_one(lens, new, more, monkeypatch):
    """room for more tokens than the batch has, as for a captured prompt"""
    got = plain(monkeypatch)
    W, T = weights(), sum(new)
    cache = torch.randn(PAGES, PAGE, 576, generator=torch.Generator().manual_seed(2)).to(BF)
    after = [n + t for n, t in zip(lens, new)]
    run(W, cache, TABLE, slots(lens, new, TABLE, T), T, True, cached_tokens=sum(after) + more)
    q, kv, k_rope, qo, ko = got["attention"]
    assert kv.shape[0] == k_rope.shape[0] == sum(after) + more
    assert torch.equal(k_rope[:sum(after)], rows_of(cache, TABLE, after)[:, 512:])
    assert ko.tolist()[-1] == sum(after)


@pytest.mark.parametrize("bad", [-1, -PAGES, PAGES, 2 ** 31 - 1, -2 ** 31])
def test_cached_pages_outside_the_cache_read_as_zeros(bad, monkeypatch):
    got = plain(monkeypatch)
    W, lens, new = weights(), [5, 3, 8], [1, 1, 0]
    cache = torch.randn(PAGES, PAGE, 576, generator=torch.Generator().manual_seed(2)).to(BF)
    table = TABLE.clone()
    p = slots(lens, new, table, 2)
    table[1, 0] = bad
    run(W, cache, table, p, 2, True, cached_tokens=18)
    assert torch.equal(got["attention"][2], rows_of(cache, table, [6, 4, 8])[:, 512:])
    assert not got["attention"][2][6:10].any() and not got["attention"][1][6:10].any()


@pytest.mark.parametrize("T", [4, 30])
@pytest.mark.parametrize("lens,new", [([0, 0, 0], [1, 2, 1]), ([0, 4, 0], [1, 2, 1]), ([0, 0, 3], [2, 2, 0]), ([1, 0, 0], [0, 3, 1])])
def test_keys_of_the_new_tokens_alone_are_for_batches_without_cached_ones(T, lens, new, monkeypatch):
    """else the offsets lie behind the rows, which latent_attention reports"""
    got = plain(monkeypatch)
    W, cache = weights(), torch.zeros(PAGES, PAGE, 576, dtype=BF)
    p = slots(lens, new, TABLE, T)
    run(W, cache, TABLE, p, T, True)
    q, kv, k_rope, qo, ko = got["attention"]
    assert kv.shape[0] == T and torch.equal(qo, p.q_offsets)
    if any(lens):
        assert ((ko > T) & (ko < 2 ** 31 - 1)).any()
    else:
        assert torch.equal(ko, p.k_offsets)
    assert ko.dtype == torch.int32


def test_keys_of_new_tokens_that_have_no_place(monkeypatch):
    """a prompt whose second request's last tokens found no page: its lengths and the key offsets do not count them, the
    rows of keys are the new tokens' all the same"""
    got = plain(monkeypatch)
    W, cache = weights(), torch.zeros(PAGES, PAGE, 576, dtype=BF)
    p = slots([0, 0, 0], [3, 6, 2], TABLE, 11, {7: -1, 8: -1})
    p = p._replace(lengths=i32([3, 4, 2]), k_offsets=i32([0, 3, 7, 9]))
    run(W, cache, TABLE, p, 11, True)
    assert got["attention"][4].tolist() == [0, 3, 9, 11] and got["attention"][1].shape[0] == 11


@pytest.mark.parametrize("lens,new,right", [([5, 2, 0], [1, 1, 1], True), ([5, 2, 0], [1, 1, 0], True), ([5, 2, 6], [1, 0, 0], True),
                                            ([0, 0, 0], [0, 0, 0], True), ([5, 2, 6], [1, 0, 1], False), ([5, 0, 0], [0, 1, 1], False),
                                            ([5, 2, 6], [2, 1, 0], False), ([5, 2, 6], [0, 0, 1], False)])
def test_a_decoded_token_belongs_to_its_row_s_sequence(lens, new, right, monkeypatch):
    """a request without a token ahead of one with one, or two tokens of one: lengths that latent_decode reports"""
    got = plain(monkeypatch)
    W, cache = weights(), torch.zeros(PAGES, PAGE, 576, dtype=BF)
    p = slots(lens, new, TABLE, 3)
    run(W, cache, TABLE, p, 3, False)
    lengths = got["decode"][3]
    assert lengths.dtype == torch.int32
    if right:
        assert torch.equal(lengths, p.lengths)
    else:
        assert (lengths < 0).any()


@pytest.mark.parametrize("T", [1, 2, 4])
def test_a_decoded_row_for_each_request(T, monkeypatch):
    plain(monkeypatch)
    cache = torch.zeros(PAGES, PAGE, 576, dtype=BF)
    with pytest.raises(ValueError):
        run(weights(), cache, TABLE, slots([5, 2, 6], [1, 0, 0], TABLE, T), T, False)
    assert not cache.any()


def test_rows_to_a_cache_of_no_pages():
    cache = torch.zeros(0, PAGE, 576, dtype=BF)
    block.write_rows(cache, torch.tensor([0, -1, 7]), torch.ones(3, 576, dtype=BF))
    block.write_rows(cache, torch.zeros(0, dtype=torch.int64), torch.ones(0, 576, dtype=BF))


@pytest.mark.parametrize("rows", [torch.ones(3, 576, dtype=torch.float16), torch.ones(3, 576), torch.ones(2, 576, dtype=BF),
                                  torch.ones(3, 512, dtype=BF), torch.ones(576, dtype=BF), torch.ones(1, 576, dtype=BF)])
def test_rows_of_another_type_or_number_are_refused(rows):
    cache = torch.zeros(PAGES, PAGE, 576, dtype=BF)
    with pytest.raises(ValueError):
        block.write_rows(cache, torch.tensor([0, -1, 7]), rows)
    assert not cache.any()


@pytest.mark.parametrize("cache", [torch.zeros(PAGES, PAGE, 576, dtype=torch.float16), torch.zeros(PAGES, PAGE, 512, dtype=BF),
                                   torch.zeros(PAGES, PAGE, 640, dtype=BF)[:, :, :576]])
def test_another_cache_is_refused(cache):
    with pytest.raises(ValueError):
        block.write_rows(cache, torch.tensor([0, -1, 7]), torch.ones(3, 576, dtype=BF))


def test_rows_of_any_strides():
    wide = torch.randn(5, 601, generator=torch.Generator().manual_seed(1)).to(BF)
    cache = torch.zeros(PAGES, PAGE, 576, dtype=BF)
    block.write_rows(cache, torch.tensor([3, -1, 0, 23, 8]), wide[:, 3:579])
    want = torch.zeros(PAGES * PAGE, 576, dtype=BF)
    want[[3, 0, 23, 8]] = wide[[0, 2, 3, 4], 3:579]
    assert torch.equal(cache.view(-1, 576), want)
