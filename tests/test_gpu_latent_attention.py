"""Latent attention in its expanded form against its definition in 64 bits
(tests/_latent_util.py says how far off a result may be)."""
import pytest
import torch

import fp4_mixture_experts_gb300 as moe
from tests._latent_util import attend, check
from tests.test_gpu_ops_waits import planted, right_or_untouched

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SCALE = 192 ** -0.5


def offsets(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=DEV)


def make(q_lens, k_lens, H, seed=0, before=0, after=0):
    """`before` and `after` rows of NaN around the sequences' own"""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def rows(n, *shape):
        t = torch.full((before + n + after, *shape), float("nan"), device=DEV, dtype=BF)
        t[before:before + n] = torch.randn(n, *shape, generator=g, device=DEV, dtype=BF)
        return t

    return (rows(sum(q_lens), H, 192), rows(sum(k_lens), H, 256), rows(sum(k_lens), 64), offsets(q_lens, before),
            offsets(k_lens, before))


def check_all(out, q, kv, rope, qo, ko, causal, scale=SCALE, heads=None, what=""):
    assert out.shape == (q.shape[0], q.shape[1], 128) and out.dtype == BF
    qo, ko = qo.tolist(), ko.tolist()
    for b in range(len(qo) - 1):
        nq, nk = qo[b + 1] - qo[b], ko[b + 1] - ko[b]
        if nq == 0:
            continue
        seen = torch.arange(nq, device=DEV)[:, None] + (nk - nq) >= torch.arange(nk, device=DEV)[None] if causal else None
        for h in range(q.shape[1]) if heads is None else heads:
            got = out[qo[b]:qo[b + 1], h]
            if nk == 0:
                assert not got.any()
                continue
            k = torch.cat([kv[ko[b]:ko[b + 1], h, :128], rope[ko[b]:ko[b + 1]]], 1)
            check(got, *attend(q[qo[b]:qo[b + 1], h], k, kv[ko[b]:ko[b + 1], h, 128:], scale, seen),
                  f"{what} sequence {b} ({nq}, {nk}), head {h}")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 2), (2, 1), (127, 127), (128, 128), (129, 129), (255, 256), (256, 256), (257, 300),
                                   (300, 257), (384, 384), (513, 513), (1, 1000), (100, 0), (200, 50), (700, 900), (64, 1500)])
def test_one_sequence(nq, nk, causal):
    t = make([nq], [nk], 3, seed=nq + nk)
    check_all(moe.latent_attention(*t, SCALE, causal=causal), *t, causal)
    moe.ops_check()


# ragged: empty sequences, single tokens, cached prefixes, more queries than keys; NaN before and behind them, and more
# heads than one round of the SMs
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([5, 0, 1, 300, 0, 64], [9, 7, 1, 300, 0, 1000], 4), ([1] * 40, [3 * i for i in range(40)], 2),
                                             ([257, 129, 1], [600, 129, 0], 24), ([40, 33] * 35, [41, 33] * 35, 1),
                                             ([0, 0], [5, 0], 2), ([1000, 3, 700], [1000, 500, 1400], 16)])
def test_ragged(q_lens, k_lens, H, causal):
    t = make(q_lens, k_lens, H, seed=H, before=3, after=5)
    out = torch.full((t[0].shape[0], H, 128), 7.0, dtype=BF, device=DEV)
    got = moe.latent_attention(*t, SCALE, causal=causal, out=out)
    assert got.data_ptr() == out.data_ptr()
    check_all(out, *t, causal)
    assert (out[:3] == 7).all() and (out[3 + sum(q_lens):] == 7).all()
    assert torch.equal(out[3:3 + sum(q_lens)], moe.latent_attention(*t, SCALE, causal=causal)[3:3 + sum(q_lens)])
    moe.ops_check()


# sequences of few queries and keys, at the limits of their own kernel and beyond, alone and beside long ones
FEW = [(8, 32), (4, 32), (1, 32), (3, 0), (5, 2), (1, 1), (0, 7), (7, 18), (8, 1), (2, 31), (5, 25), (4, 4)]
MORE = [(8, 33), (9, 32), (1, 33), (2, 600), (16, 16)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("pairs,H", [(FEW, 160), (FEW * 3 + MORE, 50), (FEW * 100 + [(1000, 1500)], 2), ([(1, 1)] * 300, 130), ([(4, 30)], 1), (FEW + MORE, 3)])
def test_few_queries_and_keys(pairs, H, causal):
    q_lens, k_lens = [p[0] for p in pairs], [p[1] for p in pairs]
    t = make(q_lens, k_lens, H, seed=H, before=1, after=2)
    out = moe.latent_attention(*t, SCALE, causal=causal)
    check_all(out, *t, causal, heads=sorted({0, H // 2, H - 1}))
    assert torch.equal(out[1:1 + sum(q_lens)], moe.latent_attention(*t, SCALE, causal=causal)[1:1 + sum(q_lens)])
    if causal:                                                    # a key that a query does not see
        for b in (i for i, (nq, nk) in enumerate(pairs) if nq > 1 and nk > 1):
            last_q, last_k = int(t[3][b + 1]) - 1, int(t[4][b + 1]) - 1
            if (nq := pairs[b][0]) <= pairs[b][1]:
                t[1][last_k, :, :128], t[2][last_k] = float("nan"), float("inf")
                again = moe.latent_attention(*t, SCALE)
                assert torch.equal(again[last_q - nq + 1:last_q], out[last_q - nq + 1:last_q])
                break
    moe.ops_check()


def test_a_sequence_is_the_same_beside_any_neighbours():
    """infinities and NaN in the sequences around it, in the same tiles, do not reach it"""
    q_lens, k_lens = [70, 90, 60], [70, 150, 60]
    t = make(q_lens, k_lens, 2, seed=1)
    want = moe.latent_attention(*t, SCALE)
    for value in (float("nan"), float("inf"), -float("inf")):
        q, kv, rope = (x.clone() for x in t[:3])
        q[:70] = value
        q[160:] = value
        for x in (kv, rope):
            x[:70] = value
            x[220:] = value
        assert torch.equal(moe.latent_attention(q, kv, rope, *t[3:], SCALE)[70:160], want[70:160])
    # and a key of its own that a query does not see
    kv, rope = t[1].clone(), t[2].clone()
    kv[69, :, :128] = float("inf")
    rope[69] = float("nan")
    assert torch.equal(moe.latent_attention(t[0], kv, rope, *t[3:], SCALE)[:69], want[:69])


def test_scores_that_grow_and_that_are_far_apart():
    for step in (0.02, 0.3, 3.0, -0.3):
        t = make([300], [2000], 2, seed=3)
        t[1][:, :, 0] = (torch.arange(2000, device=DEV) * step / 8).to(BF)[:, None]
        t[0][:, :, 0] = 8.0
        t[0][5, :, 0] = -8.0
        t[0][6] = 0
        check_all(moe.latent_attention(*t, SCALE), *t, True, what=f"step {step}")
    for scale in (1e-6, 1.0, 4.0):
        t = make([130], [300], 1, seed=4)
        check_all(moe.latent_attention(*t, scale), *t, True, scale, what=f"scale {scale}")


# items of many keys, cut over the SMs: few queries behind long prefixes, ends of pieces at the items' ends, tiles that see
# fewer keys than their item, more queries than keys, more sequences than a block's threads
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([1], [20000], 1), ([130], [9000], 3), ([3, 200, 1], [7000, 300, 30000], 2),
                                             ([2500], [2500], 5), ([300, 1, 0, 64] * 10, [3000, 1, 9, 1200] * 10, 3),
                                             ([4000], [1500], 2), ([1, 2] * 250 + [600], [1, 3] * 250 + [4000], 2),
                                             ([255] * 7, [1100] * 7, 24), ([1] * 30, [1024 + i for i in range(30)], 1)])
def test_items_cut_over_the_sms(q_lens, k_lens, H, causal):
    t = make(q_lens, k_lens, H, seed=len(q_lens), before=2, after=9)
    ws = torch.full((moe.latent_attention_workspace_bytes(),), 255, dtype=torch.uint8, device=DEV)
    out = moe.latent_attention(*t, SCALE, causal=causal, workspace=ws)
    check_all(out, *t, causal, heads=(0, H - 1))
    ws.fill_(1)
    assert torch.equal(out[2:2 + sum(q_lens)], moe.latent_attention(*t, SCALE, causal=causal, workspace=ws)[2:2 + sum(q_lens)])
    moe.ops_check()


def test_many_items_an_sm():
    t = make([2000, 1100], [2000, 2300], 64, seed=5)
    out = moe.latent_attention(*t, SCALE)
    check_all(out, *t, True, heads=(0, 17, 63))
    assert torch.equal(out, moe.latent_attention(*t, SCALE))
    moe.ops_check()


def test_strides_streams_and_graphs():
    q_lens, k_lens, H = [200, 31], [200, 400], 6
    t = make(q_lens, k_lens, H)
    q, kv, rope, qo, ko = t
    want = moe.latent_attention(*t, SCALE)
    wide_q = torch.zeros(231, H + 2, 208, dtype=BF, device=DEV)
    wide_q[:, 1:-1, 8:200] = q
    wide_kv = torch.zeros(600, H, 320, dtype=BF, device=DEV)
    wide_kv[:, :, :256] = kv
    wide_rope = torch.zeros(600, 576, dtype=BF, device=DEV)     # the rotary part of the latent vectors themselves
    wide_rope[:, 512:] = rope
    assert torch.equal(moe.latent_attention(wide_q[:, 1:-1, 8:200], wide_kv[:, :, :256], wide_rope[:, 512:], qo, ko, SCALE), want)
    heads_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, kv)]
    assert torch.equal(moe.latent_attention(*heads_first, rope, qo, ko, SCALE), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.latent_attention(*t, SCALE, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.full_like(want, 7.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.latent_attention(*t, SCALE, out=out)
    graph.replay()
    assert torch.equal(out, want)
    qo.copy_(offsets([100, 131]))                               # other lengths, the same graph
    ko.copy_(offsets([300, 300]))
    graph.replay()
    check_all(out, q, kv, rope, qo, ko, True)
    none = moe.latent_attention(q[:0], kv, rope, offsets([0]), offsets([5]), SCALE)
    assert none.shape == (0, H, 128)
    assert not moe.latent_attention(q, kv[:0], rope[:0], offsets([231]), offsets([0]), SCALE).any()
    moe.ops_check()


def test_offsets_outside_the_rows_are_taken_into_them():
    t = make([100, 100], [150, 150], 2)
    want = moe.latent_attention(*t, SCALE)
    qo, ko = t[3].clone(), t[4].clone()
    qo[0], ko[0], qo[2], ko[2] = -5, -1000, 2 ** 31 - 1, 2 ** 31 - 1
    assert torch.equal(moe.latent_attention(*t[:3], qo, ko, SCALE), want)


@pytest.mark.parametrize("q_lens,k_lens,H", [([300], [300], 1), ([2000, 100], [2000, 3000], 24), ([100, 300], [20000, 4000], 1)])
def test_a_wait_that_runs_out_stores_nothing_wrong(q_lens, k_lens, H):
    t = make(q_lens, k_lens, H)
    want = moe.latent_attention(*t, SCALE)
    out = torch.full_like(want, 7.0)
    planted(lambda: moe.latent_attention(*t, SCALE, out=out))
    right_or_untouched(out, want, torch.full_like(want, 7.0))
    assert torch.equal(moe.latent_attention(*t, SCALE), want)


def test_places_beyond_32_bits():
    """keys whose elements lie beyond 2^32"""
    H, n = 128, 300
    t = make([n], [n], H, seed=7)
    want = moe.latent_attention(*t, SCALE)
    rows = 2 ** 32 // (H * 256) + 500
    kv = torch.empty(rows, H, 256, dtype=BF, device=DEV)
    rope = torch.empty(rows, 64, dtype=BF, device=DEV)
    kv[rows - n:], rope[rows - n:] = t[1], t[2]
    assert torch.equal(moe.latent_attention(t[0], kv, rope, t[3], offsets([n], rows - n), SCALE), want)
    moe.ops_check()


def test_two_streams_at_once():
    a, b = make([700, 70], [9000, 70], 3, seed=1), make([300] * 9, [500] * 9, 24, seed=2)
    wa, wb = moe.latent_attention(*a, SCALE), moe.latent_attention(*b, SCALE)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        ga, gb = moe.latent_attention(*a, SCALE, stream=one), moe.latent_attention(*b, SCALE, stream=two)
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    moe.ops_check()


@pytest.mark.parametrize("q_lens,k_lens,H", [([300, 1, 0, 33], [300, 700, 5, 20], 5), ([200], [5000], 2), ([3, 1, 8], [3, 30, 8], 7)])
def test_results_that_start_on_16_bytes_only(q_lens, k_lens, H):
    """the same bits as where they start on 32, and nothing beside them"""
    t = make(q_lens, k_lens, H, seed=9)
    expect = moe.latent_attention(*t, SCALE)
    flat = torch.full((expect.numel() + 16,), 7.0, dtype=BF, device=DEV)
    out = flat[8:-8].view(expect.shape)
    assert out.data_ptr() % 32 == 16
    moe.latent_attention(*t, SCALE, out=out)
    assert torch.equal(out, expect) and (flat[:8] == 7).all() and (flat[-8:] == 7).all()
    moe.ops_check()


# a tile of queries or less: steps of keys, of either half, whole and cut, between others of two tiles
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("q_lens,k_lens,H", [([128], [129], 1), ([1], [257], 3), ([100, 300, 20], [400, 300, 1100], 2),
                                             ([64], [9000], 5), ([37, 129, 128, 256, 1, 90], [700, 640, 385, 900, 384, 1921], 40),
                                             ([130, 120, 5], [100, 60, 3], 3), ([128] * 9, [128 * i + 7 for i in range(9)], 16)])
def test_one_tile_of_queries(q_lens, k_lens, H, causal):
    t = make(q_lens, k_lens, H, seed=21)
    out = torch.full((sum(q_lens), H, 128), 7.0, dtype=BF, device=DEV)
    moe.latent_attention(*t, SCALE, causal=causal, out=out)
    check_all(out, *t, causal)
    assert torch.equal(out, moe.latent_attention(*t, SCALE, causal=causal))
    moe.ops_check()


def test_one_tile_of_queries_scores_far_apart():
    """the halves' maxima differ by more than any sum can bridge, in either order"""
    for far in (40, 300, 700):
        t = make([50], [1000], 2, seed=far)
        t[1][far:far + 20, :, :128] *= 30
        check_all(moe.latent_attention(*t, SCALE), *t, True)
    moe.ops_check()
