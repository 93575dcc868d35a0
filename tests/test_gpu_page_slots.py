"""Block tables and slots against a list-by-list account of them."""
import numpy as np
import pytest
import torch

import fp4_mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def make(lens, new, page, spare=5, width=2, seed=0):
    rng = np.random.default_rng(seed)
    owned = [-(-n // page) for n in lens]
    after = [-(-(n + t) // page) for n, t in zip(lens, new)]
    ids = rng.permutation(sum(after) + spare).tolist()
    table = np.full((len(lens), max(after + [0]) + width), -1, dtype=np.int32)
    for b, k in enumerate(owned):
        table[b, :k] = [ids.pop() for _ in range(k)]
    return table, ids


def account(lens, new, table, free, page):
    table, slots, positions, taken = table.copy(), [], [], 0
    for b, (n, t) in enumerate(zip(lens, new)):
        for i in range(n, n + t):
            if i % page == 0:
                table[b, i // page] = free[taken]
                taken += 1
            slots.append(int(table[b, i // page]) * page + i % page)
            positions.append(i)
    return table, slots, positions, taken


def check(lens, new, page, pad=0, **kw):
    table, free = make(lens, new, page, **kw)
    want, slots, positions, taken = account(lens, new, table, free, page)
    gt, T = i32(table), sum(new) + pad
    p = moe.page_slots(i32(lens), i32(new), gt, i32(free), page, T)
    np.testing.assert_array_equal(gt.cpu().numpy(), want)
    assert p.slots.dtype == torch.int64 and p.slots.tolist() == slots + [-1] * pad
    assert p.positions.tolist() == positions + [0] * pad
    assert p.lengths.tolist() == [n + t for n, t in zip(lens, new)]
    assert p.q_offsets.tolist() == np.cumsum([0] + list(new)).tolist()
    assert p.k_offsets.tolist() == np.cumsum([0] + [n + t for n, t in zip(lens, new)]).tolist()
    assert p.taken.shape == () and int(p.taken) == taken
    moe.ops_check()


@pytest.mark.parametrize("page", [1, 7, 16, 64, 128])
@pytest.mark.parametrize("lens,new", [([0], [1]), ([5], [0]), ([63, 64, 65], [1, 1, 1]), ([0, 0, 0], [0, 0, 0]),
                                      ([0, 3, 100, 0, 17], [200, 0, 28, 0, 1]), ([1000], [3000]), ([128, 0, 64], [0, 64, 128])])
def test_tables_and_slots(lens, new, page):
    check(lens, new, page)
    check(lens, new, page, pad=9)


@pytest.mark.parametrize("B", [255, 256, 257, 1000, 8192])
def test_many_requests(B):
    rng = np.random.default_rng(B)
    lens, new = rng.integers(0, 90, B).tolist(), (rng.integers(0, 5, B) * rng.integers(0, 2, B)).tolist()
    check(lens, new, 16, pad=3)
    check([0] * B, [1] * B, 64)


def test_many_tokens():
    check([100, 0, 7], [40000, 1, 50001], 64)


def test_no_requests_and_no_tokens():
    p = moe.page_slots(i32([]), i32([]), torch.zeros(0, 4, dtype=torch.int32, device=DEV), i32([1, 2]), 64, 3)
    assert p.slots.tolist() == [-1, -1, -1] and p.q_offsets.tolist() == [0] and int(p.taken) == 0 and p.lengths.numel() == 0
    p = moe.page_slots(i32([4]), i32([0]), i32([[3, 9]]), i32([]), 64, 0)
    assert p.slots.numel() == 0 and p.lengths.tolist() == [4] and p.k_offsets.tolist() == [0, 4]
    moe.ops_check()


def test_strided_tables_graphs_and_given_results():
    lens, new, page = [100, 7, 64], [1, 1, 1], 64
    table, free = make(lens, new, page)
    wide = torch.full((3, table.shape[1] + 6), -1, dtype=torch.int32, device=DEV)
    view = wide[:, :table.shape[1]]
    view.copy_(i32(table))
    gl, gn, gf = i32(lens), i32(new), i32(free)
    out = moe.page_slots(gl, gn, view, gf, page, 5)
    assert (wide[:, table.shape[1]:] == -1).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = moe.page_slots(gl, gn, view, gf, page, 5, out=out)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(again, out))
    for _ in range(70):                                     # decode steps
        lens = out.lengths.tolist()
        now = wide.cpu().numpy()[:, :table.shape[1]]
        gl.copy_(out.lengths)
        gf.copy_(gf.roll(-int(out.taken)))
        if max(lens) + 1 > table.shape[1] * page:
            break
        want = account(lens, new, now, gf.tolist(), page)
        graph.replay()
        np.testing.assert_array_equal(view.cpu().numpy(), want[0])
        assert out.slots.tolist() == want[1] + [-1, -1] and out.positions.tolist() == want[2] + [0, 0]
    moe.ops_check()


def fails():
    with pytest.raises(moe.MoeFp4Error):
        moe.ops_check()
    moe.ops_check()


def test_what_does_not_fit_is_reported_and_gets_no_slot():
    # too few free pages: the second request's second page
    t = i32([[4, -1, -1], [-1, -1, -1]])
    p = moe.page_slots(i32([64, 0]), i32([1, 65]), t, i32([8, 9]), 64, 66)
    fails()
    assert t.tolist() == [[4, 8, -1], [9, -1, -1]] and int(p.taken) == 2
    assert p.slots.tolist() == [8 * 64] + list(range(9 * 64, 10 * 64)) + [-1]
    # a request beyond its row
    t = i32([[4], [5]])
    p = moe.page_slots(i32([60, 3]), i32([6, 1]), t, i32([8, 9]), 64, 7)
    fails()
    assert p.slots.tolist() == [4 * 64 + 60 + i for i in range(4)] + [-1, -1, 5 * 64 + 3] and p.lengths.tolist() == [64, 4]
    assert int(p.taken) == 0 and t.tolist() == [[4], [5]]
    # more new tokens than places for them
    p = moe.page_slots(i32([0, 0]), i32([3, 4]), i32([[1], [2]]), i32([5, 6]), 16, 5)
    fails()
    assert p.slots.tolist() == [80, 81, 82, 96, 97] and p.q_offsets.tolist() == [0, 3, 5]
    # negative numbers
    p = moe.page_slots(i32([-3, 1]), i32([2, -9]), i32([[1], [2]]), i32([5, 6]), 16, 4)
    fails()
    assert p.slots.tolist() == [80, 81, -1, -1] and p.lengths.tolist() == [2, 1]
    # a length above the row, and sums that pass 32 bits
    p = moe.page_slots(i32([2 ** 31 - 1] * 3), i32([2 ** 31 - 1] * 3), i32([[1], [2], [3]]), i32([5]), 16, 2)
    fails()
    assert p.slots.tolist() == [-1, -1] and p.lengths.tolist() == [16, 16, 16] and p.q_offsets.tolist() == [0, 2, 2, 2]


def z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def call(lengths=None, new=None, table=None, free=None, page=16, tokens=4, **kw):
    return moe.page_slots(z(2) if lengths is None else lengths, z(2) if new is None else new, z(2, 3) if table is None else table,
                          z(4) if free is None else free, page, tokens, **kw)


REFUSED = {
    "int64 lengths": lambda: call(lengths=z(2, dtype=torch.int64)),
    "strided lengths": lambda: call(lengths=z(4)[::2]),
    "lengths not a tensor": lambda: call(lengths=[1, 2]),
    "other requests": lambda: call(new=z(3)),
    "the table's rows": lambda: call(table=z(3, 3)),
    "the table's type": lambda: call(table=z(2, 3, dtype=torch.int64)),
    "the table's columns apart": lambda: call(table=z(3, 2).t()),
    "one row for all": lambda: call(table=z(1, 3).expand(2, 3)),
    "int64 pages": lambda: call(free=z(4, dtype=torch.int64)),
    "no page": lambda: call(page=0),
    "half a page": lambda: call(page=1.5),
    "negative tokens": lambda: call(tokens=-1),
    "many tokens": lambda: call(tokens=2 ** 31),
    "out of other sizes": lambda: call(out=call(tokens=5)),
    "out's types": lambda: call(out=call()._replace(slots=z(4))),
    "out's strides": lambda: call(out=call()._replace(positions=z(8)[::2])),
}


@pytest.mark.parametrize("name", list(REFUSED))
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()
    moe.ops_check()


def test_the_library_refuses():
    lens = z(2)
    for f in (lambda: call(lengths=z(8193), new=z(8193), table=z(8193, 3)), lambda: call(table=z(2, 0)),
              lambda: call(page=2 ** 30), lambda: call(lengths=lens, out=call()._replace(lengths=lens)),
              lambda: call(new=lens, out=call()._replace(lengths=lens))):
        with pytest.raises(moe.MoeFp4Error):
            f()
    moe.ops_check()
