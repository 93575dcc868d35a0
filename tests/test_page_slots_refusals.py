"""Refusals of page_slots, without a GPU: every bad argument is caught on the host,
before anything is enqueued; and no read-only loads in its source."""
import ctypes
import os
import re

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import PageSlotsArgs
from tests.test_early_launch_loads import CSRC, code

FAKE = 0x100000  # never dereferenced
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


def test_arguments(lib):
    names = ("lengths", "new_tokens", "free_pages", "table", "slots", "positions", "out_lengths", "q_offsets", "k_offsets", "taken")
    base = dict(B=4, page=64, width=3, tokens=10, free_count=5, table_stride=3, **{n: FAKE + 256 * i for i, n in enumerate(names)})

    def call(**kw):
        a = PageSlotsArgs()
        for k, v in {**base, **kw}.items():
            setattr(a, k, v)
        return lib.moe_fp4_page_slots(ctypes.byref(a), None)

    assert lib.moe_fp4_page_slots(None, None) == -1
    for bad in (dict(B=-1), dict(B=8193), dict(page=0), dict(width=0), dict(tokens=-1), dict(tokens=2**31), dict(free_count=-1),
                dict(free_count=2**31), dict(table_stride=2), dict(slots=FAKE + 4),
                *(dict([(n, None)]) for n in names), *(dict([(n, FAKE + 2)]) for n in names)):
        assert call(**bad) == -1, bad
    # results over the inputs that other CTAs still read
    for i in ("lengths", "new_tokens"):
        for o in ("out_lengths", "q_offsets", "k_offsets"):
            assert call(**{o: base[i]}) == -1 and call(**{o: base[i] + 12}) == -1 and call(**{o: base[i] - 16}) == -1
    assert call(page=2**20, width=2**11, table_stride=2**11) == -2


def on(device, *shape, dtype=I32):
    with FakeTensorMode():
        return torch.empty(shape, dtype=dtype, device=device)


def calls(o):
    a = [on("cuda:0", 2), on("cuda:0", 2), on("cuda:0", 2, 3), on("cuda:0", 5)]
    out = moe.PageSlots(on("cuda:0", 4, dtype=torch.int64), on("cuda:0", 4), on("cuda:0", 2), on("cuda:0", 3), on("cuda:0", 3),
                        on("cuda:0"))
    return {
        "new_tokens": lambda: moe.page_slots(a[0], on(o, 2), a[2], a[3], 64, 4),
        "block_table": lambda: moe.page_slots(a[0], a[1], on(o, 2, 3), a[3], 64, 4),
        "free_pages": lambda: moe.page_slots(a[0], a[1], a[2], on(o, 5), 64, 4),
        "out": lambda: moe.page_slots(*a, 64, 4, out=out._replace(positions=on(o, 4))),
    }


@pytest.mark.parametrize("other,message", [("cuda:1", "same GPU"), ("cpu", "GPU tensors")])
@pytest.mark.parametrize("name", list(calls("cpu")))
def test_operands_elsewhere_are_refused(name, other, message):
    with pytest.raises(ValueError, match=message):
        calls(other)[name]()


@pytest.mark.parametrize("what", [r"__ldg\b", r"ld\.global(\.\w+)*\.nc\b", r"__restrict__"])
def test_no_read_only_loads(what):
    assert not re.search(what, code(os.path.join(CSRC, "page_slots.cu")))
