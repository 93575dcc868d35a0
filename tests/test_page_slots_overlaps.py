"""page_slots' outputs lie apart from its inputs and from one another; without a GPU: what
overlaps is refused on the host, before anything is enqueued."""
import ctypes
import itertools
import os

import pytest

import fp4_mixture_experts_gb300 as moe
from fp4_mixture_experts_gb300 import build as build_mod
from fp4_mixture_experts_gb300._ops import PageSlotsArgs

FAKE = 0x100000  # never dereferenced
B, WIDTH, STRIDE, TOKENS, FREE = 4, 3, 20, 10, 5
INPUTS = {"lengths": 4 * B, "new_tokens": 4 * B, "free_pages": 4 * FREE}
OUTPUTS = {"slots": 8 * TOKENS, "positions": 4 * TOKENS, "out_lengths": 4 * B, "q_offsets": 4 * B + 4, "k_offsets": 4 * B + 4, "taken": 4}
PLACES = {n: FAKE + 4096 * i for i, n in enumerate([*INPUTS, *OUTPUTS, "table"])}


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.lib_path()):
        build_mod.build()
    return moe.load_library()


def refused(lib, **kw):
    """whether the arguments are refused.  (The sizes are refused last: a batch that is not is not enqueued either.)"""
    a = PageSlotsArgs()
    for k, v in {**dict(B=B, page=64, width=WIDTH, tokens=TOKENS, free_count=FREE, table_stride=STRIDE), **PLACES, **kw}.items():
        setattr(a, k, v)
    return lib.moe_fp4_page_slots(ctypes.byref(a), None) == -1


@pytest.mark.parametrize("out,other", [(o, i) for o in OUTPUTS for i in [*INPUTS, *OUTPUTS] if o != i])
def test_an_output_over_another_operand(lib, out, other):
    size = {**INPUTS, **OUTPUTS}
    step = 8 if out == "slots" else 4
    at = PLACES[other]
    assert refused(lib, **{out: at})
    assert refused(lib, **{out: at + (size[other] - 4) // step * step})             # its last bytes
    if size[out] > step:
        assert refused(lib, **{out: at - (size[out] - step)})                       # the output's last ones


@pytest.mark.parametrize("name", [*INPUTS, *OUTPUTS])
@pytest.mark.parametrize("row", range(B))
def test_an_operand_over_the_table(lib, name, row):
    at = PLACES["table"] + 4 * STRIDE * row
    step = 8 if name == "slots" else 4
    size = {**INPUTS, **OUTPUTS}[name]
    assert refused(lib, **{name: at}) and refused(lib, **{name: at + 4 * (WIDTH - 1) // step * step})
    assert refused(lib, **{name: (at - size + 4 + step - 1) // step * step})
