"""The load warps of the absorbed form, without a GPU.

A wait on a barrier's parity is right only if the barrier cannot run two phases ahead of
the waiting warp: the phase it waits for then looks as if it had not completed.  So each
warp that waits for a stage to be given back has to arrive on the barrier that the
stage's next use begins with.  Which warps wait, and how many arrivals that barrier
counts, are read from the kernel; a model of the barriers then lets one warp fall as far
behind as the others allow."""
import os
import re

import pytest

from tests.test_early_launch_loads import CSRC, code

STAGES = 2


class Barrier:
    """an mbarrier: arrivals of the phase that runs, and its number"""

    def __init__(self, count):
        self.count, self.left, self.phase = count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def completed(self, parity):
        return (self.phase & 1) != parity


def loads(warp, tiles, announces, full, empty):
    """the loading warp's steps; None: it waits"""
    for g in range(tiles):
        s = g % STAGES
        while not empty[s].completed(((g // STAGES) & 1) ^ 1):
            yield False
        if announces:
            full[s].arrive()
        yield True


def multiplies(tiles, full, empty):
    for g in range(tiles):
        s = g % STAGES
        while not full[s].completed((g // STAGES) & 1):
            yield False
        empty[s].arrive()
        yield True


def ends(waiting, announcing, arrivals, tiles, last):
    """whether all warps end if `last` runs only when no other one can"""
    full, empty = [Barrier(arrivals) for _ in range(STAGES)], [Barrier(1) for _ in range(STAGES)]
    warps = {w: loads(w, tiles, w in announcing, full, empty) for w in waiting}
    warps[2] = multiplies(tiles, full, empty)
    while warps:
        moved = False
        for w in sorted(warps, key=lambda w: w == last):
            step = next(warps[w], None)
            if step is None:
                del warps[w]
            if step is not False:
                moved = True
                break
        if not moved:
            return False
    return True


def test_the_model():
    """one that waits without arriving is overtaken; one that arrives is not"""
    assert not ends({0, 1}, {0}, 1, 5, last=1)
    assert ends({0}, {0}, 1, 5, last=0) and ends({0, 1}, {0, 1}, 2, 5, last=1) and ends({0, 1}, {0, 1}, 2, 5, last=0)


def walking_warps(source, copies):
    """the warps that walk the loading loop where a tile's slab comes in `copies` copies"""
    body = source[source.index("if (warp < 2) {"):source.index("} else if (warp == 2) {")]
    condition, = re.findall(r"while \((ok && .*w\.next\(P\))\) \{", body)
    return {w for w in (0, 1) if "warp < loaders" not in condition or w < (1 if copies == 1 else 2)}


@pytest.mark.parametrize("copies", [1, 2, 4])
@pytest.mark.parametrize("tiles", [1, 2, 3, 4, 7, 32])
def test_every_warp_that_waits_for_a_stage_begins_its_next_use(copies, tiles):
    source = code(os.path.join(CSRC, "latent_decode.cu"))
    arrivals = 1 if copies == 1 else 2
    assert re.search(r"mbar_init\(&kv_full\[s\], (loaders|P\.box == kTile \? 1 : 2)\)", source)
    assert "loaders" not in source or "const int loaders = P.box == kTile ? 1 : 2;" in source
    waiting = walking_warps(source, copies)
    announcing = {0} if copies == 1 else {0, 1}
    for last in waiting | {2}:
        assert ends(waiting, announcing, arrivals, tiles, last), f"warp {last} is overtaken"
