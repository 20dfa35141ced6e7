"""The prompt kernel's barriers over 4-bit pages: a half tile's codes come by one TMA transaction, its group scales by copies of the filling warp's lanes,
each of which arrives when its own have landed (tests/test_prompt_schedule_cpu.py holds the model)."""
import os
import random
import re

import pytest

import test_prompt_schedule_cpu as barriers
from test_paged4_cpu import SHAPES, sizes  # noqa: F401

LANES = 4  # stand for the 32 of a warp


class Flying(list):
    """Copies under way; each half tile's brings its lanes' along, except `missing` of them."""

    def __init__(self, missing):
        super().__init__()
        self.missing = missing

    def append(self, entry):
        super().append(entry)
        if entry[1][0] == "raw_full":
            for _ in range(LANES - self.missing):
                super().append(entry)


class Block4(barriers.Block):
    def __init__(self, units, shape, rings, rng, arrivals=1 + LANES, missing=0):
        super().__init__(units, shape, rings, rng)
        self.flying = Flying(missing)
        for name, bar in self.bar.items():
            if name[0] == "raw_full":
                bar.count = bar.pending = arrivals
        self.landed = {name: 0 for name in self.bar if name[0] == "raw_full"}
        for name in self.landed:
            self.watch(name)

    def watch(self, name):
        arrive = self.bar[name].arrive

        def counted():
            self.landed[name] += 1
            arrive()

        self.bar[name].arrive = counted

    def converter(self):
        # a half tile that is read has all of its copies
        waits = super().converter()
        for wait in waits:
            yield wait
            if wait is not None and wait[0][0] == "raw_full":
                assert self.landed[wait[0]] >= (wait[1] + 1) * (1 + LANES), f"{wait[0]} is read before its copies have landed"


def test_the_source_counts_every_lane():
    text = open(barriers.SOURCE).read()
    assert re.search(r"mbar_init\(&sh\.raw_full\[i\], BITS == 4 \? 1 \+ 32 : 1\)", text)
    assert len(re.findall(r"cp\.async\.mbarrier\.arrive\.noinc", text)) == 1  # without it an arrival would not count against those 33


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bits%d_tiles%d" % s)
def test_half_tiles_are_read_when_codes_and_scales_have_landed(sizes, shape):  # noqa: F811
    rings = tuple(sizes[shape][:3])
    for seed in range(10):
        rng = random.Random(seed)
        Block4(barriers.some_units(rng), shape, rings, rng).run()


def test_the_model_sees_a_wrong_count(sizes):  # noqa: F811
    units, shape = [(6, True)] * 4, SHAPES[0]
    rings = tuple(sizes[shape][:3])
    with pytest.raises(AssertionError):  # the codes alone: halves are read without their scales
        for seed in range(10):
            Block4(units, shape, rings, random.Random(seed), arrivals=1).run()
    with pytest.raises(AssertionError, match="nobody moves"):  # a lane that does not arrive
        for seed in range(10):
            Block4(units, shape, rings, random.Random(seed), missing=1).run()
