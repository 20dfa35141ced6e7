"""The barriers of the prompt attention kernel (csrc/clo_paged_prompt.cu) under random schedules, as a model on the CPU.

Every role of the kernel is a generator that walks over a block's units as the kernel does; a scheduler runs them in random
order.  Checked: every wait that passes by its phase's parity is for the phase that was meant, nobody waits for ever, operand
slots are filled in order, and lane 0 reads the sums that lane 1 left for the same unit."""
import os
import random
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "host_offloaded_kv_gb300", "csrc", "clo_paged_prompt.cu")
SHAPES = [(d, bits, tiles) for d in (64, 128) for bits in (16, 8) for tiles in (1, 2)]
WARPS = 2  # of a lane, and of the converters: two stand for four


class Bar:
    """An mbarrier: phases done, arrivals pending."""

    def __init__(self, count):
        self.count = self.pending = count
        self.done = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.done += 1
            self.pending = self.count


class Block:
    """One block: `units` are (token tiles, whether the last V tile's end is cleared).  join_always: lane 1 leaves its sums for
    units without tiles too, as the kernel must not."""

    def __init__(self, units, shape, sizes, rng, join_always=False):
        (_, self.bits, self.tiles), (self.slots, self.raw, self.meta) = shape, sizes
        self.units, self.rng, self.join_always = units, rng, join_always
        lane = WARPS  # arrivals of a lane's warps
        conv = 2 * WARPS  # two halves of a tile, each by all converters
        self.bar = {}
        for i in range(self.slots):
            self.bar["full", i] = Bar(1 if self.bits == 16 else conv)
            self.bar["empty", i] = Bar(1)
            self.bar["tail", i] = Bar(1)
        for side in range(2):
            for i in range(self.raw):
                self.bar["raw_full", side, i] = Bar(1)
                self.bar["raw_empty", side, i] = Bar(WARPS)
        for i in range(self.meta):
            self.bar["meta", i] = Bar(1)
        for t in range(2):
            self.bar["q", t] = Bar(lane if self.tiles == 2 else 2 * lane)
            self.bar["s", t] = Bar(1)
            self.bar["p_half", t] = Bar(lane)
            self.bar["p_all", t] = Bar(lane)
        self.flying = []  # copies (land in any order) and commits (in order)
        self.named = {}  # named barriers: [arrived, times passed]
        self.filled = {}  # operand slot -> the element last put there
        self.join = {}

    # -- the kernel's order of operand tiles
    def at_k(self, j):
        return 0 if j == 0 else 2 * j - 1

    def at_v(self, j, n):
        return 2 * j + 2 - (1 if j + 1 >= n else 0)

    def first(self, t):
        return 0 if self.tiles == 2 else t

    def count(self, t, n):
        return n if self.tiles == 2 else (n + 1 - t) // 2

    @property
    def step(self):
        return 1 if self.tiles == 2 else 2

    def sync(self, name, count):
        b = self.named.setdefault(name, [0, 0])
        want = b[1] + 1
        b[0] += 1
        if b[0] == count:
            b[0], b[1] = 0, want
        while b[1] < want:
            yield None

    # -- roles: they yield a wait (barrier, phase) or None for a step
    def producer(self, side):
        e_base = done = 0
        for n, tail in self.units:
            for j in range(n):
                e = e_base + (self.at_k(j) if side == 0 else self.at_v(j, n))
                if self.bits == 16:
                    slot, use = e % self.slots, e // self.slots
                    if use > 0:
                        yield ("empty", slot), use - 1
                        assert self.filled[slot] == e - self.slots
                    self.filled[slot] = e
                    self.flying.append((False, ("tail" if tail and side == 1 and j == n - 1 else "full", slot)))
                else:
                    for h in range(2):
                        x = 2 * (done + j) + h
                        if x >= self.raw:
                            yield ("raw_empty", side, x % self.raw), x // self.raw - 1
                        self.flying.append((False, ("raw_full", side, x % self.raw)))
                        yield None
                if side == 0:
                    self.bar["meta", (done + j) % self.meta].arrive()
                yield None
            e_base += 2 * n
            done += n

    def converter(self):
        e_base = 0
        for n, _ in self.units:
            for i in range(2 * n):
                e = e_base + i
                slot = e % self.slots
                if e >= self.slots:
                    yield ("empty", slot), e // self.slots - 1
                is_v = i > 0 and (i % 2 == 0 or i == 2 * n - 1)
                j = (i + 1) // 2 if not is_v else n - 1 if i == 2 * n - 1 else i // 2 - 1
                assert e == e_base + (self.at_v(j, n) if is_v else self.at_k(j))
                for h in range(2):
                    x = e_base + 2 * j + h
                    buf = x % self.raw
                    yield ("raw_full", int(is_v), buf), x // self.raw
                    self.bar["full", slot].arrive()
                    yield None
                    self.bar["raw_empty", int(is_v), buf].arrive()
                    yield None
            e_base += 2 * n

    def clearer(self):
        phase, e_base = {}, 0
        for n, tail in self.units:
            if tail:
                slot = (e_base + 2 * n - 1) % self.slots
                yield ("tail", slot), phase.get(slot, 0)
                phase[slot] = phase.get(slot, 0) + 1
                self.bar["full", slot].arrive()
            e_base += 2 * n

    def commit(self, *name):
        self.flying.append((True, name))

    def issuer(self):
        q = e_base = 0
        p = [0, 0]
        for n, _ in self.units:
            if n == 0:
                continue
            for t in range(2):
                if self.tiles == 2 or t == 0:
                    yield ("q", t), q
                if self.count(t, n) == 0:
                    break
                e = e_base + self.at_k(self.first(t))
                yield ("full", e % self.slots), e // self.slots
                self.commit("s", t)
                if self.tiles == 1 or t == 1:
                    self.commit("empty", e % self.slots)
            q += 1
            for j in range(n):
                ev, more = e_base + self.at_v(j, n), j + self.step < n
                ek = e_base + self.at_k(j + self.step) if more else 0
                yield ("full", ev % self.slots), ev // self.slots
                if more:
                    yield ("full", ek % self.slots), ek // self.slots
                for v in range(self.tiles):
                    t = v if self.tiles == 2 else j & 1
                    yield ("p_half", t), p[t]
                    yield ("p_all", t), p[t]
                    p[t] += 1
                    if v == self.tiles - 1:
                        self.commit("empty", ev % self.slots)
                    self.commit("s", t)
                if more:
                    self.commit("empty", ek % self.slots)
            e_base += 2 * n

    def softmax(self, t, warp):
        q = s = done = 0
        tile = t if self.tiles == 2 else 0
        threads = WARPS * (1 if self.tiles == 2 else 2)
        for unit, (n, _) in enumerate(self.units):
            if n > 0:
                yield from self.sync(("load", tile), threads)
                self.bar["q", tile].arrive()
                yield ("q", tile), q
                q += 1
            mine = self.count(t, n)
            for i in range(mine):
                j = self.first(t) + i * self.step
                yield ("meta", (done + j) % self.meta), (done + j) // self.meta
                yield ("s", t), s
                s += 1
                self.bar["p_half", t].arrive()
                yield None
                self.bar["p_all", t].arrive()
                yield None
            if mine > 0:
                yield ("s", t), s
                s += 1
            if self.tiles == 1 and (n > 0 or self.join_always):
                if t == 1:
                    self.join[warp] = unit
                yield from self.sync("join", threads)
            if self.tiles == 1 and t == 0 and self.count(1, n) > 0:
                yield None  # lane 0 gets to it in its own time
                assert self.join[warp] == unit, f"lane 0 reads the sums of unit {self.join[warp]} for unit {unit}"
            done += n

    def run(self):
        roles = [self.producer(0), self.producer(1), self.issuer()]
        roles += [self.softmax(t, w) for t in range(2) for w in range(WARPS)]
        roles += [self.clearer()] if self.bits == 16 else [self.converter() for _ in range(WARPS)]
        rng, waits = self.rng, [None] * len(roles)
        live = list(range(len(roles)))
        speed = [rng.random() ** 3 + 1e-3 for _ in roles]
        land, idle = rng.random() ** 2 + 1e-2, 0
        while live:
            if self.flying and rng.random() < land:
                k = rng.randrange(len(self.flying))
                if self.flying[k][0]:
                    k = next(i for i, f in enumerate(self.flying) if f[0])
                self.bar[self.flying.pop(k)[1]].arrive()
                idle = 0
                continue
            i = rng.choices(live, [speed[k] for k in live])[0]
            if waits[i] is not None:
                name, phase = waits[i]
                b = self.bar[name]
                if (b.done & 1) == (phase & 1):
                    idle += 1
                    assert idle < 100000, f"nobody moves: {waits}"
                    continue
                assert b.done > phase, f"{name} passes before phase {phase}"
                waits[i] = None
            idle = 0
            try:
                waits[i] = next(roles[i])
            except StopIteration:
                live.remove(i)


@pytest.fixture(scope="module")
def sizes(tmp_path_factory):
    """(operand slots, 8-bit buffers of a side, tiles of page data) of every shape, from the kernel's source."""
    text = open(SOURCE).read()
    parts = re.findall(r"^constexpr int k(?:Tok|Rows) = \d+;", text, re.M)
    parts += re.findall(r"^template <int D, int BITS, int TILES>\nstruct Cfg \{.*?^\};", text, re.M | re.S)
    assert len(parts) == 3
    body = "".join(f'printf("%d %d %d\\n", Cfg<{d}, {b}, {t}>::kSlots, Cfg<{d}, {b}, {t}>::kRawSide, Cfg<{d}, {b}, {t}>::kMeta);'
                   for d, b, t in SHAPES)
    src = tmp_path_factory.mktemp("cfg") / "cfg.cpp"
    src.write_text("#include <cstdint>\n#include <cstdio>\n" + "\n".join(parts) + "\nint main() {" + body + "}\n")
    exe = str(src)[:-4]
    subprocess.run(["g++", "-std=c++17", str(src), "-o", exe], check=True)
    rows = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    return {shape: tuple(map(int, row.split())) for shape, row in zip(SHAPES, rows)}


def some_units(rng, most=12):
    units = []
    for _ in range(rng.randint(1, 8)):
        n = rng.choice([0, 1, 1, 2, 3, rng.randint(1, most)])
        units.append((n, n > 0 and rng.random() < 0.5))
    return units


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "d%d_bits%d_tiles%d" % s)
def test_every_schedule_keeps_the_barriers_in_step(sizes, shape):
    for seed in range(10):
        rng = random.Random(seed)
        Block(some_units(rng), shape, sizes[shape], rng).run()


def test_units_without_tiles_leave_the_sums_of_the_unit_before(sizes):
    # one row tile: lane 0 may still be reading when lane 1 is at the next unit, which has no token
    shape = (128, 16, 1)
    units = [(4, False), (0, False), (0, False), (3, True), (0, False), (2, False)] * 2
    for seed in range(30):
        Block(units, shape, sizes[shape], random.Random(seed)).run()
    with pytest.raises(AssertionError, match="reads the sums"):  # the model sees the fault where sums are left for every unit
        for seed in range(30):
            Block(units, shape, sizes[shape], random.Random(seed), join_always=True).run()
