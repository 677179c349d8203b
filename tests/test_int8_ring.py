"""The ring of block infos of attend_int8's prompts, as a model of its barriers on the host: makers, products and the two halves
of the columns go through the same units under random schedules.  A wait for a phase by its parity tells only neighbouring
phases apart, so the model keeps the number of completed phases beside it and says where a wait passed on another one than
was meant, where an entry was read that holds another batch, and where one was overwritten that was still to be read."""
import os
import random
import re

import pytest

from conftest import ROOT

with open(os.path.join(ROOT, "compressed_kv_cache_gb300", "csrc", "tq_int8_prompt.cu")) as f:
    SOURCE = f.read()
RING = int(re.search(r"kInfo = (\d+);", SOURCE).group(1))
BATCH = int(re.search(r"kBatch = (\d+);", SOURCE).group(1))


class Bar:
    def __init__(self, count):
        self.count, self.here, self.done = count, 0, 0

    def arrive(self):
        self.here += 1
        if self.here == self.count:
            self.here, self.done = 0, self.done + 1


class Model:
    """An agent is a generator that yields (barrier, phase) where it waits and None between two steps.  `follow`: the second half
    goes along with the batches of units that have no columns for it, as the kernel's does."""

    def __init__(self, units, follow, batch=BATCH, ring=RING):
        self.units, self.follow, self.batch, self.ring, self.wrong = units, follow, batch, ring, []
        self.full, self.free = [Bar(1) for _ in range(ring)], [Bar(4) for _ in range(ring)]      # two warps of each half
        self.k_full, self.k_free, self.v_full, self.v_free = ([Bar(1), Bar(1)] for _ in range(4))
        self.s_full, self.p_full = [Bar(1), Bar(1)], [Bar(2), Bar(2)]
        self.info, self.pending = [None] * ring, {}
        self.agents = [self.makers(), self.products()] + [self.columns(half) for half in (0, 0, 1, 1)]

    def makers(self):
        tile = batch = 0
        for n, halves in self.units:
            for i in range(n):
                if i % self.batch == 0:
                    b = batch + i // self.batch
                    if self.follow:
                        yield self.free[b % self.ring], b // self.ring - 1
                    self.write(b, halves)
                    self.full[b % self.ring].arrive()
                yield self.k_free[tile & 1], tile // 2 - 1
                self.k_full[tile & 1].arrive()
                yield self.v_free[tile & 1], tile // 2 - 1
                self.v_full[tile & 1].arrive()
                tile += 1
            batch += -(-n // self.batch)

    def write(self, b, halves):
        old = self.info[b % self.ring]
        if old is not None and self.pending.get(old):
            self.wrong.append(f"batch {old} overwritten before it was read")
        self.info[b % self.ring] = b
        self.pending[b] = 2 * halves

    def products(self):
        tile, done = 0, [0, 0]
        for n, halves in self.units:
            def logits(i):
                yield self.k_full[(tile + i) & 1], (tile + i) // 2
            for i in range(n):
                if i == 0:
                    yield from logits(0)
                    for half in range(halves):
                        self.s_full[half].arrive()
                    self.k_free[tile & 1].arrive()
                yield self.v_full[(tile + i) & 1], (tile + i) // 2
                for half in range(halves):
                    yield self.p_full[half], done[half] + i
                    if half == halves - 1:
                        self.v_free[(tile + i) & 1].arrive()
                    if i + 1 < n:
                        if half == 0:
                            yield from logits(i + 1)
                        self.s_full[half].arrive()
                        if half == halves - 1:
                            self.k_free[(tile + i + 1) & 1].arrive()
            tile += n
            for half in range(halves):
                done[half] += n

    def columns(self, half):
        batch = done = 0
        for n, halves in self.units:
            if half < halves:
                for i in range(n):
                    b = batch + i // self.batch
                    if i % self.batch == 0:
                        yield self.full[b % self.ring], b // self.ring
                    if self.info[b % self.ring] != b:
                        self.wrong.append(f"half {half} reads batch {self.info[b % self.ring]} for {b}")
                    yield None
                    yield self.s_full[half], done + i
                    yield None
                    if i % self.batch == self.batch - 1 or i == n - 1:
                        self.pending[b] = self.pending.get(b, 0) - 1
                    self.p_full[half].arrive()
                    if self.follow and (i % self.batch == self.batch - 1 or i == n - 1):
                        self.free[b % self.ring].arrive()
                done += n
            elif self.follow:
                for i in range(0, n, self.batch):
                    b = batch + i // self.batch
                    yield self.full[b % self.ring], b // self.ring
                    self.free[b % self.ring].arrive()
            batch += -(-n // self.batch)

    def run(self, rng):
        waits = {}
        for a in self.agents:
            waits[a] = next(a, "end")
        while any(w != "end" for w in waits.values()) and not self.wrong:
            ready = [a for a, w in waits.items() if w is None or (w != "end" and w[0].done & 1 != w[1] & 1)]
            if not ready:
                self.wrong.append("nothing can go on")
                break
            a = rng.choices(ready, [rng.choice((1, 1, 50)) for _ in ready])[0]
            if waits[a] is not None and waits[a][0].done != waits[a][1] + 1:
                self.wrong.append(f"a wait for phase {waits[a][1]} passed after {waits[a][0].done} phases")
            waits[a] = next(a, "end")
        return self.wrong


def draw(rng):
    most = rng.choice((1, 2, BATCH, 3 * BATCH))
    return [(rng.choice((0, 1, rng.randint(1, most))), rng.choice((1, 1, 1, 1, 2))) for _ in range(rng.randint(1, 40))]


@pytest.mark.parametrize("seed", range(300))
def test_every_wait_is_for_its_own_phase(seed):
    rng = random.Random(seed)
    units = draw(rng)
    assert not Model(units, True).run(rng), units


def test_without_following_the_ring_it_goes_wrong():
    """Units of one half, then one of two: the second half comes to a barrier that is a phase behind."""
    rng = random.Random(1)
    assert any(Model([(1, 1)] * 6 + [(3, 2)], False).run(rng) for _ in range(20))
    assert any(Model([(3 * BATCH, 1)] * 2 + [(3, 2)], False).run(rng) for _ in range(20))
    assert not any(Model([(7, 2)] * 12, False).run(rng) for _ in range(20))


def test_the_kernel_follows_the_ring():
    """The model's arrivals are the kernel's: each warp of both halves frees an entry, the makers wait for it."""
    assert re.search(r"bar_init\(info_free \+ 8 \* i, 8\)", SOURCE) and re.search(r"bar_init\(info_full \+ 8 \* i, kMakers\)", SOURCE)
    makers = SOURCE[SOURCE.index("codes to operands"):SOURCE.index("a column: its query")]
    assert makers.index("wait_all(info_free") < makers.index("to = f;") < makers.index("arrive(info_full")
    assert "arrive(info_free" in SOURCE[SOURCE.index("auto give_back"):SOURCE.index("if (half >= halves)")]
    skip = SOURCE[SOURCE.index("if (half >= halves)"):SOURCE.index("a column: its query")]
    assert skip.index("wait_all(info_full") < skip.index("give_back(batch)") < skip.index("end();")


def test_no_load_is_under_way_where_the_columns_give_up():
    """The logits read ahead land in registers: they are waited for before the loop can be left, whose end uses registers anew."""
    role = SOURCE[SOURCE.index("a column: its query"):]
    ahead = role.index("at the end the first again, for the weights")
    leave = role.index("if (lost) break;", ahead)
    assert ahead < role.index("tmem_loaded(za);", role.index("largest(zb, k + 1, e1);")) < leave
    assert "break" not in role[leave + len("if (lost) break;"):role.index("out, or a part for the join")]
