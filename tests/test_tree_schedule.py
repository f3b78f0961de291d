"""The barriers of the tree attention kernel (csrc/rkv_dense_tree.cu) under random schedules, on the CPU.

The kernel's warps are generators that name, at each wait, the phase they mean; a wait passes by
parity, as the hardware's does.  A wait that passes in another phase, a ring slot, operand tile or
query tile written while something still reads it, and a state in which nothing can go on are errors.
"""
import random

import pytest


class Fault(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.bytes, self.phase = name, count, count, 0, 0

    def arrive(self):
        if self.left <= 0:
            raise Fault("%s: one arrival too many in phase %d" % (self.name, self.phase))
        self.left -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.bytes == 0:
            self.phase += 1
            self.left = self.count


def bars(name, count, n):
    return [Bar("%s[%d]" % (name, i), count) for i in range(n)]


class Cta:
    """One CTA: runs of blocks of one sequence each; two row tiles or one; scores' buffers; ring slots."""

    def __init__(self, runs, two, bufs, slots, ordered, rng):
        self.runs, self.two, self.bufs, self.slots, self.ordered, self.rng = runs, two, bufs, slots, ordered, rng
        self.raw_full, self.raw_empty = bars("raw_full", 1, slots), bars("raw_empty", 2, slots)
        self.full = [bars("k_full", 4, 2), bars("v_full", 4, 2)]
        self.empty = [bars("k_empty", 2, 2), bars("v_empty", 2, 2)]
        self.s_full, self.p_full, self.o_done = bars("s_full", 1, 4), bars("p_full", 4, 4), bars("o_done", 1, 4)
        self.q_full = bars("q_full", 8, 4)
        self.ring, self.query, self.met = [None] * slots, None, {}
        self.copies, self.products = [], []      # under way: (slot, block); (half, 0 K / 1 V, tile, barriers)
        self.warps = {"producer": self.producer()}
        for w in range(4):
            self.warps["K%d" % w], self.warps["V%d" % w] = self.codes(w, 0), self.codes(w, 1)
        for t in range(2):
            self.warps["products%d" % t] = self.mma(t)
            for w in range(4):
                self.warps["rows%d%d" % (t, w)] = self.rows(t)

    def steps(self, t, blocks):
        ns = (blocks + 1) // 2
        return ns if self.two else (ns + 1 - t) // 2

    def producer(self):
        for i in range(sum(self.runs)):
            slot = i % self.slots
            yield self.raw_empty[slot], i // self.slots - 1
            self.raw_full[slot].bytes += 1
            self.raw_full[slot].arrive()
            self.copies.append((slot, i))

    def codes(self, w, v):
        tile0 = block0 = 0
        for blocks in self.runs:
            for i in range(tile0, tile0 + (blocks + 3) // 4):
                j = 4 * (i - tile0) + w
                block, slot = block0 + j, (block0 + j) % self.slots
                yield self.empty[v][i & 1], (i >> 1) - 1
                if self.ordered and i > 0:
                    yield self.full[v][(i - 1) & 1], (i - 1) >> 1
                if j < blocks:
                    yield self.raw_full[slot], block // self.slots
                for _, kind, tile, _ in self.products:
                    if kind == v and (tile ^ i) & 1 == 0 and tile != i:
                        raise Fault("tile %d written while products read tile %d" % (i, tile))
                yield
                if j < blocks and self.ring[slot] != block:
                    raise Fault("slot %d has block %s for %d" % (slot, self.ring[slot], block))
                self.full[v][i & 1].arrive()
                if j < blocks:
                    self.raw_empty[slot].arrive()
            tile0 += (blocks + 3) // 4
            block0 += blocks

    def mma(self, t):
        tile0 = step0 = 0
        for r, blocks in enumerate(self.runs):
            ns, end = (blocks + 1) // 2, self.steps(t, blocks)

            def place(j):
                g = j if self.two else 2 * j + t
                leaves = not self.two or g & 1 or g + 1 == ns
                return tile0 + (g >> 1), 2 * t + (step0 + j) % self.bufs, (step0 + j) // self.bufs, leaves

            def scores(j):
                tile, buf, phase, leaves = place(j)
                yield self.full[0][tile & 1], tile >> 1
                if phase > 0:
                    yield self.o_done[buf], phase - 1
                if self.query != r:
                    raise Fault("query rows of run %s in run %d" % (self.query, r))
                self.products.append((t, 0, tile, [self.s_full[buf]] + ([self.empty[0][tile & 1]] if leaves else [])))
                yield

            yield self.q_full[r & 3], r >> 2
            for j in range(min(self.bufs, end)):
                yield from scores(j)
            for j in range(end):
                tile, buf, phase, leaves = place(j)
                yield self.full[1][tile & 1], tile >> 1
                yield self.p_full[buf], phase
                self.products.append((t, 1, tile, [self.o_done[buf]] + ([self.empty[1][tile & 1]] if leaves else [])))
                yield
                if j + self.bufs < end:
                    yield from scores(j + self.bufs)
            if not self.two and t == 1 and ns & 1:
                tile = tile0 + (ns >> 1)
                for v in range(2):
                    yield self.full[v][tile & 1], tile >> 1
                for v in range(2):
                    self.empty[v][tile & 1].arrive()
            tile0 += (blocks + 3) // 4
            step0 += end

    def rows(self, t):
        step0 = 0
        for r, blocks in enumerate(self.runs):
            yield self.meet((r, "start"))
            if any(kind == 0 for _, kind, _, _ in self.products):
                raise Fault("query rows written while products read them")
            self.query = r
            self.q_full[r & 3].arrive()
            yield
            end = self.steps(t, blocks)
            for j in range(step0, step0 + end):
                buf, phase = 2 * t + j % self.bufs, j // self.bufs
                yield self.s_full[buf], phase
                if j > step0 and self.rng.random() < 0.3:   # the running maximum grows
                    yield self.o_done[2 * t + (j - 1) % self.bufs], (j - 1) // self.bufs
                yield
                self.p_full[buf].arrive()
            step0 += end
            if end:
                yield self.o_done[2 * t + (step0 - 1) % self.bufs], (step0 - 1) // self.bufs
            yield self.meet((r, "outputs"))
            yield self.meet((r, "end"))

    def meet(self, key):
        self.met[key] = self.met.get(key, 0) + 1
        return key

    def play(self):
        rng = self.rng
        speed = {w: rng.choice([1, 1, 3, 10, 60]) for w in self.warps}
        landing, multiplying = rng.choice([0.5, 0.1, 0.02]), rng.choice([0.5, 0.1, 0.02])
        at = dict.fromkeys(self.warps)

        def ready(w):
            x = at[w]
            return x is None or (self.met[x] == 8 if isinstance(x[1], str) else (x[0].phase ^ x[1]) & 1)

        while self.warps:
            if self.copies and rng.random() < landing:       # in any order
                slot, block = self.copies.pop(rng.randrange(len(self.copies)))
                self.ring[slot] = block
                self.raw_full[slot].bytes -= 1
                self.raw_full[slot].turn()
            if self.products and rng.random() < multiplying:  # in order
                for bar in self.products.pop(0)[3]:
                    bar.arrive()
            can = [w for w in self.warps if ready(w)]
            if not can:
                if self.copies or self.products:
                    continue
                raise Fault("nothing goes on: %s" % {w: x and str(x[0]) for w, x in at.items()})
            w = rng.choices(can, [speed[x] for x in can])[0]
            x = at[w]
            if x and not isinstance(x[1], str) and x[0].phase != x[1] + 1:
                raise Fault("%s passed %s, meant phase %d, in phase %d" % (w, x[0].name, x[1], x[0].phase))
            try:
                at[w] = next(self.warps[w])
            except StopIteration:
                del self.warps[w], at[w]


def play(seed, slots, ordered, lengths):
    rng = random.Random(seed)
    Cta(lengths(rng), rng.random() < 0.5, rng.choice([1, 2]), slots, ordered, rng).play()


def one_run(rng):
    return [rng.choice([3, 16, 25])]


def short_runs(rng):
    return [rng.choice([1, 1, 2, 3, 4, 5, 6, 9, 17]) for _ in range(rng.randint(2, 14))]


# ring slots of the kernel's variants; with fewer than two tiles of them its warps wait for the last tile
@pytest.mark.parametrize("slots", [5, 8])
@pytest.mark.parametrize("lengths", [one_run, short_runs])
def test_no_schedule_goes_wrong(slots, lengths):
    for seed in range(150):
        play(seed, slots, slots < 8, lengths)


def test_a_short_ring_needs_the_wait_for_the_last_tile():
    wrong = 0
    for seed in range(60):
        try:
            play(seed, 5, False, one_run)
        except Fault:
            wrong += 1
    assert wrong > 0
