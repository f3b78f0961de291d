"""The barriers of the prompt attention kernel (csrc/rkv_prompt_attention.cu) under random schedules, on
the CPU.

The kernel's warps are generators that name, at each wait, the phase they mean; a wait passes by
parity, as the hardware's does.  A wait that passes in another phase; a ring stage, query tile, score
buffer, probabilities, outputs or item slot that is written while something still needs it, or read
before it is there; and a state in which nothing can go on are errors.
"""
import random

import pytest


class Fault(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.copies, self.phase = name, count, count, 0, 0

    def arrive(self):
        if self.left <= 0:
            raise Fault("%s: one arrival too many in phase %d" % (self.name, self.phase))
        self.left -= 1
        self.turn()

    def landed(self):
        self.copies -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.copies == 0:
            self.phase += 1
            self.left = self.count


def bars(name, count, n):
    return [Bar("%s[%d]" % (name, i), count) for i in range(n)]


class Cta:
    """items: (key tiles of half 0, of half 1, first key tile that is looked through)."""

    def __init__(self, items, halves, bufs, parts, stages, turns, rng, q_copied=False, issued=True, order=True):
        self.items, self.halves, self.bufs, self.parts, self.stages = items, halves, bufs, parts, stages
        self.turns, self.rng, self.issued, self.order = turns, rng, issued, order
        self.q_copied, self.q_there, self.rows_q = q_copied, Bar("q_there", 4), [None] * 4     # queries in tensor memory
        self.kv_full, self.kv_empty = bars("kv_full", 1, stages), bars("kv_empty", halves, stages)
        self.q_full, self.q_empty = bars("q_full", 1, 2), bars("q_empty", 4 if q_copied else 1, 2)
        self.s_full = [bars("s_full%d" % h, 1, bufs) for h in range(halves)]
        self.p_full = [bars("p_full%d" % h, 4, max(bufs, parts)) for h in range(halves)]
        self.pv_done = [bars("pv_done%d" % h, 1, max(bufs, parts)) for h in range(halves)]
        self.o_empty, self.turn = bars("o_empty", 4, 2), bars("turn", 1, 2)
        self.v_issued, self.v_clean = bars("v_issued", 1, 4), bars("v_clean", 1, 4)
        self.w_full, self.w_empty = bars("w_full", 1, 4), bars("w_empty", 1 + 5 * halves, 4)
        self.ring, self.works, self.query = [None] * stages, [None] * 4, [None] * 2
        self.s = [[None] * bufs for _ in range(halves)]      # the step whose scores are there
        self.p = [[[None] * 4 for _ in range(parts * bufs)] for _ in range(halves)]
        self.o = [[None, 0] for _ in range(halves)]          # item whose outputs are there, warps that have read them
        self.cleaned, self.slow, self.done = {}, {}, [0] * (4 * halves)
        self.copies, self.queues = [], [[] for _ in range(halves)]
        self.warps = {"producer": self.producer(), "looker": self.looker()}
        for h in range(halves):
            self.warps["products%d" % h] = self.products(h)
            for w in range(4):
                self.warps["rows%d%d" % (h, w)] = self.rows(h, w)

    def count(self, i):
        return max(self.items[i][: self.halves])

    # ---- warps: they yield (barrier, phase) to wait for; None: let others go on
    def take(self, i):
        yield self.w_full[i & 3], i >> 2
        if self.works[i & 3] != i:
            raise Fault("item slot of %d holds %s" % (i, self.works[i & 3]))
        yield None
        if self.works[i & 3] != i:
            raise Fault("item slot of %d was taken" % i)
        self.w_empty[i & 3].arrive()

    def producer(self):
        loads, cleans, uses = 0, 0, [0, 0]
        for i in range(len(self.items) + 1):
            yield self.w_empty[i & 3], (i >> 2) - 1
            self.works[i & 3] = i
            self.w_full[i & 3].arrive()
            if i == len(self.items):
                return
            for j in range(self.count(i)):
                for kv in range(2):
                    if j == 0 and kv < self.halves and self.items[i][kv] > 0:
                        yield self.q_empty[kv], uses[kv] - 1
                        uses[kv] += 1
                        self.query[kv] = None
                        self.q_full[kv].copies += 1
                        self.q_full[kv].arrive()
                        self.copies.append(("q", kv, i, self.q_full[kv]))
                    st = loads % self.stages
                    yield self.kv_empty[st], loads // self.stages - 1
                    self.ring[st] = None
                    self.kv_full[st].copies += 1
                    self.kv_full[st].arrive()
                    self.copies.append(("kv", st, loads, self.kv_full[st]))
                    loads += 1
                    if kv == 1 and j >= self.items[i][2]:
                        self.v_issued[cleans & 3].arrive()
                        cleans += 1

    def looker(self):
        loads = cleans = 0
        for i in range(len(self.items)):
            yield from self.take(i)
            for j in range(self.items[i][2], self.count(i)):
                ld = loads + 2 * j + 1
                st = ld % self.stages
                if self.issued:
                    yield self.v_issued[cleans & 3], cleans >> 2
                yield self.kv_full[st], ld // self.stages
                for _ in range(self.rng.randrange(3)):
                    if self.ring[st] != ld:
                        raise Fault("looks through load %s for %d" % (self.ring[st], ld))
                    yield None
                if self.rng.random() < 0.2:                  # values that are not finite
                    spins = 0
                    while min(self.done) < i:
                        spins += 1
                        if spins > 20000:
                            raise Fault("nothing goes on but the look through V")
                        yield None
                self.cleaned[ld] = True
                self.v_clean[cleans & 3].arrive()
                cleans += 1
            loads += 2 * self.count(i)
        yield from self.take(len(self.items))

    def products(self, h):
        loads = cleans = steps = rounds = had = 0
        for i in range(len(self.items)):
            yield from self.take(i)
            mine, count, part0 = self.items[i][h], self.count(i), self.items[i][2]
            k_next = [loads]

            def scores(j):
                ld, t = k_next[0], steps + j
                k_next[0] += 2
                if ld != loads + 2 * j:
                    raise Fault("scores of tile %d from load %d" % (j, ld))
                done = [self.s_full[h][t % self.bufs], self.kv_empty[ld % self.stages]]
                if j == mine - 1 and not self.q_copied:
                    done.append(self.q_empty[h])
                self.queues[h].append(("scores", i, t, ld, 0, False, done))

            if mine:
                yield self.q_there if self.q_copied else self.q_full[h], had
            for j in range(min(self.bufs, mine)):
                yield self.kv_full[(loads + 2 * j) % self.stages], (loads + 2 * j) // self.stages
                scores(j)
            for j in range(mine):
                t, ld = steps + j, loads + 2 * j + 1
                if j + self.bufs < mine:
                    nxt = loads + 2 * (j + self.bufs)
                    yield self.kv_full[nxt % self.stages], nxt // self.stages
                yield self.kv_full[ld % self.stages], ld // self.stages
                if j >= part0:
                    cl = cleans + j - part0
                    yield self.v_clean[cl & 3], cl >> 2
                    if not self.cleaned.get(ld):
                        raise Fault("V of load %d is not looked through" % ld)
                if j == 0:
                    yield self.o_empty[h], had - 1
                for part in range(self.parts):
                    b = t % self.bufs if self.bufs > 1 else part
                    yield self.p_full[h][b], t // self.bufs
                    if self.turns and part == 0:
                        yield self.turn[h], rounds if h else rounds - 1
                    done = [self.pv_done[h][b]]
                    if part == self.parts - 1:
                        done.append(self.kv_empty[ld % self.stages])
                    self.queues[h].append(("outputs", i, t, ld, part, j == 0 and part == 0, done))
                if j + self.bufs < mine:
                    scores(j + self.bufs)
                if self.turns:
                    self.turn[1 - h].arrive()
                rounds += 1
            for j in range(mine, count):
                for ld in (loads + 2 * j, loads + 2 * j + 1):
                    yield self.kv_full[ld % self.stages], ld // self.stages
                    self.kv_empty[ld % self.stages].arrive()
                if self.turns:
                    yield self.turn[h], rounds if h else rounds - 1
                    self.turn[1 - h].arrive()
                rounds += 1
            loads += 2 * count
            cleans += max(0, count - part0)
            steps += mine
            had += mine > 0
        yield from self.take(len(self.items))
        while self.queues[h]:
            yield None

    def rows(self, h, w):
        steps = had = 0
        for i in range(len(self.items)):
            yield from self.take(i)
            mine = self.items[i][h]
            if self.q_copied and mine:
                yield self.q_full[h], had
                had += 1
                yield None
                if self.query[h] != i:
                    raise Fault("query rows of %s for item %d" % (self.query[h], i))
                if any(q[0] == "scores" for q in self.queues[h]):
                    raise Fault("query rows written under a product")
                self.rows_q[w] = i
                self.q_empty[h].arrive()
                self.q_there.arrive()
            for j in range(mine):
                t = steps + j
                buf = t % self.bufs
                yield self.s_full[h][buf], t // self.bufs
                if self.s[h][buf] != t:
                    raise Fault("scores of step %s for %d" % (self.s[h][buf], t))
                yield None
                if self.s[h][buf] != t:
                    raise Fault("scores of step %d were taken" % t)
                for part in range(self.parts):
                    if (j > 0 or part > 0) and self.rng.random() < 0.3:      # another reference: the outputs so far
                        if self.bufs > 1:
                            yield self.pv_done[h][(t - 1) % self.bufs], (t - 1) // self.bufs
                        elif part > 0:
                            yield self.pv_done[h][0], t
                        if any(q[0] == "outputs" for q in self.queues[h]):
                            raise Fault("outputs rescaled under a product")
                    self.p[h][buf * self.parts + part][w] = t
                    self.p_full[h][buf if self.bufs > 1 else part].arrive()
                    yield None
            if mine:
                t = steps + mine - 1
                yield self.pv_done[h][t % self.bufs if self.bufs > 1 else self.parts - 1], t // self.bufs
                if self.o[h][0] != i:
                    raise Fault("outputs of item %s for %d" % (self.o[h][0], i))
                yield None
                self.o[h][1] += 1
                self.o_empty[h].arrive()
            steps += mine
            yield None
            self.done[4 * h + w] = i + 1
        yield from self.take(len(self.items))

    # ---- what goes on by itself
    def land(self):
        kind, at, what, bar = self.copies.pop(self.rng.randrange(len(self.copies)))
        if kind == "kv":
            self.ring[at] = what
        else:
            self.query[at] = what
        bar.landed()

    def product(self, h):
        # those of one warp are carried out in the order of issue
        kind, i, t, ld, part, first, done = self.queues[h].pop(0 if self.order else self.rng.randrange(len(self.queues[h])))
        if self.ring[ld % self.stages] != ld:
            raise Fault("%s of step %d read load %s for %d" % (kind, t, self.ring[ld % self.stages], ld))
        buf = t % self.bufs
        if kind == "scores":
            if (self.rows_q != [i] * 4) if self.q_copied else (self.query[h] != i):
                raise Fault("scores of item %d with the query of %s, %s" % (i, self.query[h], self.rows_q))
            if t >= self.bufs and any(self.p[h][buf * self.parts + x] != [t - self.bufs, "done"] for x in range(self.parts)):
                raise Fault("scores of step %d over probabilities that are still needed" % t)
            self.s[h][buf] = t
            for x in range(self.parts):
                self.p[h][buf * self.parts + x] = [None] * 4
        else:
            if self.p[h][buf * self.parts + part] != [t] * 4:
                raise Fault("probabilities %s for step %d" % (self.p[h][buf * self.parts + part], t))
            self.p[h][buf * self.parts + part] = [t, "done"]
            if first:
                if self.o[h][0] is not None and self.o[h][1] != 4:
                    raise Fault("outputs of item %s were overwritten" % self.o[h][0])
                self.o[h] = [i, 0]
            elif self.o[h][0] != i or self.o[h][1]:
                raise Fault("outputs of item %d under way with those of %s" % (i, self.o[h][0]))
        for b in done:
            b.arrive()

    def run(self):
        at = {k: None for k in self.warps}                   # what each warp waits for
        alive = dict(self.warps)
        slow = {k: self.rng.choice([1, 1, 1, 8]) for k in self.warps}
        while alive:
            can = []
            for k in alive:
                wait = at[k]
                if wait is None or (wait[0].phase & 1) != (wait[1] & 1):
                    can.append(k)
            moves = [("warp", k) for k in can if self.rng.randrange(slow[k]) == 0]
            moves += [("land", None)] * (len(self.copies) > 0)
            moves += [("product", h) for h in range(self.halves) if self.queues[h]]
            if not moves:
                if can or self.copies:
                    continue
                raise Fault("nothing can go on: %s" % {k: (w[0].name, w[1], w[0].phase) for k, w in at.items() if k in alive and w})
            kind, x = self.rng.choice(moves)
            if kind == "land":
                self.land()
            elif kind == "product":
                self.product(x)
            else:
                wait = at[x]
                if wait is not None and wait[0].phase != wait[1] + 1:
                    raise Fault("%s passed %s in phase %d, meaning %d" % (x, wait[0].name, wait[0].phase, wait[1]))
                try:
                    at[x] = next(alive[x])
                except StopIteration:
                    del alive[x]


KINDS = {64: dict(halves=2, bufs=2, parts=1, stages=8, turns=False), 128: dict(halves=2, bufs=1, parts=2, stages=5, turns=True),
         256: dict(halves=1, bufs=2, parts=1, stages=5, turns=False, q_copied=True)}


def random_items(rng, halves):
    items = []
    for _ in range(rng.randint(1, 7)):
        c1 = rng.choice([0, 1, 1, 2, 3, rng.randint(1, 9)]) if halves == 2 else 0
        c0 = max(0, c1 - rng.choice([0, 0, 1, 2])) if c1 else rng.choice([1, 1, 2, rng.randint(1, 9)])
        most = max(c0, c1)
        items.append((c0, c1, rng.choice([0, max(0, most - 1), max(0, most - 3), most])))
    return items


@pytest.mark.parametrize("D", [64, 128, 256])
def test_no_schedule_breaks_it(D):
    rng = random.Random(D)
    for _ in range(400):
        Cta(random_items(rng, KINDS[D]["halves"]), rng=rng, **KINDS[D]).run()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_short_items(D):
    rng = random.Random(D + 1)
    for _ in range(60):
        Cta([(1, rng.choice([0, 1]) if KINDS[D]["halves"] == 2 else 0, 0) for _ in range(25)], rng=rng, **KINDS[D]).run()


def faults(D, n, **kw):
    rng, found = random.Random(D + 2), 0
    for _ in range(n):
        try:
            Cta(random_items(rng, KINDS[D]["halves"]), rng=rng, **dict(KINDS[D], **kw)).run()
        except Fault:
            found += 1
    return found


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_model_finds_a_look_before_the_load(D):
    # without v_issued, a stage's barrier may still be at the load before
    assert faults(D, 200, issued=False) > 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_model_finds_products_out_of_order(D):
    assert faults(D, 200, order=False) > 0


def test_the_model_finds_a_ring_too_short():
    # six stages of V tiles would need more than four barriers to name them
    assert faults(64, 400, stages=12) > 0
