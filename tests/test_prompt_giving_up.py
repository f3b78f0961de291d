"""The prompt attention kernel (csrc/rkv_prompt_attention.cu) where a wait runs out, on the CPU: its roles and
barriers as tests/test_prompt_schedule.py plays them, with warps that give up, and what the source has to hold for it."""
import random

import pytest

from test_kernel_sources import block_at, source
from test_prompt_schedule import KINDS, Cta, Fault, random_items


class Copies(list):
    """Copies under way; load number `skip` of K or V is never begun, so that its barrier stays behind."""

    def __init__(self, skip):
        super().__init__()
        self.skip = skip

    def append(self, x):
        if x[0] != "kv" or x[2] != self.skip:
            super().append(x)


class GivingUp(Cta):
    """Once a warp has given up, each wait that does not pass at once makes its warp leave: the producer
    when its copies have landed, the products' warps when what they issued is complete, the others at once."""

    def __init__(self, items, rng, skip=-1, hurry=0.01, drains=("producer", "products"), **kind):
        super().__init__(items, rng=rng, **kind)
        self.copies, self.hurry, self.drains = Copies(skip), hurry, drains
        self.first = None

    def landed(self, loads, uses):
        for k in range(max(0, loads - self.stages), loads):
            yield self.kv_full[k % self.stages], k // self.stages
        for h in range(2):
            if uses[h]:
                yield self.q_full[h], uses[h] - 1

    def producer(self):
        yield from super().producer()
        if "producer" in self.drains:
            halves = range(self.halves)
            yield from self.landed(2 * sum(map(self.count, range(len(self.items)))),
                                   [sum(x[h] > 0 for x in self.items) if h in halves else 0 for h in range(2)])

    def leaving(self, who, local):
        if who == "producer" and "producer" in self.drains and "loads" in local:
            yield from self.landed(local["loads"], local["uses"])
        if who.startswith("products") and "products" in self.drains:
            while self.queues[int(who[-1])]:
                yield None

    def run(self):
        at, alive, leaving = {k: None for k in self.warps}, dict(self.warps), set()

        def leave(k):
            self.first = self.first or k
            g = alive[k]
            while g.gi_yieldfrom is not None and "loads" not in g.gi_frame.f_locals and hasattr(g.gi_yieldfrom, "gi_frame"):
                g = g.gi_yieldfrom
            local = dict(g.gi_frame.f_locals)
            alive[k].close()
            alive[k], at[k] = self.leaving(k, local), None
            leaving.add(k)

        looks = 0                                            # moves in a row of the look through V alone
        for _ in range(200000):
            if not alive:
                break
            blocked = [k for k in alive if at[k] is not None and (at[k][0].phase & 1) == (at[k][1] & 1)]
            can = [k for k in alive if k not in blocked]
            stay = [k for k in blocked if k not in leaving]
            if stay and self.first is None and self.rng.random() < self.hurry:
                leave(self.rng.choice(stay))                 # its limit was the first to pass
                continue
            moves = [("warp", k) for k in can] + [("land", None)] * (len(self.copies) > 0)
            moves += [("product", h) for h in range(self.halves) if self.queues[h]]
            if self.first is not None:
                # the look through V also leaves while it waits for the rows
                moves += [("leave", k) for k in stay + [k for k in can if k == "looker" and k not in leaving]]
            looks = looks + 1 if moves == [("warp", "looker")] else 0
            if not moves or looks > 100:
                if stay:
                    leave(self.rng.choice(stay))
                    continue
                for k in blocked:                            # waits for what will not come run out as well
                    del alive[k]
                continue
            kind, x = self.rng.choice(moves)
            if kind == "land":
                self.land()
            elif kind == "product":
                self.product(x)
            elif kind == "leave":
                leave(x)
            else:
                if at[x] is not None and at[x][0].phase != at[x][1] + 1:
                    raise Fault("%s passed %s in phase %d, meaning %d" % (x, at[x][0].name, at[x][0].phase, at[x][1]))
                try:
                    at[x] = next(alive[x])
                except StopIteration:
                    del alive[x]
        if alive:
            raise Fault("still there: %s" % list(alive))
        if self.copies or any(self.queues):
            raise Fault("left with copies %s and products %s under way" % (list(self.copies), self.queues))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_all_leave_when_one_gives_up(D):
    rng, first = random.Random(D + 3), set()
    for _ in range(400):
        cta = GivingUp(random_items(rng, KINDS[D]["halves"]), rng, hurry=rng.choice([0.003, 0.01, 0.05]), **KINDS[D])
        cta.run()
        first.add((cta.first or "nobody").rstrip("0123456789"))
    assert first >= {"producer", "looker", "products", "rows"}


@pytest.mark.parametrize("D", [64, 128, 256])
def test_all_leave_when_a_load_is_left_out(D):
    rng, gave_up = random.Random(D + 4), 0
    for _ in range(300):
        items = random_items(rng, KINDS[D]["halves"])
        loads = sum(2 * max(x[: KINDS[D]["halves"]]) for x in items)
        cta = GivingUp(items, rng, skip=rng.randrange(loads + 2), hurry=0.0, **KINDS[D])
        cta.run()
        assert (cta.first is not None) == (cta.copies.skip < loads)
        gave_up += cta.first is not None
    assert gave_up > 100


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("drains", [("products",), ("producer",)])
def test_the_model_finds_what_is_left_under_way(D, drains):
    rng, found = random.Random(D + 5), 0
    for _ in range(300):
        try:
            GivingUp(random_items(rng, KINDS[D]["halves"]), rng, hurry=0.05, drains=drains, **KINDS[D]).run()
        except Fault:
            found += 1
    assert found > 0


# ------------------------------------------------------------------ the source
@pytest.fixture(scope="module")
def kernel():
    src = source("rkv_prompt_attention.cu")
    return block_at(src, src.index("k_prompt_attention(const __grid_constant__"))


def test_no_store_to_tensor_memory_is_under_way_when_it_is_freed(kernel):
    # a wait for the products so far comes between a tile's first exponentials, which are stored, and
    # the wait for stores behind the second ones
    rows = block_at(kernel, kernel.index("else if (warp >= 4)"))
    loop_at = rows.index("take(i, w)")
    loop = block_at(rows, loop_at)
    behind = rows[rows.index(loop, loop_at) + len(loop):]
    assert "tmem_st16(" in loop and "break;" in loop
    assert "tmem_wait_st();" in behind
    assert kernel.index(behind) < kernel.index("um::tmem_dealloc(")


def test_every_wait_has_the_calls_limit(kernel):
    waits = kernel.count("um::mbar_wait(") + kernel.count("clock() - t0")
    assert waits == kernel.count("a.wait_cycles") and "kWaitCycles" not in kernel
    # what polls without a limit of its own is within such a loop, or looks once
    assert kernel.count("um::mbar_try_wait(") == 2
