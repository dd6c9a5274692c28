"""All barriers of the attention kernel as a model, random schedules over random
lists of parts: the scheduler, the issuer, the two loaders and the two softmax
groups, with copies that land at any later time and products that complete in
the order in which they were issued.

A wait knows a phase by its parity alone. The model finds waits that pass on the
wrong phase, waits that never end, and data that is replaced before its last
reader is done: ring slots, query buffers, scores, weights and outputs. It is a
transcription by hand of the waits and arrivals in csrc/attend.cuh and has to be
changed along with them."""
import random

import pytest

QUEUE = 4  # kAtQueue


class Fault(Exception):
    pass


class Barrier:
    def __init__(self, count):
        self.count, self.arrived, self.done = count, 0, 0  # done: completed phases

    def arrive(self, n=1):
        self.arrived += n
        if self.arrived > self.count:
            raise Fault("more arrivals than a phase takes")
        if self.arrived == self.count:
            self.arrived, self.done = 0, self.done + 1


class Cta:
    """One CTA. parts: [(two row tiles, key tiles, ragged)]."""

    def __init__(self, parts, slots, mistake, rng):
        self.parts, self.slots, self.mistake, self.rng = parts, slots, mistake, rng
        bars = lambda n, count: [Barrier(count) for _ in range(n)]  # noqa: E731
        self.kv_full, self.kv_empty = bars(slots, 1), bars(slots, 1)
        self.part_full, self.part_empty = bars(QUEUE, 1), bars(QUEUE, 11)
        self.q_full, self.q_empty, self.s_full, self.o_full = bars(2, 1), bars(2, 1), bars(2, 1), bars(2, 1)
        self.p_full, self.meet, self.done = bars(2, 4), bars(2, 8), Barrier(1)
        self.ring, self.ring_readers = [None] * slots, [0] * slots  # occupant, reads still to come
        self.queue = [None] * QUEUE
        self.q, self.q_readers = [None, None], [0, 0]
        self.S, self.P, self.O = [None, None], [None, None], [None, None]
        self.O_readers = [0, 0]
        self.copies, self.pipe = [], []

    # ---- what the actors share ----
    def tile_of(self, two, g, j):
        return j if two else 2 * j + g

    def k_at(self, two, t):
        return 2 * t if two else (0 if t == 0 else 2 * t - 1)

    def v_at(self, two, t, tiles):
        return 2 * t + 1 if two else min(2 * t + 2, 2 * tiles - 1)

    def base_of(self, n):
        return sum(2 * p[1] for p in self.parts[:n])

    # ---- warps ----
    def scheduler(self):
        loads = [0, 0]
        late = None

        def load(n):
            two, tiles, _ = self.parts[n]
            for g in range(2):
                if g == 1 and not two and tiles == 1:
                    continue
                if loads[g] > 0:
                    yield self.q_empty[g], loads[g] - 1
                if self.q_readers[g]:
                    raise Fault("queries replaced before their last use")
                mine = tiles if two else (tiles + 1 - g) // 2
                self.q[g], self.q_readers[g] = None, mine
                self.copies.append(("q", g, n))
                loads[g] += 1
                yield None

        for n in range(len(self.parts) + 1):
            if n >= QUEUE:
                yield self.part_empty[n % QUEUE], n // QUEUE - 1
            if n == len(self.parts) and late is not None:
                yield from load(late)
                late = None
            self.queue[n % QUEUE] = n
            self.part_full[n % QUEUE].arrive()
            yield None
            if n == len(self.parts):
                break
            if n == 0:
                yield from load(0)
            else:
                if late is not None:
                    yield from load(late)
                late = n
        for g in range(2):
            if loads[g]:
                yield self.q_full[g], loads[g] - 1

    def part(self, n, weight):
        """The next part, or None; the place is free again after `weight` arrivals."""
        yield self.part_full[n % QUEUE], n // QUEUE
        got = self.queue[n % QUEUE]
        if got != n:
            raise Fault("a part replaced before all have read it")
        self.part_empty[n % QUEUE].arrive(weight)
        yield None
        return None if n == len(self.parts) else self.parts[n]

    def issuer(self):
        waited, qs, ps = 0, [0, 0], [0, 0]
        n = 0
        while True:
            part = yield from self.part(n, 1)
            if part is None:
                break
            two, tiles, _ = part
            base = self.base_of(n)

            def landed(i):
                nonlocal waited
                while waited <= i:
                    yield self.kv_full[waited % self.slots], waited // self.slots
                    waited += 1

            def qk(g, t, last):
                i = base + self.k_at(two, t)
                self.pipe.append(("qk", g, n, t, i))
                self.pipe.append(("arrive", self.s_full[g]))
                if not two or g == 1:
                    self.pipe.append(("arrive", self.kv_empty[i % self.slots]))
                if last:
                    self.pipe.append(("arrive", self.q_empty[g]))

            for g in range(2):
                t = self.tile_of(two, g, 0)
                if t >= tiles:
                    continue
                yield self.q_full[g], qs[g]
                qs[g] += 1
                yield from landed(base + self.k_at(two, t))
                qk(g, t, self.tile_of(two, g, 1) >= tiles)
                yield None
            for j in range(tiles if two else (tiles + 1) // 2):
                for g in range(2):
                    t, nxt = self.tile_of(two, g, j), self.tile_of(two, g, j + 1)
                    if t >= tiles:
                        continue
                    vi = base + self.v_at(two, t, tiles)
                    yield from landed(vi)
                    if nxt < tiles:
                        yield from landed(base + self.k_at(two, nxt))
                    yield self.p_full[g], ps[g]
                    ps[g] += 1
                    self.pipe.append(("pv", g, n, t, vi, j == 0))
                    if not two or g == 1:
                        self.pipe.append(("arrive", self.kv_empty[vi % self.slots]))
                    if nxt < tiles:
                        qk(g, nxt, self.tile_of(two, g, j + 2) >= tiles)
                    else:
                        self.pipe.append(("arrive", self.o_full[g]))
                    yield None
            n += 1
        self.pipe.append(("arrive", self.done))
        yield self.done, 0

    def loader(self, values):
        n = 0
        while True:
            part = yield from self.part(n, 1)
            if part is None:
                return
            two, tiles, _ = part
            for t in range(tiles):
                at = self.base_of(n) + (self.v_at(two, t, tiles) if values else self.k_at(two, t))
                slot, use = at % self.slots, at // self.slots
                if use > 0 and self.mistake != "no wait for a free slot":
                    yield self.kv_empty[slot], use - 1
                if self.ring_readers[slot]:
                    raise Fault("a ring slot filled before its last reader was done")
                self.ring[slot], self.ring_readers[slot] = None, 2 if two else 1
                self.copies.append(("kv", slot, (n, t, "v" if values else "k")))
                yield None
            n += 1

    def group(self, g):
        s, o, meets = 0, [0, 0], 0
        n = 0
        while True:
            part = yield from self.part(n, 4)
            if part is None:
                return
            two, tiles, ragged = part
            mine = tiles if two else (tiles + 1 - g) // 2
            for i in range(mine):
                t = self.tile_of(two, g, i)
                yield self.s_full[g], s
                s += 1
                if self.S[g] != (n, t):
                    raise Fault("scores of another tile")
                yield None
                self.S[g], self.P[g] = None, (n, t)  # the weights take the scores' place
                if ragged and t == tiles - 1:
                    at = self.base_of(n) + self.v_at(two, t, tiles)
                    yield self.kv_full[at % self.slots], at // self.slots
                    if self.ring[at % self.slots] != (n, t, "v"):
                        raise Fault("another tile's values cleared")
                yield None
                self.p_full[g].arrive(4)
                yield None
            used = [x for x in range(2) if (tiles if two else (tiles + 1 - x) // 2)]
            for x in [g] if two else used:
                yield self.o_full[x], o[x]
                o[x] += 1
            if not two:
                self.meet[0].arrive(4)
                yield self.meet[0], meets
            for x in [g] if two else used:
                if self.O[x] != (n, sum(1 for t in range(tiles) if two or t % 2 == x)):
                    raise Fault("an output that is not the part's")
                self.O_readers[x] -= 1
                yield None
            if two:
                if self.mistake == "a wait for the other group's products":
                    yield self.o_full[1 - g], o[1 - g]
                o[1 - g] += 1
            elif self.mistake != "no meeting at a part's end":
                self.meet[1].arrive(4)
                yield self.meet[1], meets
                meets += 1
            else:
                self.meet[1].arrive(4)
                meets += 1
            n += 1

    # ---- copies and products ----
    def land(self):
        kind, place, what = self.copies.pop(self.rng.randrange(len(self.copies)))
        if kind == "q":
            self.q[place] = what
            self.q_full[place].arrive()
        else:
            self.ring[place] = what
            self.kv_full[place].arrive()

    def product(self):
        op = self.pipe.pop(0)
        if op[0] == "arrive":
            op[1].arrive()
        elif op[0] == "qk":
            _, g, n, t, i = op
            slot = i % self.slots
            if self.ring[slot] != (n, t, "k") or self.q[g] != n:
                raise Fault("a product of other keys or queries")
            if self.S[g] is not None or self.P[g] is not None:
                raise Fault("scores over weights that are not used yet")
            self.ring_readers[slot] -= 1
            self.q_readers[g] -= 1
            self.S[g] = (n, t)
        else:
            _, g, n, t, i, first = op
            slot = i % self.slots
            if self.ring[slot] != (n, t, "v") or self.P[g] != (n, t):
                raise Fault("a product of other values or weights")
            self.ring_readers[slot] -= 1
            self.P[g] = None
            if first:
                if self.O_readers[g]:
                    raise Fault("an output replaced before it was read")
                self.O[g], self.O_readers[g] = (n, 1), 1 if self.parts[n][0] else 2
            else:
                self.O[g] = (n, self.O[g][1] + 1)

    def run(self):
        """None, or what went wrong."""
        actors = [self.scheduler(), self.issuer(), self.loader(False), self.loader(True), self.group(0), self.group(1)]
        waits = [None] * len(actors)  # (barrier, phase)
        # some actors are slow for a while, so that others run far ahead
        while True:
            ready = []
            for i, a in enumerate(actors):
                if a is not None and (waits[i] is None or waits[i][0].done % 2 != waits[i][1] % 2):
                    ready.append(i)
            choices = ready + ["land"] * bool(self.copies) + ["product"] * bool(self.pipe)
            if not choices:
                return None if all(a is None for a in actors) else "a wait that never ends"
            if self.rng.random() < 0.05:
                self.slow = self.rng.choice([0, 1, 2, 3, 4, 5, "land", "product", None])
            fast = [c for c in choices if c != getattr(self, "slow", None)] or choices
            pick = self.rng.choice(fast)
            try:
                if pick == "land":
                    self.land()
                elif pick == "product":
                    self.product()
                else:
                    if waits[pick] is not None and waits[pick][0].done != waits[pick][1] + 1:
                        return "a wait that passes on another phase"
                    try:
                        waits[pick] = next(actors[pick])
                    except StopIteration:
                        actors[pick] = waits[pick] = None
            except Fault as e:
                return str(e)


def _parts(rng):
    kind = rng.random()
    n = rng.randint(1, 14)
    if kind < 0.3:  # short parts, one after the other
        return [(rng.random() < 0.5, rng.randint(1, 2), rng.random() < 0.3) for _ in range(n)]
    return [(rng.random() < 0.5, rng.choice([1, 1, 2, 3, 4, 7]), rng.random() < 0.3) for _ in range(n)]


def _first_fault(mistake, slots, tries, seed=0):
    for i in range(tries):
        rng = random.Random(f"{seed} {mistake} {slots} {i}")
        parts = _parts(rng)
        fault = Cta(parts, slots, mistake, rng).run()
        if fault is not None:
            return fault, parts, i
    return None


@pytest.mark.parametrize("slots", [5, 10])  # head dims 128 and 64
def test_no_schedule_goes_wrong(slots):
    assert _first_fault(None, slots, 1500) is None


@pytest.mark.parametrize("mistake,slots,found", [
    ("a wait for the other group's products", 5, {"a wait that never ends"}),
    ("no wait for a free slot", 5, {"a ring slot filled before its last reader was done", "more arrivals than a phase takes"}),
    ("no meeting at a part's end", 5, {"an output replaced before it was read", "a wait that passes on another phase",
                                       "a wait that never ends", "more arrivals than a phase takes"}),
])
def test_planted_mistakes_are_found(mistake, slots, found):
    fault = _first_fault(mistake, slots, 1500)
    assert fault is not None and fault[0] in found, fault


def test_a_ring_of_two_slots_is_too_short():
    """The loaders' waits count on five slots or more; two cannot hold the tiles
    that a part's first products need."""
    assert _first_fault(None, 2, 300) is not None
