"""All barriers of the 8-bit attention kernel as a model, random schedules over random
lists of parts: the scheduler, the issuer, the two loaders, the converters and the two
softmax groups, with copies that land at any later time and products that complete in
the order in which they were issued.

As tests/test_attend_barriers_cpu.py for the 16-bit kernel: a wait knows a phase by its
parity alone, and the model finds waits that pass on another phase, waits that never
end, and data that is replaced before its last reader is done. It is a transcription by
hand of the waits and arrivals in csrc/attend8.cuh and has to be changed along with them."""
import random

import pytest

from tests.test_attend_barriers_cpu import Barrier, Fault

QUEUE = 2  # kQ8Queue


class Cta:
    """One CTA. parts: [(over 64 rows, key tiles)]; bf16: queries are converted and the
    groups look at the values' unit."""

    def __init__(self, parts, slots, bf16, mistake, rng):
        self.parts, self.slots, self.bf16, self.mistake, self.rng = parts, slots, bf16, mistake, rng
        self.start = [sum(p[1] for p in parts[:n]) for n in range(len(parts) + 1)]
        self.tile_part = [n for n, p in enumerate(parts) for _ in range(p[1])]
        bars = lambda n, count: [Barrier(count) for _ in range(n)]  # noqa: E731
        self.raw_full, self.raw_empty = [bars(slots, 1) for _ in "kv"], [bars(slots, 4) for _ in "kv"]
        self.kc_full, self.vc_full, self.s_full, self.pv_done = bars(2, 4), bars(2, 4), bars(2, 1), bars(2, 1)
        self.p_full, self.meet, self.o_free, self.done = bars(2, 4), bars(2, 8), Barrier(8), Barrier(1)
        self.q_full, self.q_ready, self.q_empty = bars(2, 1), bars(2, 4), bars(2, 1)
        self.part_full, self.part_empty = bars(QUEUE, 1), bars(QUEUE, 15)
        self.queue = [None] * QUEUE
        self.ring = [[None] * slots for _ in "kv"]
        self.K, self.V, self.S, self.P = [None] * 2, [None] * 2, [None] * 2, [None] * 2  # what a place holds
        self.S_readers, self.V_info = [0, 0], [None, None]
        self.exps = [None] * 4
        self.Q, self.O, self.O_readers = [None, None], [None, None], [0, 0]
        self.copies, self.pipe = [], []

    def wide(self, j):
        return self.parts[self.tile_part[j]][0]

    def owners(self, j):
        return (0, 1) if self.wide(j) else (j % 2,)

    def part(self, n, weight, before=None):
        yield self.part_full[n % QUEUE], n // QUEUE
        if self.queue[n % QUEUE] != n:
            raise Fault("a part replaced before all have read it")
        if n < len(self.parts) and before is not None:
            yield before
        self.part_empty[n % QUEUE].arrive(weight)
        yield None
        return None if n == len(self.parts) else self.parts[n]

    def scheduler(self):
        for n in range(len(self.parts) + 1):
            if n >= QUEUE:
                yield self.part_empty[n % QUEUE], n // QUEUE - 1
            self.queue[n % QUEUE] = n
            self.part_full[n % QUEUE].arrive()
            yield None
            if n < len(self.parts):
                if n >= 2:
                    yield self.q_empty[n % 2], n // 2 - 1
                self.Q[n % 2] = None
                self.copies.append(("q", n))
                yield None

    def loader(self, v):
        n = 0
        while (yield from self.part(n, 1)) is not None:
            for j in range(self.start[n], self.start[n + 1]):
                slot, use = j % self.slots, j // self.slots
                if use > 0:
                    yield self.raw_empty[v][slot], use - 1
                self.ring[v][slot] = None
                self.copies.append(("kv", v, j))
                yield None
            n += 1

    def converters(self):
        n = 0
        while (yield from self.part(n, 4)) is not None:
            if self.bf16:
                yield self.q_full[n % 2], n // 2
                if self.Q[n % 2] != n:
                    raise Fault("queries of another part converted")
                yield None
                self.q_ready[n % 2].arrive(4)
            for j in range(self.start[n], self.start[n + 1]):
                b, slot, use = j % 2, j % self.slots, j // self.slots
                yield self.raw_full[0][slot], use
                if self.ring[0][slot] != j:
                    raise Fault("another tile's keys converted")
                if j >= 2:
                    yield self.s_full[b], j // 2 - 1
                if self.K[b] is not None:
                    raise Fault("keys replaced before their product")
                self.K[b], self.exps[j % 4] = j, j
                yield None
                self.kc_full[b].arrive(4)
                self.raw_empty[0][slot].arrive(4)
                yield None
                yield self.raw_full[1][slot], use
                if j >= 2 and self.mistake != "values do not wait for their product":
                    yield self.pv_done[b], j // 2 - 1
                if self.ring[1][slot] != j:
                    raise Fault("another tile's values converted")
                if self.V[b] is not None:
                    raise Fault("values replaced before their product")
                self.V[b] = self.V_info[b] = j
                yield None
                self.vc_full[b].arrive(4)
                self.raw_empty[1][slot].arrive(4)
                yield None
            n += 1

    def issuer(self):
        n, ps = 0, [0, 0]
        while (yield from self.part(n, 1)) is not None:
            yield (self.q_ready if self.bf16 else self.q_full)[n % 2], n // 2
            first, end = self.start[n], self.start[n + 1]

            def qk(j):
                yield self.kc_full[j % 2], j // 2
                self.pipe.append(("qk", j))
                self.pipe.append(("arrive", self.s_full[j % 2]))
                if j + 1 == end:
                    self.pipe.append(("arrive", self.q_empty[n % 2]))
                yield None

            for j in range(first, min(first + 2, end)):
                yield from qk(j)
            for j in range(first, end):
                yield self.vc_full[j % 2], j // 2
                if j == first and n > 0 and self.mistake != "outputs are not waited for":
                    yield self.o_free, n - 1
                for g in self.owners(j):
                    yield self.p_full[g], ps[g]
                    ps[g] += 1
                if self.V_info[j % 2] != j:
                    raise Fault("another tile's type")
                self.pipe.append(("pv", j))
                self.pipe.append(("arrive", self.pv_done[j % 2]))
                yield None
                if j + 2 < end:
                    yield from qk(j + 2)
            n += 1
        self.pipe.append(("arrive", self.done))
        yield self.done, 0

    def group(self, g):
        n, last, meets = 0, None, 0  # last: the last tile whose weights this group wrote
        while True:
            before = (self.q_ready[n % 2], n // 2) if self.bf16 and self.mistake != "queries waited for late" else None
            part = yield from self.part(n, 4, before)
            if part is None:
                return
            if self.bf16 and self.mistake == "queries waited for late":
                yield self.q_ready[n % 2], n // 2
            mine = [j for j in range(self.start[n], self.start[n + 1]) if g in self.owners(j)]
            for j in mine:
                b = j % 2
                yield self.s_full[b], j // 2
                if self.S[b] != j or self.exps[j % 4] != j:
                    raise Fault("scores or scales of another tile")
                yield None
                if self.bf16:
                    yield self.vc_full[b], j // 2
                    if self.V_info[b] != j:
                        raise Fault("another tile's unit")
                if last is not None and (self.mistake != "weights over weights" or self.rng.random() < 0.5):
                    yield self.pv_done[last % 2], last // 2
                if self.P[g] is not None:
                    raise Fault("weights replaced before their product")
                yield None
                if self.S[b] != j or self.exps[j % 4] != j:  # read again where a reference rose
                    raise Fault("scores or scales of another tile, read again")
                self.P[g], last = j, j
                self.S_readers[b] -= 1
                if self.S_readers[b] == 0:
                    self.S[b] = None
                yield None
                self.p_full[g].arrive(4)
                yield None
            if last is not None:
                yield self.pv_done[last % 2], last // 2
            if not part[0]:
                self.meet[0].arrive(4)
                yield self.meet[0], meets
            tiles = range(self.start[n], self.start[n + 1])
            for x in ([g] if part[0] else [0, 1]):
                own = [j for j in tiles if x in self.owners(j)]
                if not own:
                    continue
                if self.O[x] != (n, len(own)):
                    raise Fault("an output that is not the part's")
                self.O_readers[x] -= 1
                yield None
            if not part[0]:
                self.meet[1].arrive(4)
                if self.mistake != "outputs are not waited for":
                    yield self.meet[1], meets
                meets += 1
            self.o_free.arrive(4)
            yield None
            n += 1

    def land(self):
        what = self.copies.pop(self.rng.randrange(len(self.copies)))
        if what[0] == "q":
            self.Q[what[1] % 2] = what[1]
            self.q_full[what[1] % 2].arrive()
        else:
            _, v, j = what
            self.ring[v][j % self.slots] = j
            self.raw_full[v][j % self.slots].arrive()

    def product(self):
        op = self.pipe.pop(0)
        if op[0] == "arrive":
            op[1].arrive()
            return
        kind, j = op
        b, n = j % 2, self.tile_part[j]
        if kind == "qk":
            if self.K[b] != j or self.Q[n % 2] != n:
                raise Fault("a product of other keys or queries")
            if self.S[b] is not None:
                raise Fault("scores over scores that are not read yet")
            self.K[b], self.S[b], self.S_readers[b] = None, j, len(self.owners(j))
        else:
            if self.V[b] != j or any(self.P[g] != j for g in self.owners(j)):
                raise Fault("a product of other values or weights")
            self.V[b] = None
            for g in self.owners(j):
                self.P[g] = None
                if self.O[g] is None or self.O[g][0] != n:
                    if self.O_readers[g]:
                        raise Fault("an output replaced before it was read")
                    self.O[g], self.O_readers[g] = (n, 1), 1 if self.parts[n][0] else 2
                else:
                    self.O[g] = (n, self.O[g][1] + 1)

    def run(self):
        """None, or what went wrong."""
        actors = [self.scheduler(), self.issuer(), self.loader(0), self.loader(1), self.converters(), self.group(0), self.group(1)]
        waits = [None] * len(actors)
        slow = None
        while True:
            ready = [i for i, a in enumerate(actors) if a is not None and (waits[i] is None or waits[i][0].done % 2 != waits[i][1] % 2)]
            choices = ready + ["land"] * bool(self.copies) + ["product"] * bool(self.pipe)
            if not choices:
                return None if all(a is None for a in actors) else "a wait that never ends"
            if self.rng.random() < 0.05:  # some actors are slow for a while, so that others run far ahead
                slow = self.rng.choice([*range(len(actors)), "land", "product", None])
            pick = self.rng.choice([c for c in choices if c != slow] or choices)
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


def _first_fault(mistake, slots, bf16, tries):
    for i in range(tries):
        rng = random.Random(f"{mistake} {slots} {bf16} {i}")
        lengths = [1, 1, 2] if rng.random() < 0.4 else [1, 1, 2, 3, 4, 7]
        parts = [(rng.random() < 0.5, rng.choice(lengths)) for _ in range(rng.randint(1, 14))]
        fault = Cta(parts, slots, bf16, mistake, rng).run()
        if fault is not None:
            return fault, parts, i
    return None


@pytest.mark.parametrize("slots", [2, 4])  # head dims 128 and 64
@pytest.mark.parametrize("bf16", [True, False])
def test_no_schedule_goes_wrong(slots, bf16):
    assert _first_fault(None, slots, bf16, 1000) is None


@pytest.mark.parametrize("mistake", ["values do not wait for their product", "outputs are not waited for", "weights over weights",
                                     "queries waited for late"])
def test_planted_mistakes_are_found(mistake):
    # (outputs: neither by the issuer nor at a narrow part's end)
    assert _first_fault(mistake, 2, True, 1500) is not None
