"""A model of the tree kernel's waits, on the CPU: the roles of a CTA as coroutines, its
mbarriers with their phases and parities, and a scheduler that starves roles at random.

A wait for a phase ends when the barrier's current phase has the other parity, as on the
device.  The model knows which phase is meant: a wait that ends before that phase has, or
a state in which no role can go on, is a fault."""
from __future__ import annotations

import random

import pytest

Q_SLOTS, UNITS = 2, 4


class Fault(AssertionError):
    pass


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.phase += 1
            self.pending = self.count

    def passes(self, meant):
        if (self.phase & 1) == (meant & 1):
            return False  # (meant = -1: the phase before the first)
        if self.phase <= meant:
            raise Fault(f"a wait for phase {meant} ended in phase {self.phase}")
        return True


class Cta:
    def __init__(self, units, kv_slots, mma_arrives):
        self.units = units  # (two row tiles, key tiles)
        self.kv_slots = kv_slots
        self.mma_arrives = mma_arrives
        self.q_full = [Bar(1) for _ in range(Q_SLOTS)]
        self.q_empty = [Bar(2) for _ in range(Q_SLOTS)]
        self.kv_full = [Bar(1) for _ in range(kv_slots)]
        self.kv_empty = [Bar(2) for _ in range(kv_slots)]
        self.u_full = [Bar(1) for _ in range(UNITS)]
        self.u_empty = [Bar(5) for _ in range(UNITS)]
        self.s_full = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.p_full = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.pv_done = [[Bar(1) for _ in range(2)] for _ in range(2)]
        self.o_free = Bar(2 + (2 if mma_arrives else 0))
        self.meet = Bar(2)  # the softmax warps' named barrier
        self.copies = []  # copies on their way: any may land next
        self.commits = [[], []]  # of an MMA warp: end in order

    def next_unit(self, at):
        yield self.u_full[at % UNITS], at // UNITS
        self.u_empty[at % UNITS].arrive()

    def walker(self):
        q = 0
        for at, (pair, _) in enumerate(self.units):
            yield self.u_empty[at % UNITS], at // UNITS - 1
            self.u_full[at % UNITS].arrive()
            for _ in range(2 if pair else 1):
                yield self.q_empty[q % Q_SLOTS], q // Q_SLOTS - 1
                self.copies.append(self.q_full[q % Q_SLOTS])
                q += 1

    def producer(self):
        pos = 0
        for at, (_, nt) in enumerate(self.units):
            yield from self.next_unit(at)
            for _ in range(2 * nt):
                yield self.kv_empty[pos % self.kv_slots], pos // self.kv_slots - 1
                self.copies.append(self.kv_full[pos % self.kv_slots])
                pos += 1

    def mma(self, h):
        cnt = q = kt0 = kv_at = 0
        commit = self.commits[h].append

        def wait_kv(pos):
            return self.kv_full[pos % self.kv_slots], pos // self.kv_slots

        def pass_to(pos):
            nonlocal kv_at
            while kv_at < pos:
                yield wait_kv(kv_at)
                self.kv_empty[kv_at % self.kv_slots].arrive()
                kv_at += 1

        def take(pos):
            nonlocal kv_at
            yield from pass_to(pos)
            yield wait_kv(pos)
            kv_at = pos + 1

        def pass_q(i):
            yield self.q_full[i % Q_SLOTS], i // Q_SLOTS
            self.q_empty[i % Q_SLOTS].arrive()

        for at, (pair, nt) in enumerate(self.units):
            yield from self.next_unit(at)
            tiles = nt if pair else (nt - h + 1) >> 1
            mine = q + h if pair else q

            def position(x):
                return 2 * (kt0 + ((x >> 1) if pair else 2 * (x >> 1) + h))

            def scores(x):
                half, pos = x & 1, position(x)
                if half == 0:
                    yield from take(pos)
                yield self.pv_done[h][half], cnt + (x >> 1) - 1
                commit(self.s_full[h][half])
                if half:
                    commit(self.kv_empty[pos % self.kv_slots])
                if x == 2 * tiles - 1:
                    commit(self.q_empty[mine % Q_SLOTS])

            if pair and h == 1:
                yield from pass_q(q)
            if tiles == 0:
                yield from pass_q(mine)
            else:
                yield self.q_full[mine % Q_SLOTS], mine // Q_SLOTS
                yield from scores(0)
                yield from scores(1)
            yield self.o_free, at - 1
            if self.mma_arrives:
                self.o_free.arrive()
            for x in range(2 * tiles):
                half, pos = x & 1, position(x) + 1
                if half == 0:
                    yield from take(pos)
                yield self.p_full[h][half], cnt + (x >> 1)
                commit(self.pv_done[h][half])
                if half:
                    commit(self.kv_empty[pos % self.kv_slots])
                if x + 2 < 2 * tiles:
                    yield from scores(x + 2)
            yield from pass_to(2 * (kt0 + nt))
            if pair and h == 0:
                yield from pass_q(q + 1)
            q += 2 if pair else 1
            cnt += tiles
            kt0 += nt

    def softmax(self, h):
        cnt = met = 0
        for at, (pair, nt) in enumerate(self.units):
            yield self.u_full[at % UNITS], at // UNITS
            tiles = nt if pair else (nt - h + 1) >> 1
            for x in range(2 * tiles):
                half = x & 1
                yield self.s_full[h][half], cnt + (x >> 1)
                if x > 0:  # (a raised maximum: after the product of the step before)
                    yield self.pv_done[h][half ^ 1], cnt + ((x - 1) >> 1)
                self.p_full[h][half].arrive()
            cnt += tiles
            if tiles:
                yield self.pv_done[h][1], cnt - 1
            if not pair:
                for _ in range(2):
                    self.meet.arrive()
                    yield self.meet, met
                    met += 1
            self.u_empty[at % UNITS].arrive()
            self.o_free.arrive()

    def run(self, rng):
        roles = {f.__name__ + str(a): f(*a) for f, a in (
            (self.walker, ()), (self.producer, ()), (self.mma, (0,)), (self.mma, (1,)),
            (self.softmax, (0,)), (self.softmax, (1,)))}
        waits = {}

        def step(name):
            try:
                waits[name] = next(roles[name])
            except StopIteration:
                del roles[name]
                waits.pop(name, None)

        for name in list(roles):
            step(name)
        late = {name: 10.0 ** -rng.uniform(0, 4) for name in (*roles, "copy", "commit0", "commit1")}
        while roles or self.copies or self.commits[0] or self.commits[1]:
            ready = [n for n in roles if waits[n][0].passes(waits[n][1])]
            ready += ["copy"] * bool(self.copies)
            ready += [f"commit{h}" for h in (0, 1) if self.commits[h]]
            if not ready:
                raise Fault("no role can go on: " + ", ".join(sorted(roles)))
            name = rng.choices(ready, [late[n] for n in ready])[0]
            if name == "copy":
                self.copies.pop(rng.randrange(len(self.copies))).arrive()
            elif name.startswith("commit"):
                self.commits[int(name[-1])].pop(0).arrive()
            else:
                step(name)


def some_units(rng):
    kind = rng.random()
    if kind < 0.4:  # many units of one tile, and pairs between them
        return [(rng.random() < 0.3, 1) for _ in range(12)]
    return [(rng.random() < 0.4, rng.randint(1, 7)) for _ in range(8)]


@pytest.mark.parametrize("kv_slots", [5, 8])
def test_every_wait_ends_and_none_ends_early(kv_slots):
    for seed in range(400):
        rng = random.Random(seed)
        Cta(some_units(rng), kv_slots, mma_arrives=True).run(rng)


def test_the_model_sees_a_unit_that_a_late_stream_misses():
    # without the MMA warps' own arrivals a unit can end before a stream without a tile
    # in it has looked: the model has to find the schedule in which that stream then
    # waits for good
    faults = 0
    for seed in range(400):
        rng = random.Random(seed)
        try:
            Cta(some_units(rng), 5, mma_arrives=False).run(rng)
        except Fault:
            faults += 1
    assert faults > 0
