"""CPU model of the chunk kernel's barrier protocol (csrc/paged_chunk.cu).

A producer, two MMA warps (one per 128-row tile) and two softmax warpgroups run
as coroutines over mbarriers with the hardware's parity waits, in random order.
Products complete in issue order per warp, some time after they are issued; a
commit arrives when everything its warp issued before it has completed.  The
model checks that no agent waits forever, that every product reads the K, V, Q,
P and S it is meant to, and that a stage is not refilled while a product still
reads it.
"""
import random

import pytest

STAGES = 4


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, count, 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0
        if self.pending == 0:
            self.pending = self.count
            self.phase += 1

    def passed(self, parity):
        return (self.phase & 1) != parity  # the phase of that parity has completed


class Model:
    def __init__(self, units, seed, skip_ahead=False, close_on_s=False):
        self.units, self.rng, self.skip_ahead = units, random.Random(seed), skip_ahead
        self.close_on_s = close_on_s
        self.q_full, self.q_empty = Bar(1), Bar(2)
        self.full, self.empty = [Bar(1) for _ in range(STAGES)], [Bar(2) for _ in range(STAGES)]
        self.s_full = [Bar(1) for _ in range(4)]
        self.p_full = [Bar(1) for _ in range(4)]
        self.o_prev, self.o_full = [Bar(1), Bar(1)], [Bar(1), Bar(1)]
        self.stage, self.q = [None] * STAGES, None
        self.s, self.o = [None] * 4, [None, None]
        self.pipe = [[], []]  # issued and not yet completed, per MMA warp
        self.done = []

    # -------------------------------------------------------------- agents
    def producer(self):
        fill = n_q = 0
        for u, (T, two) in enumerate(self.units):
            if T == 0:
                continue
            yield lambda: self.q_empty.passed((n_q & 1) ^ 1)
            assert not any(op[0] == "S" for p in self.pipe for op in p), "Q replaced under a product"
            self.q = u
            self.q_full.arrive()
            n_q += 1
            for j in range(T):
                for kind in "KV":
                    st, par = fill % STAGES, ((fill // STAGES) & 1) ^ 1
                    yield lambda: self.empty[st].passed(par)
                    assert not any(op[2] == st for p in self.pipe for op in p if op[0] in "SO"), "stage under a product"
                    self.stage[st] = (kind, u, j)
                    self.full[st].arrive()
                    fill += 1

    def mma(self, t):
        used = n_q = 0
        pp = [0, 0]

        def full(f):
            return lambda: self.full[f % STAGES].passed((f // STAGES) & 1)

        def issue_s(h, f, u, j):
            assert self.stage[f % STAGES] == ("K", u, j) and self.q == u
            self.pipe[t].append(("S", (u, j, h), f % STAGES, 2 * t + h))

        def commit(bar):
            self.pipe[t].append(("commit", bar, None, None))

        for u, (T, two) in enumerate(self.units):
            if T == 0:
                continue
            if t == 1 and not two:
                if self.skip_ahead:
                    used, n_q = used + 2 * T, n_q + 1
                    continue
                yield lambda: self.q_full.passed(n_q & 1)
                n_q += 1
                self.q_empty.arrive()
                for _ in range(2 * T):
                    yield full(used)
                    self.empty[used % STAGES].arrive()
                    used += 1
                continue
            yield lambda: self.q_full.passed(n_q & 1)
            yield full(used)
            n_q += 1
            twice = self.skip_ahead and t == 0 and not two
            for h in range(2):
                issue_s(h, used, u, 0)
                commit(self.s_full[2 * t + h])
            commit(self.empty[used % STAGES])
            if twice:
                commit(self.empty[used % STAGES])
            if T == 1:
                commit(self.q_empty)
                if twice:
                    commit(self.q_empty)
            for j in range(T):
                fv, fk, more = used + 1, used + 2, j + 1 < T
                for h in range(2):
                    b = 2 * t + h
                    yield lambda: self.p_full[b].passed(pp[h])
                    pp[h] ^= 1
                    if h == 0:
                        yield full(fv)
                    assert self.stage[fv % STAGES] == ("V", u, j)
                    assert self.s[b] == ("P", u, j, h), (self.s[b], u, j, h)
                    self.pipe[t].append(("O", (u, j, h), fv % STAGES, b))
                    if more:
                        if h == 0:
                            yield full(fk)
                        issue_s(h, fk, u, j + 1)
                    if more or self.close_on_s:
                        commit(self.s_full[b])
                    else:
                        commit((self.o_full if h else self.o_prev)[t])
                commit(self.empty[fv % STAGES])
                if twice:
                    commit(self.empty[fv % STAGES])
                if more:
                    commit(self.empty[fk % STAGES])
                    if twice:
                        commit(self.empty[fk % STAGES])
                    if j + 2 == T:
                        commit(self.q_empty)
                        if twice:
                            commit(self.q_empty)
                used += 2

    def softmax(self, t):
        sp, op = [0, 0], 0
        for u, (T, two) in enumerate(self.units):
            if t == 1 and not two:
                continue
            for i in range(2 * T):
                h, b = i & 1, 2 * t + (i & 1)
                yield lambda: self.s_full[b].passed(sp[h])
                sp[h] ^= 1
                assert self.s[b] == ("S", u, i >> 1, h), (self.s[b], u, i)
                if i and self.rng.random() < 0.3:  # the maximum moved: O must hold every step before this one
                    if i + 1 < 2 * T or self.close_on_s:
                        yield lambda: self.s_full[b ^ 1].passed(sp[h ^ 1])
                    else:
                        yield lambda: self.o_prev[t].passed(op)
                    assert self.o[t] == (u, (i - 1) >> 1, (i - 1) & 1)
                self.s[b] = ("P", u, i >> 1, h)
                self.p_full[b].arrive()
            if T:
                if self.close_on_s:
                    yield lambda: self.s_full[2 * t + 1].passed(sp[1])
                    sp = [sp[0] ^ 1, sp[1] ^ 1]
                else:
                    yield lambda: self.o_full[t].passed(op)
                    op ^= 1
                assert self.o[t] == (u, T - 1, 1)
            self.done.append((t, u))

    def complete(self, t):
        kind, what, st, b = self.pipe[t].pop(0)
        if kind == "S":
            u, j, h = what
            assert self.s[b] is None or self.s[b][0] == "used", self.s[b]
            self.s[b] = ("S", u, j, h)
        elif kind == "O":
            assert self.s[b] == ("P",) + what
            self.s[b] = ("used",)
            self.o[t] = what
        else:
            what.arrive()

    def run(self):
        agents = {"p": self.producer(), "m0": self.mma(0), "m1": self.mma(1), "s0": self.softmax(0),
                  "s1": self.softmax(1)}
        waits = {k: next(a, None) for k, a in agents.items()}
        while any(w is not None for w in waits.values()):
            ready = [k for k, w in waits.items() if w is not None and w()]
            moves = ready + [t for t in (0, 1) if self.pipe[t]]
            assert moves, "deadlock"
            m = self.rng.choice(moves)
            if m in (0, 1):
                self.complete(m)
            else:
                waits[m] = next(agents[m], None)
        want = [(t, u) for t in (0, 1) for u, (_, two) in enumerate(self.units) if t == 0 or two]
        assert sorted(self.done) == sorted(want)


def random_units(rng):
    return [(rng.choice([0, 1, 1, 2, 3, 5]), rng.random() < 0.5) for _ in range(rng.randint(1, 9))]


def test_protocol_holds_for_random_units_and_schedules():
    rng = random.Random(0)
    for seed in range(600):
        Model(random_units(rng), seed).run()


@pytest.mark.parametrize("fault", ["skip_ahead", "close_on_s"])
def test_protocol_model_catches_faults(fault):
    """Two designs that can take an older phase for the awaited one, or miss it: an MMA warp that
    passes units of one row tile without taking their stages, and a unit's end signalled on the
    barriers of S, which the next unit's S completes again."""
    rng, caught = random.Random(1), 0
    for seed in range(200):
        try:
            Model(random_units(rng), seed, **{fault: True}).run()
        except AssertionError:
            caught += 1
    assert caught > 0


@pytest.mark.parametrize("units", [[(1, True)], [(1, False)], [(0, True), (2, False), (1, True)],
                                   [(3, False), (3, False), (2, True)]])
def test_protocol_small_unit_lists(units):
    for seed in range(50):
        Model(units, seed).run()


def test_rows_make_at_most_the_row_tile_pairs_that_the_plan_allows():
    """Rising starts never exceed the limit above which the plan refuses to work: hkv (total / 2 tpt + n_seqs)."""
    rng = random.Random(4)
    for _ in range(2000):
        tpt, hkv = rng.choice([1, 2, 3, 10, 32, 128]), rng.choice([1, 2, 8])
        lens = [rng.choice([0, 1, rng.randrange(1, 600), 2 * tpt, 2 * tpt + 1]) for _ in range(rng.randrange(1, 30))]
        pairs = hkv * sum(-(-n // (2 * tpt)) for n in lens)
        assert pairs <= hkv * (sum(lens) // (2 * tpt) + len(lens))
    # starts that name the same rows again pass it, and 32-bit sums of them would wrap
    n, seqs, tpt = 1 << 24, 2048, 128
    assert seqs * -(-n // (2 * tpt)) > n // (2 * tpt) + 2 * seqs
    assert seqs * (n // 16) >= 1 << 31
