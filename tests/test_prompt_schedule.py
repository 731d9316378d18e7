"""The prompt kernel's schedule on the tensor cores, on the CPU: its roles (the
thread that copies, the two that issue products, the softmax of either tile) as
they wait and arrive, with mbarriers that only know the parity of a phase and
products and copies that complete late, stepped in random order.  Checked: the
one S of both tiles is not written before it has been read, operands are what
the product is to read, and every role comes to its end."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.done = 0  # phases completed

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1

    def test(self, parity):
        """What mbarrier.try_wait.parity tells: the phase of this parity is not the one that is open."""
        return (self.done & 1) != (parity & 1)


class Kernel:
    """items: (blocks of tile 0, blocks of tile 1 or 0) each; fixed: with the second tile's wait for the first tile's S."""

    def __init__(self, items, stages, rng, fixed=True):
        self.items, self.stages, self.rng, self.fixed = items, stages, rng, fixed
        self.q_full, self.q_empty = [Barrier(1), Barrier(1)], Barrier(2)
        self.kv_full, self.kv_empty = ([Barrier(n) for _ in range(stages)] for n in (1, 2))
        self.s_full, self.s_free, self.p_ready, self.o_done, self.o_free = ([Barrier(1), Barrier(1)] for _ in range(5))
        self.ring, self.q = [None] * stages, [None, None]
        self.S, self.S_read, self.P, self.O = None, True, [None, None], [None, None]
        self.late = []            # copies under way, in any order
        self.pipe = []            # products and commits, in order

    def load(self):
        g = 0
        for i, blocks in enumerate(self.items):
            for x in range(2 * max(blocks)):
                stage = g % self.stages
                yield lambda: self.kv_empty[stage].test((g // self.stages & 1) ^ 1)
                self.ring[stage] = None

                def land(stage=stage, what=(i, x)):
                    self.ring[stage] = what
                    self.kv_full[stage].arrive()
                self.late.append(land)
                g += 1
                if x == 0:
                    yield lambda: self.q_empty.test((i & 1) ^ 1)
                    for t in range(2):
                        if blocks[t]:
                            def land_q(t=t, i=i):
                                self.q[t] = i
                                self.q_full[t].arrive()
                            self.q[t] = None
                            self.late.append(land_q)

    def products(self, t):
        g, done, with_t, last_t = 0, [0, 0], 0, -1
        for i, blocks in enumerate(self.items):
            mine, theirs, most = blocks[t], blocks[t ^ 1], max(blocks)

            def loaded(x):
                return lambda: self.kv_full[x % self.stages].test(x // self.stages)

            def scores(j):
                yield loaded(g + 2 * j)
                if t == 1:
                    pt, pj = (0, j) if j < theirs else (1, j - 1)
                else:
                    pt, pj = (1, j - 1) if j - 1 < theirs else (0, j - 1)
                if pj < 0:
                    pt = last_t
                if pt >= 0:
                    if self.fixed and t == 1 and j == 0 and last_t == 0:
                        yield lambda: self.s_full[0].test(done[0])
                    yield lambda: self.s_free[pt].test(done[pt] + pj)
                stage = (g + 2 * j) % self.stages

                def product(stage=stage, j=j, i=i):
                    assert self.q[t] == i and self.ring[stage] == (i, 2 * j), "operands of S"
                    assert self.S_read, "S is overwritten unread"
                    self.S, self.S_read = (i, t, j), False
                self.pipe.append(product)
                self.pipe.append(self.s_full[t].arrive)
                self.pipe.append(self.kv_empty[stage].arrive)
                if j + 1 == mine:
                    self.pipe.append(self.q_empty.arrive)

            if mine:
                yield lambda: self.q_full[t].test(with_t)
                yield from scores(0)
            else:
                yield lambda: self.q_full[0].test(i)
                self.q_empty.arrive()
            for j in range(mine):
                if j + 1 < mine:
                    yield from scores(j + 1)
                yield loaded(g + 2 * j + 1)
                yield lambda: self.p_ready[t].test(done[t] + j)
                if j == 0 and with_t:
                    yield lambda: self.o_free[t].test(with_t - 1)
                stage = (g + 2 * j + 1) % self.stages

                def product(stage=stage, j=j, i=i):
                    assert self.ring[stage] == (i, 2 * j + 1) and self.P[t] == (i, j), "operands of O"
                    assert self.O[t] in ((i, j - 1), None) if j else self.O[t] is None, "O"
                    self.O[t] = (i, j)
                self.pipe.append(product)
                self.pipe.append(self.o_done[t].arrive)
                self.pipe.append(self.kv_empty[stage].arrive)
            for x in range(2 * mine, 2 * most):
                yield loaded(g + x)
                self.kv_empty[(g + x) % self.stages].arrive()
            g += 2 * most
            done = [done[0] + blocks[0], done[1] + blocks[1]]
            with_t += mine > 0
            last_t = 1 if blocks[1] else 0

    def softmax(self, t):
        done = 0
        for i, blocks in enumerate(self.items):
            for j in range(blocks[t]):
                yield lambda: self.s_full[t].test(done + j)
                assert self.S == (i, t, j), "the softmax reads its own S"
                self.S_read = True
                self.s_free[t].arrive()
                if j:
                    yield lambda: self.o_done[t].test(done + j - 1)
                yield lambda: True
                self.P[t] = (i, j)
                self.p_ready[t].arrive()
            if blocks[t]:
                done += blocks[t]
                yield lambda: self.o_done[t].test(done - 1)
                assert self.O[t] == (i, blocks[t] - 1)
                self.O[t] = None
                for _ in range(self.rng.choice([0, 0, 3])):
                    yield lambda: True
                self.o_free[t].arrive()
                for _ in range(self.rng.choice([0, 0, 0, 5, 40])):  # rows are written, now and then slowly
                    yield lambda: True

    def run(self):
        roles = {name: [f, None] for name, f in (("load", self.load()), ("mma0", self.products(0)),
                                                ("mma1", self.products(1)), ("soft0", self.softmax(0)),
                                                ("soft1", self.softmax(1)))}
        idle = 0
        while roles or self.late or self.pipe:
            choice = self.rng.choice(list(roles) + ["late", "pipe"])
            moved = True
            if choice == "late":
                moved = bool(self.late)
                if moved:
                    self.late.pop(self.rng.randrange(len(self.late)))()
            elif choice == "pipe":
                moved = bool(self.pipe)
                if moved:
                    self.pipe.pop(0)()
            else:
                f, wait = roles[choice]
                if wait is None or wait():
                    try:
                        roles[choice][1] = next(f)
                    except StopIteration:
                        del roles[choice]
                else:
                    moved = False
            idle = 0 if moved else idle + 1
            assert idle < 2000, f"nothing moves any more: {sorted(roles)}"


def _items(kind, rng, n=24):
    """Pairs of tiles of the sequences that one CTA takes; blocks of keys of either tile."""
    if kind == "even":      # an even number of heads: two tiles of the same rows
        return [(b, b) for b in (rng.choice([1, 1, 2, 3, 6]) for _ in range(n))]
    if kind == "odd":       # 3 heads to a kv head, one row tile: two tiles, then one
        return [(1, 1 - (i & 1)) for i in range(n)]
    if kind == "neighbours":  # one head to a kv head: row tiles 2 i and 2 i + 1, the last alone
        return [(b, rng.choice([0, b + 1])) for b in (rng.choice([1, 1, 2, 3]) for _ in range(n))]
    return [(b, rng.choice([0, 0, b, b, b + 1])) for b in (rng.choice([1, 1, 1, 2, 4]) for _ in range(n))]


@pytest.mark.parametrize("stages", [4, 8])
@pytest.mark.parametrize("kind", ["even", "odd", "neighbours", "any"])
def test_the_schedule_keeps_its_order(kind, stages):
    for seed in range(150):
        rng = random.Random(seed)
        Kernel(_items(kind, rng), stages, rng).run()


def test_without_the_wait_for_the_other_tiles_s_it_does_not():
    """A wait by parity that passes over phases takes an older phase for the one meant."""
    failed = 0
    for seed in range(150):
        rng = random.Random(seed)
        try:
            Kernel(_items("odd", rng), 4, rng, fixed=False).run()
        except AssertionError:
            failed += 1
    assert failed > 0
