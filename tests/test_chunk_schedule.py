"""The chunk kernel's schedule on the tensor cores, on the CPU: its roles (the
warp that finds items and fetches q, the one that copies keys, those that widen
an 8-bit cache's, the two threads of products, the softmax warps of either slot)
as they wait and arrive, with mbarriers that only know the parity of a phase and
products and copies that complete late, stepped in random order.  Checked: S,
weights, O, q and the rings hold what each reader is to find, nothing is
overwritten unread, and every role comes to its end."""
import random

import pytest

from test_prompt_schedule import Barrier

TODOS, WARPS, WIDEN = 4, 2, 2  # (a slot's softmax warps and the widening ones stand for four and eight)


class Kernel:
    """items: (tiles, blocks) each; e4: over an 8-bit cache; without: a wait that is left out."""

    def __init__(self, items, e4, rng, without=""):
        self.items, self.e4, self.rng, self.without = items, e4, rng, without
        self.stages, self.raws = (3, 3) if e4 else (4, 0)
        two = lambda n: [Barrier(n), Barrier(n)]  # noqa: E731
        self.q_full, self.q_empty, self.s_full, self.o_done = two(1), two(1), two(1), two(1)
        self.s_free, self.s_last, self.p_ready, self.o_free = (two(WARPS) for _ in range(4))
        self.kv_full = [Barrier(WIDEN if e4 else 1) for _ in range(self.stages)]
        self.kv_empty = [Barrier(2) for _ in range(self.stages)]
        self.raw_full, self.raw_empty = ([Barrier(n) for _ in range(self.raws)] for n in (1, WIDEN))
        readers = 2 * WARPS + 3 + (WIDEN if e4 else 0)
        self.todo_full, self.todo_empty, self.checked = ([Barrier(n) for _ in range(TODOS)] for n in (1, readers, 1))
        self.todo = [None] * TODOS
        self.ring, self.raw, self.q = [None] * self.stages, [None] * max(self.raws, 1), [None, None]
        self.S, self.read = [None, None], [set(range(WARPS))] * 2   # S, and the warps that have read it
        self.P, self.O = [[None] * WARPS for _ in range(2)], [None, None]
        self.written = []
        self.late, self.pipe = [], [[], []]  # copies in any order; a thread's products and commits in order

    # what is waited for: item i's description
    def ready(self, i):
        return lambda: self.todo_full[i % TODOS].test(i // TODOS)

    def take(self, i):
        assert self.todo[i % TODOS][0] == i, "an item's description"
        return self.todo[i % TODOS]

    def find(self):
        tiles, last, q_item = [0, 0], 1, None

        def fetch(q_item, must):
            i, two, slot = q_item
            for t in range(2):
                if two or t == slot:
                    test = lambda t=t: self.q_empty[t].test((tiles[t] & 1) ^ 1)  # noqa: E731
                    if not must and not test():
                        return False
                    yield test
            for t in range(2):
                if two or t == slot:
                    def land(t=t):
                        self.q[t] = i
                        self.q_full[t].arrive()
                    self.q[t] = None
                    self.late.append(land)
                    tiles[t] += 1
            return True

        for i in range(len(self.items) + 1):
            more = i < len(self.items)
            two, n = (self.items[i][0] == 2, self.items[i][1]) if more else (False, 0)
            slot = -1
            if more:
                slot = 0 if two or n == 0 else last ^ 1
                if n:
                    last = 1 if two else slot
            yield lambda: self.todo_empty[i % TODOS].test((i // TODOS & 1) ^ 1)
            self.todo[i % TODOS] = (i, two, n, slot)
            self.todo_full[i % TODOS].arrive()
            if q_item is not None:
                yield from fetch(q_item, True)
                q_item = None
            if not more:
                return
            if n:
                q_item = (i, two, slot)
                if (yield from fetch(q_item, False)):
                    q_item = None
            yield lambda: True
            self.checked[i % TODOS].arrive()

    def load(self):
        g, i = 0, 0
        places, empty, full = ((self.raw, self.raw_empty, self.raw_full) if self.e4 else
                               (self.ring, self.kv_empty, self.kv_full))
        size = self.raws if self.e4 else self.stages
        while True:
            yield self.ready(i)
            _, _, n, slot = self.take(i)
            self.todo_empty[i % TODOS].arrive()
            if slot < 0:
                return
            for x in range(2 * n):
                place = g % size
                yield lambda: empty[place].test((g // size & 1) ^ 1)
                places[place] = None

                def land(place=place, what=(i, x)):
                    places[place] = what
                    full[place].arrive()
                self.late.append(land)
                g += 1
            i += 1

    def widen(self, w):
        g, i = 0, 0
        while True:
            yield self.ready(i)
            _, _, n, slot = self.take(i)
            self.todo_empty[i % TODOS].arrive()
            if slot < 0:
                return
            for x in range(2 * n):
                raw, stage = g % self.raws, g % self.stages
                yield lambda: self.raw_full[raw].test(g // self.raws)
                yield lambda: self.kv_empty[stage].test((g // self.stages & 1) ^ 1)
                assert self.raw[raw] == (i, x), "codes"
                if not isinstance(self.ring[stage], list):
                    self.ring[stage] = []
                yield lambda: True
                self.ring[stage].append(w)
                if len(self.ring[stage]) == WIDEN:
                    self.ring[stage] = (i, x)
                self.kv_full[stage].arrive()
                self.raw_empty[raw].arrive()
                g += 1
            i += 1

    def products(self, t):
        g, done, mine_so_far, every, i = 0, [0, 0], 0, 0, 0
        pipe = self.pipe[t]
        while True:
            yield self.ready(i)
            _, two, n, slot = self.take(i)
            mine = two or slot == t
            self.todo_empty[i % TODOS].arrive()
            if slot < 0:
                return
            if n == 0:
                i += 1
                continue

            def loaded(x):
                return lambda: self.kv_full[x % self.stages].test(x // self.stages)

            if not self.e4 and every and self.without != "last":
                yield lambda: self.s_last[(every - 1) & 1].test((every - 1) // 2)
            at = t if self.e4 else 0  # whose S

            def scores(j):
                yield loaded(g + 2 * j)
                if self.e4:
                    if done[t] + j:
                        yield lambda: self.o_done[t].test(done[t] + j - 1)
                else:
                    pt, pj = (t ^ 1, j if t == 1 else j - 1) if two else (t, j - 1)
                    if pj >= 0:
                        yield lambda: self.s_free[pt].test(done[pt] + pj)
                stage = (g + 2 * j) % self.stages

                def product(stage=stage, j=j, i=i):
                    assert self.q[t] == i and self.ring[stage] == (i, 2 * j), "operands of S"
                    assert len(self.read[at]) == WARPS, "S is overwritten unread"
                    assert not self.e4 or self.P[t] == [None] * WARPS, "weights are overwritten unused"
                    self.S[at], self.read[at] = (i, t, j), set()
                pipe.append(product)
                pipe.append(self.s_full[t].arrive)
                pipe.append(self.kv_empty[stage].arrive)
                if j + 1 == n:
                    pipe.append(self.q_empty[t].arrive)

            if mine:
                yield lambda: self.q_full[t].test(mine_so_far)
                if not self.e4:
                    yield from scores(0)
                for j in range(n):
                    if self.e4:
                        yield from scores(j)
                    elif j + 1 < n:
                        yield from scores(j + 1)
                    yield loaded(g + 2 * j + 1)
                    yield lambda: self.p_ready[t].test(done[t] + j)
                    if j == 0 and mine_so_far:
                        yield lambda: self.o_free[t].test(mine_so_far - 1)
                    stage = (g + 2 * j + 1) % self.stages

                    def product(stage=stage, j=j, i=i):
                        assert self.ring[stage] == (i, 2 * j + 1) and self.P[t] == [(i, j)] * WARPS, "operands of O"
                        assert self.O[t] == ((i, j - 1) if j else None), "O"
                        self.O[t], self.P[t] = (i, j), [None] * WARPS
                    pipe.append(product)
                    pipe.append(self.o_done[t].arrive)
                    pipe.append(self.kv_empty[stage].arrive)
            else:
                for x in range(2 * n):
                    yield loaded(g + x)
                    self.kv_empty[(g + x) % self.stages].arrive()
            g += 2 * n
            for s in range(2):
                done[s] += n if two or slot == s else 0
            mine_so_far += mine
            every += 1
            i += 1

    def softmax(self, t, w):
        done, every, i = 0, 0, 0
        at = t if self.e4 else 0
        while True:
            yield self.ready(i)
            _, two, n, slot = self.take(i)
            if slot < 0 or not (two or slot == t):
                self.todo_empty[i % TODOS].arrive()
                if slot < 0:
                    return
                every += n > 0
                i += 1
                continue
            yield lambda: self.checked[i % TODOS].test(i // TODOS)
            idle = self.items[i][0] == 1 and w == 1 and i % 3 == 0  # (a warp without rows)
            for j in range(n):
                yield lambda: self.s_full[t].test(done + j)
                assert self.S[at] == (i, t, j), "the softmax reads its own S"
                self.read[at] = self.read[at] | {w}
                if not self.e4:
                    self.s_free[t].arrive()
                    if j == n - 1 and (t == 1 or not two):
                        self.s_last[every & 1].arrive()
                if j and (idle or not self.e4) and self.without != "idle":
                    yield lambda: self.o_done[t].test(done + j - 1)
                yield lambda: True
                assert self.P[t][w] is None, "weights are overwritten unused"
                self.P[t][w] = (i, j)
                self.p_ready[t].arrive()
            every += n > 0
            done += n
            if n:
                yield lambda: self.o_done[t].test(done - 1)
                yield lambda: True
                assert self.O[t] == (i, n - 1), "O is the item's"
                self.written.append((i, t, w))
                if sum(x[:2] == (i, t) for x in self.written) == WARPS:
                    self.O[t] = None
                self.o_free[t].arrive()
            assert self.take(i)
            self.todo_empty[i % TODOS].arrive()
            i += 1

    def run(self):
        roles = [self.find(), self.load(), self.products(0), self.products(1)]
        roles += [self.softmax(t, w) for t in range(2) for w in range(WARPS)]
        roles += [self.widen(w) for w in range(WIDEN)] if self.e4 else []
        waits = {k: (lambda: True) for k in range(len(roles))}
        while waits or self.late or any(self.pipe):
            able = [k for k, f in waits.items() if f()]
            moves = able + ["late"] * bool(self.late) + [("pipe", t) for t in range(2) if self.pipe[t]]
            assert moves, f"stuck: {sorted(waits)}"
            k = self.rng.choice(moves)
            if k == "late":
                self.late.pop(self.rng.randrange(len(self.late)))()
            elif isinstance(k, tuple):
                self.pipe[k[1]].pop(0)()
            else:
                try:
                    waits[k] = next(roles[k])
                except StopIteration:
                    del waits[k]
        want = {(i, t, w) for i, (tiles, n) in enumerate(self.items) if n for t in range(2) for w in range(WARPS)
                if tiles == 2}
        got = {x for x in self.written if self.items[x[0]][0] == 2}
        assert got == want and len(self.written) == len(set(self.written))
        assert all(sum(x[0] == i for x in self.written) == WARPS for i, (tiles, n) in enumerate(self.items)
                   if n and tiles == 1)


@pytest.mark.parametrize("e4", [False, True])
@pytest.mark.parametrize("seed", range(60))
def test_any_order(e4, seed):
    rng = random.Random(seed)
    items = [(rng.choice([1, 1, 2]), rng.choice([0, 1, 1, 2, 3, 7])) for _ in range(rng.randrange(1, 14))]
    Kernel(items, e4, rng).run()


@pytest.mark.parametrize("e4", [False, True])
@pytest.mark.parametrize("items", [[], [(1, 0)], [(2, 0), (1, 1)], [(1, 1)] * 9, [(2, 1)] * 6, [(1, 2), (2, 3)] * 4,
                                   [(2, 1), (1, 1), (1, 1)] * 3, [(1, 0)] * 9 + [(2, 2)]])
def test_some_lists(e4, items):
    for seed in range(10):
        Kernel(items, e4, random.Random(seed)).run()


@pytest.mark.parametrize("without", ["last", "idle"])
def test_without_a_wait_it_does_not(without):
    """S after the last read of the item before; weights without rows after the product with those before."""
    failed = 0
    for seed in range(100):
        rng = random.Random(seed)
        items = [(rng.choice([1, 1, 2]), rng.choice([1, 2, 3])) for _ in range(10)]
        try:
            Kernel(items, False, rng, without).run()
        except AssertionError:
            failed += 1
    assert failed > 0
