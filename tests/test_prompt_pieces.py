"""How the prompt kernels find a piece of work among many packed sequences, on
the CPU: the indexes that they reserve for each sequence and the search over
them, replayed; every piece of every sequence is found under exactly one index
of the grid, whatever the sequences' number and however many are empty."""
import random

import pytest


def _find(starts, T, index, count, first):
    """(sequence, piece) of an index, or None: the search of 32 places at a time; and the steps that it took."""
    n_seqs = len(starts) - 1
    at = lambda b: min(max(starts[b], 0), T)
    lo, hi, steps = 0, n_seqs, 0
    while steps == 0 or hi - lo > 1:
        step = (hi - lo + 31) // 32
        set_ = [i for i in range(32) if lo + i * step < hi
                and first(at(lo + i * step), min(lo + i * step, at(lo + i * step))) <= index]
        steps += 1
        if not set_:
            return None, steps
        lo += set_[-1] * step
        hi = min(hi, lo + step)
    s = at(lo)
    n = max(at(lo + 1) - s, 0)
    k = index - first(s, min(lo, s))
    pieces = count(n) if n > 0 else 0
    return ((lo, pieces - 1 - k) if 0 <= k < pieces else None), steps


def _rows(tile):
    """Tiles of f32 rows: (count, first, indexes of the grid)."""
    return (lambda n: -(-n // tile), lambda rows, seqs: rows // tile + seqs, lambda T, n: T // tile + min(n, T))


def _pairs(group, tile=128):
    """Pairs of tiles that share a kv head, of `group` query heads."""
    odd = group & 1
    return (lambda n: (-(-n // tile) * group + 1) // 2,
            lambda rows, seqs: ((rows // tile + seqs) * group + (seqs if odd else 0)) // 2,
            lambda T, n: ((T // tile + min(n, T)) * group + (min(n, T) if odd else 0)) // 2)


KINDS = [_rows(32), _rows(64), _pairs(1), _pairs(2), _pairs(3), _pairs(4), _pairs(7)]


def _packings():
    rng = random.Random(3)
    yield [1] * 200, 0, 0
    yield [0] * 500 + [1] + [0] * 500, 0, 3
    yield [0, 5] * 150 + [0] * 300, 2, 0
    yield [rng.randrange(0, 60) for _ in range(300)], 0, 0
    yield [rng.choice([0, 0, 1, 31, 32, 33, 127, 128, 129, 700]) for _ in range(150)], 7, 40
    yield [128] * 140, 0, 0
    yield [rng.choice([0, 0, 0, 0, 1]) for _ in range(2000)], 0, 0


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_every_piece_is_found_once(kind):
    count, first, grid = KINDS[kind]
    for lens, before, after in _packings():
        starts = [before]
        for n in lens:
            starts.append(starts[-1] + n)
        T = starts[-1] + after
        found = []
        for index in range(grid(T, len(lens))):
            got, steps = _find(starts, T, index, count, first)
            assert steps <= 5
            if got is not None:
                found.append(got)
        want = {(b, k) for b, n in enumerate(lens) if n for k in range(count(n))}
        assert len(found) == len(set(found)) and set(found) == want


def test_starts_of_any_kind_end_the_search():
    rng = random.Random(4)
    count, first, grid = _pairs(2)
    for _ in range(20):
        T = rng.randrange(1, 3000)
        starts = [rng.choice([-2 ** 31, 2 ** 31 - 1, rng.randrange(-5, T + 9)]) for _ in range(200)]
        for index in range(0, grid(T, 199), 7):
            got, steps = _find(starts, T, index, count, first)
            assert steps <= 5 and (got is None or 0 <= got[0] < 199)
