"""Attention where infinities and NaN of v lie in keys that a row sees and, at the
same time, in keys that it does not: the entry is what the seen ones make it."""
import pytest
import torch

import attn_ref
import chunk_ref
import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import filled, i32, rand

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
# (what a key that every row sees holds, what one that a row does not see holds)
PAIRS = [(INF, NAN), (INF, INF), (INF, -INF), (-INF, NAN), (-INF, INF), (NAN, INF), (None, INF), (None, NAN)]


def _check(got, want, tol, first, entry, odd, window, sinks, what):
    """Rows [m, Hq, D] at places first, first + 1, ...: `odd` is [(key, value)] of entry `entry`, the other values are
    finite; a row is what the values that it sees make it."""
    n = first + got.shape[0]
    ok = chunk_ref.sees(range(first, n), n, window, sinks, got.device)
    met = torch.zeros(got.shape[0], dtype=torch.float64, device=got.device)  # 0, or the sum of what is met
    for key, value in odd:
        met = torch.where(ok[:, key], met + value, met)
    met, new = met[:, None].expand(got.shape[:2]), got[..., entry]
    odd_rows = met != 0  # (NaN too)
    assert bool((new.isnan() == met.isnan()).all()), what
    assert bool((new == met)[met.isinf()].all()), what
    plain = torch.ones_like(got, dtype=torch.bool)
    plain[..., entry] = ~odd_rows
    attn_ref.assert_within(got[plain], want[plain], tol[plain], what)


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF, BF)])
@pytest.mark.parametrize("n,m,window,sinks,D", [(200, 30, 0, 0, 64), (300, 40, 50, 3, 128), (150, 7, 20, 0, 72),
                                                (200, 30, 0, 0, 136), (3000, 30, 0, 0, 64)])
def test_chunk(dtype, kind, n, m, window, sinks, D):
    P, H, Hq, entry = 16, 2, 4, 5
    cache, table = filled([n], P, H, D, dtype, kind, 3)
    q = rand((m, Hq, D), dtype, 4)
    want, tol, _ = chunk_ref.chunk(q, cache, [0, m], table, [n], 0.1, window, sinks, dtype == BF)
    at = lambda t: (int(table[0, t // P]), slice(None), t % P, entry)  # noqa: E731
    for seen, hidden in PAIRS:
        for a, b in ((n - m, n - 1), (n - m - 3, n - 2), (0, n - 1)):  # (0 may be a sink, or behind the window)
            keep = cache.v[at(a)].clone(), cache.v[at(b)].clone()
            odd = [(b, hidden)]
            cache.v[at(b)] = hidden
            if seen is not None:
                cache.v[at(a)] = seen
                odd.append((a, seen))
            got = gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.1, window, sinks)
            _check(got, want, tol, n - m, entry, odd, window, sinks, (seen, hidden, a, b))
            cache.v[at(a)], cache.v[at(b)] = keep


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,window,sinks,D", [(150, 30, 0, 64), (300, 40, 5, 128), (200, 129, 2, 72), (150, 30, 2, 136)])
def test_prompt_window(dtype, n, window, sinks, D):
    H, Hq, entry = 2, 4, 9
    q, k, v = (rand((n, h, D), dtype, 7 + i) for i, h in enumerate((Hq, H, H)))
    want, tol, _ = chunk_ref.prompt(q, k, v, [0, n], 0.1, window, sinks, dtype == BF)
    for seen, hidden in PAIRS:
        for a, b in ((0, n - 1), (60, 61), (100, 70), (70, 100), (n - 2, n - 1)):
            vv, odd = v.clone(), [(b, hidden)]
            vv[b, :, entry] = hidden
            if seen is not None:
                vv[a, :, entry] = seen
                odd.append((a, seen))
            got = gbe.attn_prompt_window(q, k, vv, i32([0, n]), window, sinks, 0.1)
            _check(got, want, tol, 0, entry, odd, window, sinks, (seen, hidden, a, b))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,D", [(150, 64), (300, 128), (200, 72), (150, 136)])
def test_prompt(dtype, n, D):
    H, Hq, entry = 2, 4, 9
    q, k, v = (rand((n, h, D), dtype, 17 + i) for i, h in enumerate((Hq, H, H)))
    want, tol, _ = attn_ref.prompt(q, k, v, [0, n], 0.1, dtype == BF)
    for seen, hidden in PAIRS:
        for a, b in ((0, n - 1), (60, 61), (100, 70), (70, 100), (n - 2, n - 1)):
            vv, odd = v.clone(), [(b, hidden)]
            vv[b, :, entry] = hidden
            if seen is not None:
                vv[a, :, entry] = seen
                odd.append((a, seen))
            got = gbe.attn_prompt(q, k, vv, i32([0, n]), 0.1)
            _check(got, want, tol, 0, entry, odd, 0, 0, (seen, hidden, a, b))


def test_chunk_over_e4m3():
    """A NaN code that a row does not see, next to rows whose own keys hold none: bf16's infinities have no code."""
    P, H, Hq, D, n, m, entry = 16, 2, 4, 64, 200, 30, 5
    cache, table = filled([n], P, H, D, BF, F8, 3)
    q = rand((m, Hq, D), BF, 4)
    want, tol, _ = chunk_ref.chunk(q, cache, [0, m], table, [n], 0.1, rounded=True)
    for b in (n - 1, n - 7, n - m + 1):
        spot = int(table[0, b // P]), slice(None), b % P, entry
        codes = cache.v.view(torch.uint8)
        keep = codes[spot].clone()
        codes[spot] = 0x7F
        got = gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.1)
        _check(got, want, tol, n - m, entry, [(b, NAN)], 0, 0, b)
        codes[spot] = keep
