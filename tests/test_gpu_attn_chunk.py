"""gbe_attn_chunk on the GPU against the definition in 64 bits: types, head
layouts, page sizes, new and cached counts around every border, windows,
poisoned memory around the live tokens, splits, batch invariance, bad pages,
streams and graphs."""
import math

import pytest
import torch

import attn_ref
import chunk_ref
import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import filled, i32, rand, starts_of

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
KINDS = [(F32, F32), (F32, F8), (BF, BF), (BF, F8)]
# (new, cached) of each sequence: nothing new, nothing cached, single tokens, borders of tiles and of blocks of keys
PAIRS = [(1, 0), (0, 40), (1, 63), (2, 62), (7, 121), (8, 120), (9, 119), (31, 1), (32, 0), (33, 95), (64, 64), (65, 200),
         (3, 300), (128, 0), (129, 127), (1, 128)]


def _check(q, cache, starts, table, lens, scale, window=0, sinks=0, what=""):
    out = torch.full_like(q, 9.0)
    n = gbe.attn_chunk_workspace(len(lens), q.shape[0], q.shape[1], cache, table.shape[1], window, sinks)
    room = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")  # (as NaN as anything)
    gbe.gbe_attn_chunk(q, out, cache, i32(starts), table, i32(lens), scale, window, sinks, room[:n] if n else None)
    want, tol, written = chunk_ref.chunk(q, cache, starts, table, lens, scale, window, sinks, q.dtype == BF)
    attn_ref.assert_within(out[written], want[written], tol[written], what)
    assert bool((out[~written] == 9.0).all()), "rows of no sequence are left as they were"
    assert bool((room[n:] == 0xA5).all()), "the workspace's end"
    return out


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 5), (130, 64)])
@pytest.mark.parametrize("Hq,H,D,P", [(4, 1, 64, 16), (8, 2, 128, 64), (3, 3, 128, 48), (2, 2, 8, 1), (7, 1, 72, 100),
                                      (16, 2, 80, 32), (14, 2, 256, 16), (40, 1, 96, 64), (24, 2, 136, 128)])
def test_borders(dtype, kind, window, sinks, Hq, H, D, P):
    new, lens = [a for a, _ in PAIRS], [a + b for a, b in PAIRS]
    cache, table = filled(lens, P, H, D, dtype, kind, 21)
    starts = starts_of(new, 2)
    q = rand((starts[-1] + 3, Hq, D), dtype, 23)
    q[:2] = q[starts[-1]:] = float("nan")
    _check(q, cache, starts, table, lens, 1.0 / math.sqrt(D), window, sinks)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("new,cached,Hq,H,D,P", [([5], [5000], 8, 1, 128, 64), ([33], [20000], 4, 2, 64, 128),
                                                 ([1, 70, 4], [4097, 2500, 9000], 6, 2, 64, 16),
                                                 ([300], [2300], 3, 1, 128, 32), ([2, 0, 17], [8000, 8000, 1], 32, 8, 128, 64)])
def test_long_walks_are_split_and_joined(dtype, kind, new, cached, Hq, H, D, P):
    lens = [a + b for a, b in zip(new, cached)]
    cache, table = filled(lens, P, H, D, dtype, kind, 31)
    q = rand((sum(new), Hq, D), dtype, 33, 2.0)
    _check(q, cache, starts_of(new), table, lens, 1.0 / math.sqrt(D))
    _check(q, cache, starts_of(new), table, lens, 1.0 / math.sqrt(D), 2111, 130, "window")


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_batch_invariance(dtype, kind):
    """A sequence alone, in a batch, and among 400 others: the same bits."""
    new, cached, Hq, H, D, P = [20, 0, 1, 133, 6], [1500, 9, 4000, 0, 9000], 8, 2, 128, 64
    lens = [a + b for a, b in zip(new, cached)]
    cache, table = filled(lens, P, H, D, dtype, kind, 51)
    starts = starts_of(new)
    q = rand((starts[-1], Hq, D), dtype, 53)
    whole = gbe.attn_chunk(q, cache, i32(starts), table, i32(lens), 0.1)
    assert torch.equal(gbe.attn_chunk(q, cache, i32(starts), table, i32(lens), 0.1), whole), "the same bits every time"
    for b in range(len(new)):
        a, z = starts[b], starts[b + 1]
        if z > a:
            one = gbe.attn_chunk(q[a:z], cache, i32([0, z - a]), table[b:b + 1], i32(lens[b:b + 1]), 0.1)
            assert torch.equal(one, whole[a:z]), b
    many = [b % 5 for b in range(400)]
    rows = torch.cat([torch.arange(starts[b], starts[b + 1]) for b in many]).cuda()
    big = gbe.attn_chunk(q[rows], cache, i32(starts_of([new[b] for b in many])), table[many], i32([lens[b] for b in many]),
                         0.1)
    assert torch.equal(big, whole[rows])


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_bad_pages_lengths_out_of_range_and_rows_that_see_nothing(dtype, kind):
    P, H, D, Hq = 16, 2, 64, 4
    new, lens = [10, 10, 30, 5, 12, 20], [40, 160, 160, 100, 33, 90]
    cache, table = filled(lens, P, H, D, dtype, kind, 61, spare_cols=1)
    table[2, 3] = -1
    table[2, 9] = cache.shape[0]          # the last rows' own page
    table[3, :] = torch.tensor([-5, 2 ** 31 - 1] * 6, dtype=torch.int32)[:table.shape[1]]
    starts = starts_of(new)
    q = rand((starts[-1], Hq, D), dtype, 63)
    asked = [-3, 160, 160, 100, 7, 90]    # no tokens; fewer than the rows
    out = _check(q, cache, starts, table, asked, 0.125)
    assert bool((out[:10] == 0).all()) and bool((out[starts[3]:starts[4]] == 0).all())
    assert bool((out[starts[4]:starts[4] + 5] == 0).all()), "rows at places below 0"
    # a length above the table's capacity counts as that
    full = table[1:2, :10].contiguous()
    a = gbe.attn_chunk(q[10:20], cache, i32([0, 10]), full, i32([10 ** 6]), 0.125)
    assert torch.equal(a, gbe.attn_chunk(q[10:20], cache, i32([0, 10]), full, i32([160]), 0.125))


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_sharp_flat_and_signed_logits(dtype, kind):
    new, cached, Hq, H, D, P = [40, 3], [700, 130], 8, 2, 64, 16
    lens = [a + b for a, b in zip(new, cached)]
    cache, table = filled(lens, P, H, D, dtype, kind, 41)
    for std, scale in ((30.0, 0.125), (0.0, 0.125), (1.0, 0.0), (1.0, -0.5), (1e-3, 1e-6)):
        _check(rand((43, Hq, D), dtype, 43, std), cache, starts_of(new), table, lens, scale,
               what=f"std {std} scale {scale}")


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF, BF)])
def test_what_no_row_sees_stays_there(dtype, kind):
    """Infinities and NaN behind a row's place and ahead of its window, in the same block of keys as its own.  On the
    tensor cores such a row is computed again without its weights' rounding: other bits, the same bounds."""
    P, H, D, Hq, n, m, window, sinks = 16, 1, 64, 4, 260, 40, 30, 2
    cache, table = filled([n], P, H, D, dtype, kind, 71)
    q = rand((m, Hq, D), dtype, 73)

    def at(t): return int(table[0, t // P]), 0, t % P

    clean = gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.2, window, sinks)
    open_ = gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.2)
    bounds = {w: chunk_ref.chunk(q, cache, [0, m], table, [n], 0.2, w, sinks, dtype == BF) for w in (window, 0)}
    for t in (n - 1, n - 20, n - m, 200, 120, 1):
        keep = cache.v[at(t)].clone(), cache.k[at(t)].clone()
        for value in (float("nan"), float("inf")):
            cache.v[at(t)] = value
            p = torch.arange(n - m, n, device="cuda")
            for got, ref, w in ((gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.2, window, sinks), clean, window),
                                (gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.2), open_, 0)):
                hit = (t <= p) & ((p - t < w) | (t < sinks)) if w else t <= p
                attn_ref.assert_within(got[~hit], bounds[w][0][~hit], bounds[w][1][~hit], (t, w))
                assert dtype == BF or torch.equal(got[~hit], ref[~hit]), (t, w)
                assert not bool(got[hit].isfinite().any()), (t, w)
        cache.v[at(t)], cache.k[at(t)] = keep


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF, BF)])
def test_infinities_and_nan_in_attended_places(dtype, kind):
    P, H, D, Hq, n, m = 16, 1, 64, 3, 200, 2
    q = rand((m, Hq, D), dtype, 73).abs() + 0.5

    def run(t, which, value):
        cache, table = filled([n], P, H, D, dtype, kind, 72)
        getattr(cache, which)[int(table[0, t // P]), 0, t % P] = value
        return gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.1), cache, table

    out, _, _ = run(50, "v", float("inf"))
    assert bool((out == float("inf")).all())
    out, _, _ = run(50, "k", float("nan"))
    assert bool(out.isnan().all())
    out, cache, table = run(50, "k", float("-inf"))  # a logit of -inf weighs nothing
    cache.k[int(table[0, 50 // P]), 0, 50 % P] = 0.0
    other = table.clone()
    k, v = (torch.cat([attn_ref.values(cache, w)[int(table[0, t // P]), 0, t % P][None] for t in range(n)]) for w in "kv")
    keep = torch.arange(n, device="cuda") != 50
    ok = chunk_ref.sees([n - 2, n - 1], n, 0, 0, "cuda")[:, keep].repeat_interleave(Hq, 0)
    want, tol = chunk_ref.masked(q.reshape(-1, D).double(), k[keep], v[keep], ok, 0.1, dtype == BF,
                                 2.0 ** -8 if dtype == BF else attn_ref.U)
    attn_ref.assert_within(out.reshape(-1, D), want, tol)
    assert torch.equal(other, table)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_strided_rows_off_the_grid_and_halves_of_one_buffer(dtype, kind):
    new, cached, Hq, H, D, P = [9, 40], [100, 60], 4, 2, 64, 16
    lens = [a + b for a, b in zip(new, cached)]
    starts = starts_of(new)
    cache, table = filled(lens, P, H, D, dtype, kind, 81)
    both = torch.stack([cache.k, cache.v], 1)  # [pages, 2, H, P, D]
    halves = gbe.KvCache(both[:, 0], both[:, 1], cache.k_scale, cache.v_scale)
    wide = rand((starts[-1], (Hq + 2) * D + 1), dtype, 83)
    for shift in (0, 1):
        q = wide[:, shift:shift + Hq * D].unflatten(1, (Hq, D))
        out = torch.full((starts[-1], (Hq + 1) * D + shift), 5.0, dtype=dtype, device="cuda")
        view = out[:, shift:shift + Hq * D].unflatten(1, (Hq, D))
        gbe.gbe_attn_chunk(q, view, halves, i32(starts), table, i32(lens), 0.1)
        want, tol, _ = chunk_ref.chunk(q, cache, starts, table, lens, 0.1, rounded=dtype == BF)
        attn_ref.assert_within(view, want, tol, f"shift {shift}")
        assert bool((out[:, :shift] == 5.0).all()) and bool((out[:, shift + Hq * D:] == 5.0).all())


def test_against_decode_and_prompt():
    """One new token each is decode, a prompt with nothing ahead of it is the prompt, within both bounds."""
    Hq, H, D, P = 8, 2, 128, 64
    for dtype, kind in KINDS:
        lens = [300, 64, 1, 2000]
        cache, table = filled(lens, P, H, D, dtype, kind, 91)
        q = rand((4, Hq, D), dtype, 92)
        a = gbe.attn_chunk(q, cache, i32([0, 1, 2, 3, 4]), table, i32(lens), 0.1)
        b = gbe.attn_decode(q, cache, table, i32(lens), 0.1)
        _, tol, _ = chunk_ref.chunk(q, cache, [0, 1, 2, 3, 4], table, lens, 0.1, rounded=dtype == BF)
        attn_ref.assert_within(a, b.double(), 2 * tol)
    for dtype in (F32, BF):
        n = 150
        q, k, v = rand((n, Hq, D), dtype, 93), rand((n, H, D), dtype, 94), rand((n, H, D), dtype, 95)
        cache, table = gbe.kv_cache(3, H, P, D, dtype), i32([[2, 0, 1]])
        slots = i32([[2, 0, 1][t // P] * P + t % P for t in range(n)])
        gbe.gbe_kv_write(k, v, slots, cache)
        a = gbe.attn_chunk(q, cache, i32([0, n]), table, i32([n]), 0.1)
        _, tol, _ = chunk_ref.chunk(q, cache, [0, n], table, [n], 0.1, rounded=dtype == BF)
        attn_ref.assert_within(a, gbe.attn_prompt(q, k, v, i32([0, n]), 0.1).double(), 2 * tol)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_captured_with_counts_that_change_and_streams(dtype, kind):
    """A graph of one call, replayed with other starts, lengths and tables; and the call on another stream."""
    Hq, H, D, P = 8, 2, 128, 16
    cache, table = filled([3000, 90, 500], P, H, D, dtype, kind, 101)
    q = rand((60, Hq, D), dtype, 102)
    starts, lens = i32([0, 20, 40, 60]), i32([3000, 90, 500])
    room = torch.empty(max(1, gbe.attn_chunk_workspace(3, 60, Hq, cache, table.shape[1])), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gbe.gbe_attn_chunk(q, out, cache, starts, table, lens, 0.1, 0, 0, room)
    for s, n in (([0, 20, 40, 60], [3000, 90, 500]), ([0, 1, 1, 60], [2999, 0, 499]), ([5, 50, 55, 58], [100, 90, 3])):
        starts.copy_(i32(s))
        lens.copy_(i32(n))
        out.zero_()
        graph.replay()
        want = torch.zeros_like(q)
        gbe.gbe_attn_chunk(q, want, cache, i32(s), table, i32(n), 0.1, 0, 0, room)
        assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = gbe.attn_chunk(q, cache, starts, table, lens, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[5:58], want[5:58])


def test_pinned_host_memory():
    Hq, H, D, P = 4, 2, 64, 16
    for dtype, kind in KINDS:
        cache, table = filled([100], P, H, D, dtype, kind, 111)
        host = gbe.KvCache(*(None if t is None else t.cpu().pin_memory() for t in (cache.k, cache.v, cache.k_scale,
                                                                                  cache.v_scale)))
        q = rand((20, Hq, D), dtype, 112)
        out = torch.empty(q.shape, dtype=dtype).pin_memory()
        gbe.gbe_attn_chunk(q.cpu().pin_memory(), out, host, i32([0, 20]).cpu().pin_memory(), table.cpu().pin_memory(),
                           i32([100]).cpu().pin_memory(), 0.1)
        torch.cuda.synchronize()
        want, tol, _ = chunk_ref.chunk(q, cache, [0, 20], table, [100], 0.1, rounded=dtype == BF)
        attn_ref.assert_within(out.cuda(), want, tol)
