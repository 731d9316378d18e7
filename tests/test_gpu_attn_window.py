"""gbe_attn_decode_window and gbe_attn_prompt_window on the GPU against the
definition in 64 bits: windows and sinks around every border, poisoned memory
in every place that no row sees, batch invariance, graphs."""
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
BORDERS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 300, 1100]


def _hide(cache, table, lens, window, sinks, P):
    """NaN into every cached token that no row sees."""
    for b, n in enumerate(lens):
        for t in range(sinks, n - window):
            page, row = int(table[b, t // P]), t % P
            for x in (cache.k, cache.v):
                if x.dtype == F8:
                    x.view(torch.uint8)[page, :, row] = 0x7F
                else:
                    x[page, :, row] = float("nan")


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (64, 17), (100, 0), (129, 100), (5000, 3)])
@pytest.mark.parametrize("Hq,H,D,P", [(8, 2, 128, 64), (3, 3, 64, 16), (7, 1, 72, 100), (14, 2, 136, 1)])
def test_decode_borders(dtype, kind, window, sinks, Hq, H, D, P):
    cache, table = filled(BORDERS, P, H, D, dtype, kind, 21)
    _hide(cache, table.cpu(), BORDERS, window, sinks, P)
    q = rand((len(BORDERS), Hq, D), dtype, 23)
    scale = 1.0 / math.sqrt(D)
    got = gbe.attn_decode_window(q, cache, table, i32(BORDERS), window, sinks, scale)
    want, tol = chunk_ref.decode(q, cache, table, BORDERS, scale, window, sinks)
    attn_ref.assert_within(got, want, tol)
    assert bool((got[0] == 0).all()), "a sequence of no tokens gives zeros"


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(1024, 4), (1500, 700), (4000, 0), (2, 1), (700, 5000)])
def test_decode_long_windows_are_split_and_joined(dtype, kind, window, sinks):
    lens, Hq, H, D, P = [9000, 1, 4100, 0, 6001], 8, 2, 128, 64
    cache, table = filled(lens, P, H, D, dtype, kind, 31)
    _hide(cache, table.cpu(), lens, window, sinks, P)
    q = rand((len(lens), Hq, D), dtype, 33, 2.0)
    got = gbe.attn_decode_window(q, cache, table, i32(lens), window, sinks, 0.1)
    want, tol = chunk_ref.decode(q, cache, table, lens, 0.1, window, sinks)
    attn_ref.assert_within(got, want, tol)
    for b in range(len(lens)):
        one = gbe.attn_decode_window(q[b:b + 1], cache, table[b:b + 1], i32(lens[b:b + 1]), window, sinks, 0.1)
        assert torch.equal(one[0], got[b]), "the same bits in any batch"


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_decode_no_window_and_pages_that_are_gone(dtype, kind):
    """Window 0 is gbe_attn_decode, bit for bit; pages between sinks and window may hold any number in the table."""
    lens, Hq, H, D, P = [700, 64, 1000], 4, 2, 64, 16
    cache, table = filled(lens, P, H, D, dtype, kind, 41)
    q = rand((3, Hq, D), dtype, 43)
    plain = gbe.attn_decode(q, cache, table, i32(lens))
    assert torch.equal(gbe.attn_decode_window(q, cache, table, i32(lens), 0, 9), plain)
    want = gbe.attn_decode_window(q, cache, table, i32(lens), 100, 20)
    gone = table.clone()
    for b, n in enumerate(lens):
        gone[b, 2:max(2, (n - 100) // P)] = torch.tensor(-7 if b else 2 ** 31 - 1, dtype=torch.int32)
    assert torch.equal(gbe.attn_decode_window(q, cache, gone, i32(lens), 100, 20), want)
    # a page within the window that is not in the cache takes no part
    gone[0, 40] = -1
    got = gbe.attn_decode_window(q, cache, gone, i32(lens), 100, 20)
    ref, tol = chunk_ref.decode(q, cache, gone, lens, 1 / 8, 100, 20)
    attn_ref.assert_within(got, ref, tol)


def test_decode_window_in_a_graph_with_lengths_that_grow():
    Hq, H, D, P = 8, 2, 128, 16
    cache, table = filled([400, 90], P, H, D, BF, BF, 51)
    q, lens = rand((2, Hq, D), BF, 52), i32([300, 20])
    room = torch.empty(max(1, gbe.attn_decode_workspace(2, Hq, cache, table.shape[1], 64, 4)), dtype=torch.uint8,
                       device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gbe.gbe_attn_decode_window(q, out, cache, table, lens, 64, 4, 0.1, room)
    for n in ([300, 20], [301, 64], [400, 90]):
        lens.copy_(i32(n))
        graph.replay()
        assert torch.equal(out, gbe.attn_decode_window(q, cache, table, i32(n), 64, 4, 0.1))


PROMPTS = [1, 2, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 200, 300]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 40), (64, 0), (100, 17), (129, 130), (5000, 3)])
@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (3, 3, 64), (7, 1, 72), (4, 4, 136), (40, 1, 96)])
def test_prompt_borders(dtype, window, sinks, Hq, H, D):
    starts = starts_of(PROMPTS, 3)
    T = starts[-1] + 5
    fused = rand((T, Hq + 2 * H, D), dtype, 61)
    fused[:3] = fused[starts[-1]:] = float("nan")
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
    out = torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    scale = 1.0 / math.sqrt(D)
    gbe.gbe_attn_prompt_window(q, k, v, out, i32(starts), window, sinks, scale)
    want, tol, written = chunk_ref.prompt(q, k, v, starts, scale, window, sinks, dtype == BF)
    attn_ref.assert_within(out[written], want[written], tol[written])
    assert bool((out[~written] == 9.0).all()), "rows of no sequence are left as they were"


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("window,sinks", [(1024, 4), (300, 0), (257, 600)])
def test_prompt_long(dtype, window, sinks):
    Hq, H, D, T = 4, 1, 128, 2500
    q, k, v = (rand((T, h, D), dtype, 71 + h, s) for h, s in ((Hq, 2.0), (H, 1.0), (H + 1, 1.0)))
    v = v[:, :H]
    got = gbe.attn_prompt_window(q, k, v, i32([0, T]), window, sinks, 0.1)
    want, tol, _ = chunk_ref.prompt(q, k, v, [0, T], 0.1, window, sinks, dtype == BF)
    attn_ref.assert_within(got, want, tol)
    # alone and packed: the same bits
    two = torch.cat([q[:100], q]), torch.cat([k[:100], k]), torch.cat([v[:100], v])
    both = gbe.attn_prompt_window(*two, i32([0, 100, 100 + T]), window, sinks, 0.1)
    assert torch.equal(both[100:], got)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_what_no_row_sees_stays_there(dtype):
    """Infinities and NaN ahead of a row's window, behind its place and in its neighbours.  On the tensor cores a row
    that shares a block of keys with one is computed again without its weights' rounding: other bits, the same bounds."""
    Hq, H, D, T, window, sinks = 4, 2, 64, 400, 50, 3
    q, k, v = (rand((T, h, D), dtype, 81 + i) for i, h in enumerate((Hq, H, H)))
    starts = [0, 130, 400]
    clean = gbe.attn_prompt_window(q, k, v, i32(starts), window, sinks, 0.2)
    want, tol, _ = chunk_ref.prompt(q, k, v, starts, 0.2, window, sinks, dtype == BF)
    for bad, kind in ((200, float("nan")), (60, float("inf")), (131 + 5, float("-inf"))):
        kk, vv = k.clone(), v.clone()
        vv[bad], kk[bad] = kind, float("nan")
        got = gbe.attn_prompt_window(q, kk, vv, i32(starts), window, sinks, 0.2)
        a, z = (0, 130) if bad < 130 else (130, 400)
        local = bad - a
        touched = torch.zeros(T, dtype=torch.bool, device="cuda")
        touched[bad:min(z, bad + window)] = True
        if local < sinks:
            touched[bad:z] = True
        attn_ref.assert_within(got[~touched], want[~touched], tol[~touched])
        other = torch.zeros(T, dtype=torch.bool, device="cuda")  # the sequence without one
        other[z if a == 0 else 0:T if a == 0 else a] = True
        assert torch.equal(got[other], clean[other])
        assert dtype == BF or torch.equal(got[~touched], clean[~touched])
        assert bool(got[touched].isnan().all())


def test_prompt_no_window_is_the_plain_call():
    q, k, v = rand((300, 4, 64), BF, 91), rand((300, 2, 64), BF, 92), rand((300, 2, 64), BF, 93)
    assert torch.equal(gbe.attn_prompt_window(q, k, v, i32([0, 300]), 0, 5), gbe.attn_prompt(q, k, v, i32([0, 300])))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_off_the_grid_and_large_values(dtype):
    Hq, H, D, T = 2, 1, 64, 150
    wide = rand((T, (Hq + 2 * H) * D + 1), dtype, 95, 8.0)

    def cut(first, n): return wide[:, first * D + 1:(first + n) * D + 1].unflatten(1, (n, D))

    q, k, v = cut(0, Hq), cut(Hq, H), cut(Hq + H, H)
    out = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    for scale in (0.125, 0.0, -1.0):
        gbe.gbe_attn_prompt_window(q, k, v, out, i32([0, 20, T]), 40, 2, scale)
        want, tol, _ = chunk_ref.prompt(q, k, v, [0, 20, T], scale, 40, 2, dtype == BF)
        attn_ref.assert_within(out, want, tol, f"scale {scale}")


def test_prompt_on_pinned_host_memory():
    q, k, v = (rand((90, h, 64), BF, 97 + i) for i, h in enumerate((4, 2, 2)))
    hq, hk, hv = (x.cpu().pin_memory() for x in (q, k, v))
    out = torch.empty_like(hq).pin_memory()
    gbe.gbe_attn_prompt_window(hq, hk, hv, out, i32([0, 90]).cpu().pin_memory(), 20, 1, 0.1)
    torch.cuda.synchronize()
    want, tol, _ = chunk_ref.prompt(q, k, v, [0, 90], 0.1, 20, 1, True)
    attn_ref.assert_within(out.cuda(), want, tol)
