"""The cache's operators together, as a layer calls them: a prompt in pieces,
each appended and attended to, then single tokens, drafts and a window; calls
at once, captured ones that are a process's first, many sequences, buffers past
2^31 entries, and an 8-bit cache's odd codes and scales."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

import attn_ref
import chunk_ref
import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import filled, i32, rand, starts_of

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
KINDS = [(F32, F32), (F32, F8), (BF, BF), (BF, F8)]


def _om(r):
    return (10000.0 ** (-torch.arange(r // 2, device="cuda").double() * 2 / r)).float()


def _turned(x, pos, om):
    """The half layout's rotation of x [T, H, D] in 64 bits, by the f32 angles pos * om."""
    half = om.numel()
    th = (pos[:, None].float() * om[None]).double()[:, None]
    a, b = x[..., :half].double(), x[..., half:2 * half].double()
    return torch.cat([a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos(), x[..., 2 * half:].double()], -1)


def _into(out, q, cache, starts, table, lens, scale, window=0, sinks=0):
    n = gbe.attn_chunk_workspace(len(lens), q.shape[0], q.shape[1], cache, table.shape[1], window, sinks)
    room = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    gbe.gbe_attn_chunk(q, out, cache, i32(starts), table, i32(lens), scale, window, sinks, room)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,r,P,window,sinks", [(8, 2, 128, 128, 64, 0, 0), (4, 4, 64, 32, 16, 50, 3),
                                                     (14, 2, 72, 72, 48, 130, 0)])
def test_a_layer_run(dtype, kind, Hq, H, D, r, P, window, sinks):
    """Three sequences of a batch: prompts in two pieces, a draft of four tokens, then single tokens."""
    pieces = [[100, 1, 37], [60, 200, 0], [4, 4, 4], [1, 1, 1], [1, 1, 1]]
    total = [sum(p[b] for p in pieces) for b in range(3)]
    pages = sum(-(-n // P) for n in total)
    cache = gbe.kv_cache(pages + 2, H, P, D, kind)
    table = attn_ref.make_table(total, P, pages + 2, 7, 0).cuda()
    om, lens, scale = _om(r), [0, 0, 0], 1.0 / math.sqrt(D)
    keys = torch.zeros(3, max(total), H, D, dtype=torch.float64, device="cuda")
    eps = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    for i, new in enumerate(pieces):
        T = sum(new)
        fused = rand((T + 2, Hq + 2 * H, D), dtype, 100 + i)  # two rows of padding
        q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
        at = [(b, lens[b] + t) for b in range(3) for t in range(new[b])]
        pos = i32([t for _, t in at] + [0, 0])
        slots = i32([int(table[b, t // P]) * P + t % P for b, t in at] + [-1, -1])
        lens = [n + m for n, m in zip(lens, new)]
        bad = torch.zeros(1, dtype=torch.int32, device="cuda")
        turned = torch.empty_like(fused)[:, :Hq]  # (q's token stride)
        gbe.gbe_rope_kv_write(q, turned, k, v, pos, slots, cache, om, r, 1.0, 0, None, bad)
        assert int(bad) == 0
        # two roundings of products, one of the sum, sine and cosine's own, and the storage's
        want = _turned(q[:T], pos[:T], om)
        size = q[:T].double().abs().amax(-1, keepdim=True)
        attn_ref.assert_within(turned[:T], want, want.abs() * eps + size * 2.0 ** -20, "q")
        for j, (b, t) in enumerate(at):
            keys[b, t] = _turned(k[j:j + 1], pos[j:j + 1], om)[0]
        starts = starts_of(new)
        if max(new) > 1:
            out = torch.full((T + 2, Hq, D), 9.0, dtype=dtype, device="cuda")
            _into(out, turned, cache, starts, table, lens, scale, window, sinks)
            assert bool((out[T:] == 9.0).all())
        else:
            rows = [b for b in range(3) if new[b]]
            out = gbe.attn_decode_window(turned[:T], cache, table[rows], i32([lens[b] for b in rows]), window, sinks, scale)
            again = gbe.attn_chunk(turned[:T], cache, i32(starts), table, i32(lens), scale, window, sinks)
        ref, tol, _ = chunk_ref.chunk(turned[:T], cache, starts, table, lens, scale, window, sinks, dtype == BF)
        attn_ref.assert_within(out[:T], ref, tol, f"step {i}")
        if max(new) == 1:
            attn_ref.assert_within(again, ref, tol, f"step {i}, as a chunk")
    # what the cache holds is what was appended: e4m3 codes are off by half a step of 4 bits, of the row's largest at most
    got = attn_ref.values(cache, "k")
    for b in range(3):
        t = torch.arange(total[b], device="cuda")
        row = got[table[b].long()[t // P], :, t % P]
        want = keys[b, :total[b]]
        size = want.abs().amax(-1, keepdim=True)
        tol = want.abs() * eps + size * 2.0 ** -20
        if kind == F8:
            tol = tol + want.abs() * 2.0 ** -4 * (1 + 2.0 ** -4) + size * 2.0 ** -16
        attn_ref.assert_within(row, want, tol, f"keys of sequence {b}")


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_a_prompt_in_pieces_is_the_whole_prompt(dtype, kind):
    """Any cut of a prompt gives its rows, within the sum of both bounds; and rows that do not move, the same bits."""
    Hq, H, D, P, n = 8, 2, 64, 16, 700
    q = rand((n, Hq, D), dtype, 5)
    cache, table = filled([n], P, H, D, dtype, kind, 3)
    whole = gbe.attn_chunk(q, cache, i32([0, n]), table, i32([n]), 0.125)
    want, tol, _ = chunk_ref.chunk(q, cache, [0, n], table, [n], 0.125, rounded=dtype == BF)
    attn_ref.assert_within(whole, want, tol)
    for cut in (1, 33, 128, 300, 699):
        for a, z in ((0, cut), (cut, n)):
            got = gbe.attn_chunk(q[a:z], cache, i32([0, z - a]), table, i32([z]), 0.125)
            attn_ref.assert_within(got, want[a:z], tol[a:z], (a, z))


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (BF, F8)])
@pytest.mark.parametrize("P", [1, 2, 3, 4, 6, 20])
@pytest.mark.parametrize("Hq,D", [(4, 64), (6, 128), (260, 16)])
def test_pages_of_few_tokens(dtype, kind, P, Hq, D):
    new, lens, H = [40, 1, 130], [333, 7, 259], 2
    cache, table = filled(lens, P, H, D, dtype, kind, 11)
    table[0, 5] = -1
    q = rand((sum(new), Hq, D), dtype, 12)
    for window, sinks in ((0, 0), (100, 9)):
        got = gbe.attn_chunk(q, cache, i32(starts_of(new)), table, i32(lens), 0.1, window, sinks)
        want, tol, _ = chunk_ref.chunk(q, cache, starts_of(new), table, lens, 0.1, window, sinks, True)
        attn_ref.assert_within(got, want, tol, (window, sinks))


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_many_sequences_most_of_them_empty(dtype, kind):
    Hq, H, D, P = 4, 2, 64, 16
    new = [0] * 300
    for b, n in ((0, 3), (1, 1), (40, 70), (41, 2), (127, 9), (128, 1), (200, 5), (299, 33)):
        new[b] = n
    lens = [n + (b * 37) % 90 if n else (b * 13) % 50 for b, n in enumerate(new)]
    lens[41] = 3000
    cache, table = filled(lens, P, H, D, dtype, kind, 13)
    starts = starts_of(new, 4)
    q = rand((starts[-1] + 6, Hq, D), dtype, 14)
    out = torch.full_like(q, 9.0)
    _into(out, q, cache, starts, table, lens, 0.1)
    want, tol, written = chunk_ref.chunk(q, cache, starts, table, lens, 0.1, rounded=dtype == BF)
    attn_ref.assert_within(out[written], want[written], tol[written])
    assert bool((out[~written] == 9.0).all())
    if kind == F8:
        return
    k, v = rand((q.shape[0], H, D), dtype, 15), rand((q.shape[0], H, D), dtype, 16)
    out.fill_(9.0)
    gbe.gbe_attn_prompt_window(q, k, v, out, i32(starts), 20, 2, 0.1)
    want, tol, written = chunk_ref.prompt(q, k, v, starts, 0.1, 20, 2, dtype == BF)
    attn_ref.assert_within(out[written], want[written], tol[written])
    assert bool((out[~written] == 9.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_odd_codes_and_scales_of_an_8_bit_cache(dtype):
    """Scales from nothing to beyond what bf16 codes are widened by in one step, every code; a NaN code reaches the rows
    that see it and no others; a scale byte of 0 is zeros whatever the codes."""
    Hq, H, D, P, n, m = 4, 1, 64, 16, 300, 20
    cache, table = filled([n], P, H, D, dtype, F8, 17)
    g = torch.Generator(device="cuda").manual_seed(18)
    for x, s, top in ((cache.k, cache.k_scale, (0, 1, 60, 120, 127, 134, 135, 136)),
                      (cache.v, cache.v_scale, (0, 1, 7, 100, 127, 134, 135, 180))):
        codes = torch.randint(0, 254, x.shape, generator=g, device="cuda")
        codes = codes + (codes >= 0x7F)  # neither 7F nor FF
        x.view(torch.uint8).copy_(codes.to(torch.uint8))
        pick = torch.randint(0, len(top), s.shape, generator=g, device="cuda")
        s.copy_(torch.tensor(top, dtype=torch.uint8, device="cuda")[pick])
    q = rand((m, Hq, D), dtype, 19, 2.0 ** -9)

    def at(t): return int(table[0, t // P]), 0, t % P

    def run(): return gbe.attn_chunk(q, cache, i32([0, m]), table, i32([n]), 0.1)

    want, tol, _ = chunk_ref.chunk(q, cache, [0, m], table, [n], 0.1, rounded=dtype == BF)
    # A weight below 2^-126 of the row's largest has no normal f32: it is off by 2^-126 at most, of a sum of 1 at least.
    # With values up to 448 2^53 that is up to 5e-20 a key, which the relative bounds (made for weights that are normal
    # numbers) leave out.
    small = 2.0 ** -126 * sum(attn_ref.values(cache, "v")[at(t)].abs() for t in range(n))
    attn_ref.assert_within(run(), want, tol + small)
    for t in (0, 150, n - m + 7):
        one = attn_ref.values(cache, "v")[at(t)].clone(), cache.v.view(torch.uint8)[at(t)].clone()
        cache.v.view(torch.uint8)[at(t)] = 0xFF
        scale = int(cache.v_scale[at(t)])
        cache.v_scale[at(t)] = 0
        zeros = run()
        ref, e, _ = chunk_ref.chunk(q, _clean(cache, at(t)), [0, m], table, [n], 0.1, rounded=dtype == BF)
        attn_ref.assert_within(zeros, ref, e + small, "a scale of nothing")
        cache.v_scale[at(t)] = 127
        got = run()
        first = max(0, t - (n - m))
        assert bool(got[first:].isnan().all())
        attn_ref.assert_within(got[:first], want[:first], tol[:first] + small)
        cache.v.view(torch.uint8)[at(t)], cache.v_scale[at(t)] = one[1], scale


def _clean(cache, at):
    """The cache with zeros in place of one row of v."""
    v = cache.v.clone()
    v.view(torch.uint8)[at] = 0
    return gbe.KvCache(cache.k, v, cache.k_scale, cache.v_scale)


def test_calls_at_once_from_threads_and_streams():
    """Four threads, each with a stream, a workspace and a cache of its own: the bits of the calls one by one."""
    jobs, got, errors = [], {}, []
    for i, (dtype, kind) in enumerate(KINDS):
        new, lens = [30, 1, 8], [3000, 4000 + i, 70]
        cache, table = filled(lens, 16, 2, 64, dtype, kind, 21 + i)
        q = rand((39, 8, 64), dtype, 31 + i)
        args = q, cache, i32(starts_of(new)), table, i32(lens), 0.1
        want = (gbe.attn_chunk(*args), gbe.attn_chunk(*args, 900, 5),
                gbe.attn_decode_window(q[:3], cache, table, i32(lens), 900, 5, 0.1))
        jobs.append((args, lens, want, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(i):
        try:
            (q, cache, starts, table, lens, scale), _, _, stream = jobs[i]
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got[i] = (gbe.attn_chunk(q, cache, starts, table, lens, scale),
                              gbe.attn_chunk(q, cache, starts, table, lens, scale, 900, 5),
                              gbe.attn_decode_window(q[:3], cache, table, lens, 900, 5, scale))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001  (a thread's failure is the test's)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for i, (_, _, want, _) in enumerate(jobs):
        for a, b in zip(got[i], want):
            assert torch.equal(a, b), i


FIRST = """
import sys, torch
sys.path[:0] = [{tests!r}, {root!r}]
import chunk_ref, elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import i32, rand
dtype, kind = {dtype}, {kind}
H, Hq, D, P = 2, 8, 128, 16
cache = gbe.kv_cache(200, H, P, D, kind)
table = torch.arange(200, dtype=torch.int32, device="cuda").view(1, 200)
q, k, v = rand((30, Hq, D), dtype, 1), rand((30, H, D), dtype, 2), rand((30, H, D), dtype, 3)
om = (10000.0 ** (-torch.arange(D // 2, device="cuda").double() * 2 / D)).float()
pos = torch.arange(3000, 3030, dtype=torch.int32, device="cuda")
starts, lens = i32([0, 30]), i32([3030])
room = torch.empty(max(1, gbe.attn_chunk_workspace(1, 30, Hq, cache, 200), gbe.attn_decode_workspace(1, Hq, cache, 200, 999, 4)),
                   dtype=torch.uint8, device="cuda")
outs = [torch.empty_like(q) for _ in range(3)] + [torch.empty_like(q[:1])]
for t in (cache.k, cache.v):
    t.view(torch.uint8).fill_(0x11)
if kind == torch.float8_e4m3fn:
    cache.k_scale.fill_(127), cache.v_scale.fill_(127)

def run():
    gbe.gbe_rope_kv_write(q, outs[0], k, v, pos, pos, cache, om, D)
    gbe.gbe_attn_chunk(outs[0], outs[1], cache, starts, table, lens, 0.1, 0, 0, room)
    gbe.gbe_attn_decode_window(outs[0][:1], outs[3], cache, table, lens, 999, 4, 0.1, room)
    if kind == dtype:
        gbe.gbe_attn_prompt_window(outs[0], k, v, outs[2], starts, 9, 1, 0.1)

graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    run()
graph.replay()
torch.cuda.synchronize()
first = [o.clone() for o in outs]
run()
torch.cuda.synchronize()
for i, (a, b) in enumerate(zip(first, outs)):
    assert (i == 2 and kind != dtype) or torch.equal(a, b), i
    assert i == 2 or bool(a.isfinite().all()), i
print("same bits")
"""


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_a_process_first_calls_are_captured(dtype, kind):
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST.format(tests=here, root=os.path.dirname(here), dtype=str(dtype), kind=str(kind))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_buffers_past_2_31_entries(dtype, kind):
    """Pages whose first entry is past 2^31 (past 2^32 bytes), and rows as far apart."""
    Hq, H, D, P = 4, 2, 128, 64
    pages = 2 ** 31 // (H * P * D) + 40
    cache = gbe.KvCache(*(torch.empty(pages, H, P, D, dtype=kind, device="cuda") for _ in range(2)),
                        *(torch.empty(pages, H, P, dtype=torch.uint8, device="cuda") if kind == F8 else None
                          for _ in range(2)))
    n, m, last = 1300, 20, pages - 1
    ids = [last - 2 * i for i in range(-(-n // P) - 3)] + [0, 5, last - 1]
    table = i32([ids])
    slots = i32([ids[t // P] * P + t % P for t in range(n)])
    k, v = rand((n, H, D), dtype, 41), rand((n, H, D), dtype, 42)
    far = torch.empty(2 * (2 ** 30 + 64) + Hq * D, dtype=dtype, device="cuda")
    q = far.as_strided((3, Hq, D), (2 ** 30 + 64, D, 1))
    q.copy_(rand((3, Hq, D), dtype, 43))
    # the last three tokens by the appending call, whose rows of q lie 2^30 entries apart
    gbe.gbe_kv_write(k[:-3], v[:-3], slots[:-3].contiguous(), cache)
    om = torch.zeros(D // 2, device="cuda")  # (turned by nothing)
    gbe.gbe_rope_kv_write(q, q, k[-3:].contiguous(), v[-3:].contiguous(), i32([0, 0, 0]), slots[-3:].contiguous(), cache, om, D)
    small = gbe.KvCache(*(None if t is None else t[torch.tensor(ids, device="cuda")] for t in (cache.k, cache.v, cache.k_scale,
                                                                                        cache.v_scale)))
    near = torch.arange(len(ids), dtype=torch.int32, device="cuda")[None]
    want_k = attn_ref.values(small, "k")[near[0].long()].transpose(1, 2).reshape(-1, H, D)[:n]
    exact = 2.0 ** -4 if kind == F8 else 0.0
    attn_ref.assert_within(want_k, k.double(), k.double().abs() * exact + k.double().abs().amax(-1, keepdim=True) * exact / 64)
    for window, sinks in ((0, 0), (300, 70)):
        want, tol, _ = chunk_ref.chunk(q.contiguous(), small, [0, 3], near, [n], 0.1, window, sinks, dtype == BF)
        out = far.new_empty(far.numel()).as_strided(q.shape, q.stride())
        _into(out, q, cache, [0, 3], table, [n], 0.1, window, sinks)
        attn_ref.assert_within(out, want, tol, (window, sinks))
        one = gbe.attn_decode_window(q[2:], cache, table, i32([n]), window, sinks, 0.1)
        attn_ref.assert_within(one, want[2:], tol[2:], (window, sinks))


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_starts_that_decrease_stay_within_the_buffers(dtype, kind):
    """Rows that one sequence has are right, rows that two have are one's or the other's, no others are written."""
    Hq, H, D, P = 4, 2, 64, 16
    starts, lens = [5, 50, 20, 60, -7, 2 ** 30], [3000, 40, 90, 7, 200]
    cache, table = filled(lens, P, H, D, dtype, kind, 51)
    q = rand((64, Hq, D), dtype, 52)
    out = torch.full_like(q, 9.0)
    _into(out, q, cache, starts[:4], table[:3], lens[:3], 0.1)
    one, tol, _ = chunk_ref.chunk(q, cache, starts[:2], table[:1], lens[:1], 0.1, rounded=dtype == BF)
    two, e, _ = chunk_ref.chunk(q, cache, starts[2:4], table[2:3], lens[2:3], 0.1, rounded=dtype == BF)
    attn_ref.assert_within(out[5:20], one[5:20], tol[5:20])
    attn_ref.assert_within(out[50:60], two[50:60], e[50:60])
    assert bool((((out[20:50] - one[20:50]).abs() <= tol[20:50]) | ((out[20:50] - two[20:50]).abs() <= e[20:50])).all())
    assert bool((out[:5] == 9.0).all()) and bool((out[60:] == 9.0).all())
    _into(out, q, cache, starts, table, lens, 0.1)  # ends outside the buffers count as these
    assert bool(out.isfinite().all()) and bool((out != 9.0).any(-1).all())
