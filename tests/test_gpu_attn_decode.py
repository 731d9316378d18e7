"""gbe_attn_decode on the GPU against the definition in 64 bits: types, head
layouts, page sizes, lengths around every border, poisoned memory around the
live tokens, batch invariance, guard regions, streams and graphs."""
import math

import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _filled(lens, P, H, D, dtype, kind, seed, spare_pages=3, spare_cols=0, std=1.0):
    """A cache whose live tokens are random and whose every other byte is NaN, and its table."""
    pages = sum(-(-n // P) for n in lens) + spare_pages
    cache = gbe.kv_cache(pages, H, P, D, kind)
    if kind == F8:
        cache.k.view(torch.uint8).fill_(0x7F)
        cache.v.view(torch.uint8).fill_(0xFF)
        cache.k_scale.fill_(254)
        cache.v_scale.fill_(254)
    else:
        cache.k.fill_(float("nan"))
        cache.v.fill_(float("nan"))
    table = attn_ref.make_table(lens, P, pages, seed, spare_cols)
    slots = [int(table[b, t // P]) * P + t % P for b, n in enumerate(lens) for t in range(n)]
    if slots:
        slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
        gbe.gbe_kv_write(_rand((len(slots), H, D), dtype, seed, std), _rand((len(slots), H, D), dtype, seed + 1),
                         slots, cache)
    return cache, table.cuda()


def _check(q, cache, table, lens, scale, what=""):
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = gbe.attn_decode(q, cache, table, lens_t, scale)
    want, tol = attn_ref.decode(q, cache, table, lens, scale, rounded=q.dtype == BF)
    attn_ref.assert_within(got, want, tol, what)
    return got


KINDS = [(F32, F32), (F32, F8), (BF, BF), (BF, F8)]
BORDERS = [0, 1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("Hq,H,D,P", [(4, 1, 64, 16), (8, 2, 128, 64), (3, 3, 128, 48), (2, 2, 8, 1), (7, 1, 72, 100),
                                      (16, 2, 80, 32), (14, 2, 256, 16), (40, 1, 96, 64), (24, 2, 136, 128)])
def test_lengths_around_the_borders(dtype, kind, Hq, H, D, P):
    cache, table = _filled(BORDERS, P, H, D, dtype, kind, 21)
    q = _rand((len(BORDERS), Hq, D), dtype, 23)
    got = _check(q, cache, table, BORDERS, 1.0 / math.sqrt(D))
    assert bool((got[0] == 0).all()), "a sequence of no tokens gives zeros"


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("lens,Hq,H,D,P", [([5000], 8, 1, 128, 64), ([4097, 0, 1, 2500, 1030], 32, 8, 128, 64),
                                           ([3001, 777], 6, 2, 64, 16), ([20000], 4, 2, 64, 128)])
def test_long_rows_are_split_and_joined(dtype, kind, lens, Hq, H, D, P):
    cache, table = _filled(lens, P, H, D, dtype, kind, 31)
    q = _rand((len(lens), Hq, D), dtype, 33, 2.0)
    _check(q, cache, table, lens, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_sharp_flat_and_signed_logits(dtype, kind):
    lens, Hq, H, D, P = [700, 130, 64], 8, 2, 64, 16
    cache, table = _filled(lens, P, H, D, dtype, kind, 41)
    for std, scale in ((30.0, 0.125), (0.0, 0.125), (1.0, 0.0), (1.0, -0.5), (1e-3, 1e-6)):
        _check(_rand((3, Hq, D), dtype, 43, std), cache, table, lens, scale, f"std {std} scale {scale}")


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_batch_invariance(dtype, kind):
    """A row alone and the same row in a batch: the same bits."""
    lens, Hq, H, D, P = [1500, 0, 333, 64, 2000, 1], 12, 2, 128, 32
    cache, table = _filled(lens, P, H, D, dtype, kind, 51)
    q = _rand((len(lens), Hq, D), dtype, 53)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    whole = gbe.attn_decode(q, cache, table, lens_t, 0.1)
    for b in range(len(lens)):
        one = gbe.attn_decode(q[b:b + 1], cache, table[b:b + 1], lens_t[b:b + 1], 0.1)
        assert torch.equal(one[0], whole[b]), b
    again = gbe.attn_decode(q, cache, table, lens_t, 0.1)
    assert torch.equal(again, whole), "the same bits every time"


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_lengths_out_of_range_and_bad_pages(dtype, kind):
    """A negative length is none, one above the table's capacity is that; tokens on a page outside the cache take no
    part, a row of nothing but such pages is zeros."""
    P, H, D, Hq = 16, 2, 64, 4
    lens = [40, 160, 160, 100, 33]
    cache, table = _filled(lens, P, H, D, dtype, kind, 61)
    table[2, 3] = -1
    table[2, 5] = cache.shape[0]
    table[3, :] = torch.tensor([-5, 2 ** 31 - 1] * 5, dtype=torch.int32)
    q = _rand((5, Hq, D), dtype, 63)
    asked = [-3, 10 ** 6, 160, 100, 33]
    got = _check(q, cache, table, asked, 0.125)
    assert bool((got[0] == 0).all()) and bool((got[3] == 0).all())


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF, BF)])
def test_infinities_and_nan_in_attended_places(dtype, kind):
    P, H, D, Hq = 16, 1, 64, 3
    lens = [200, 200, 200, 200, 200]
    cache, table = _filled(lens, P, H, D, dtype, kind, 71)

    def at(b, t): return int(table[b, t // P]), 0, t % P
    cache.k[at(1, 77)][5] = float("nan")        # every logit of that token NaN: the row is NaN
    cache.v[at(2, 150)][9] = float("inf")       # one value: its entry only
    for t in range(200):
        cache.k[at(3, t)][0] = float("nan")     # nothing but NaN
    cache.v[at(4, 3)][11] = float("nan")
    q = _rand((5, Hq, D), dtype, 73)
    got = gbe.attn_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), 0.125)
    want, tol = attn_ref.decode(q[:1], cache, table[:1], lens[:1], 0.125, dtype == BF)
    attn_ref.assert_within(got[:1], want, tol, "a row next to them")
    assert bool(got[1].isnan().all()) and bool(got[3].isnan().all())
    assert bool((got[2][:, 9] == float("inf")).all()) and int((~torch.isfinite(got[2])).sum()) == Hq
    assert bool(got[4][:, 11].isnan().all()) and int((~torch.isfinite(got[4])).sum()) == Hq


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("pad", [0, 3])
def test_strided_rows_guards_and_a_dirty_workspace(dtype, kind, pad):
    """q and out as columns of wider buffers (pad = 3: off the 16-byte grid); the workspace holds NaN and is not
    written past its size."""
    lens, Hq, H, D, P = [900, 20, 0], 6, 2, 72, 16
    cache, table = _filled(lens, P, H, D, dtype, kind, 81)
    wide = _rand((3, 2 * Hq * D + pad), dtype, 83)
    q = wide[:, pad:pad + Hq * D].unflatten(1, (Hq, D))
    out = torch.full((3, 3 * Hq * D + pad), 5.0, dtype=dtype, device="cuda")
    o = out[:, Hq * D + pad:2 * Hq * D + pad].unflatten(1, (Hq, D))
    n = gbe.attn_decode_workspace(3, Hq, cache, table.shape[1])
    raw = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gbe.gbe_attn_decode(q, o, cache, table, lens_t, 0.1, raw[256:256 + n])
    want, tol = attn_ref.decode(q, cache, table, lens, 0.1, dtype == BF)
    attn_ref.assert_within(o, want, tol)
    assert bool((raw[:256] == 0xFF).all()) and bool((raw[256 + n:] == 0xFF).all())
    assert bool((out[:, :Hq * D + pad] == 5.0).all()) and bool((out[:, 2 * Hq * D + pad:] == 5.0).all())


@pytest.mark.parametrize("kind", [BF, F8])
def test_offsets_past_32_bits(kind):
    H, P, D, N, Hq = 8, 64, 128, 70000, 32
    shape = (N, H, P, D)
    k, v = torch.empty(shape, dtype=kind, device="cuda"), torch.empty(shape, dtype=kind, device="cuda")
    s = [torch.zeros(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == F8 else [None, None]
    cache = gbe.KvCache(k, v, *s)
    lens = [300, 500]
    order = [69999, 32768, 3, 65536, 40000, 69998, 50000, 60000, 7, 32767, 65535, 12345, 54321]
    table = torch.tensor([order[:5] + [0] * 3, order[5:13]], dtype=torch.int32)
    slots = torch.tensor([int(table[b, t // P]) * P + t % P for b, n in enumerate(lens) for t in range(n)],
                         dtype=torch.int32, device="cuda")
    kn, vn = _rand((800, H, D), BF, 91), _rand((800, H, D), BF, 92)
    gbe.gbe_kv_write(kn, vn, slots, cache)
    q = _rand((2, Hq, D), BF, 93)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = gbe.attn_decode(q, cache, table.cuda(), lens_t)
    # the same tokens in a small cache: the same bits
    small = gbe.kv_cache(13, H, P, D, kind)
    t2 = torch.tensor([[0, 1, 2, 3, 4, 0, 0, 0], [5, 6, 7, 8, 9, 10, 11, 12]], dtype=torch.int32)
    slots2 = torch.tensor([int(t2[b, t // P]) * P + t % P for b, n in enumerate(lens) for t in range(n)],
                          dtype=torch.int32, device="cuda")
    gbe.gbe_kv_write(kn, vn, slots2, small)
    assert torch.equal(got, gbe.attn_decode(q, small, t2.cuda(), lens_t))
    _check(q, small, t2.cuda(), lens, 1.0 / math.sqrt(D))


def test_interleaved_halves():
    H, P, D, N, Hq = 2, 16, 128, 20, 8
    kv = torch.full((N, 2, H, P, D), float("nan"), dtype=BF, device="cuda")
    cache = gbe.KvCache(kv[:, 0], kv[:, 1])
    lens = [130, 70]
    table = attn_ref.make_table(lens, P, N, 3)
    slots = torch.tensor([int(table[b, t // P]) * P + t % P for b, n in enumerate(lens) for t in range(n)],
                         dtype=torch.int32, device="cuda")
    gbe.gbe_kv_write(_rand((200, H, D), BF, 1), _rand((200, H, D), BF, 2), slots, cache)
    _check(_rand((2, Hq, D), BF, 3), cache, table.cuda(), lens, 0.09)


@pytest.mark.parametrize("kind", [BF, F8])
def test_graph_replay_with_growing_sequences(kind):
    """One captured step (store the token, attend) replayed as the sequences grow, while an eager call with a
    workspace of its own runs on another stream."""
    H, P, D, Hq, B = 2, 16, 64, 8, 3
    cache = gbe.kv_cache(64, H, P, D, kind)
    table = torch.randperm(60, generator=torch.Generator().manual_seed(2)).view(3, 20).to(torch.int32).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.zeros(B, dtype=torch.int32, device="cuda")
    k, v, q = (torch.zeros((B, h, D), dtype=BF, device="cuda") for h in (H, H, Hq))
    out = torch.zeros_like(q)
    ws = torch.empty(max(1, gbe.attn_decode_workspace(B, Hq, cache, 20)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gbe.gbe_kv_write(k, v, slots, cache)
        gbe.gbe_attn_decode(q, out, cache, table, lens, 0.125, ws)
    n = [0, 100, 255]
    for b in range(B):  # the prompts
        if n[b]:
            sl = torch.tensor([int(table[b, t // P]) * P + t % P for t in range(n[b])], dtype=torch.int32, device="cuda")
            gbe.gbe_kv_write(_rand((n[b], H, D), BF, b), _rand((n[b], H, D), BF, 10 + b), sl, cache)
    other = torch.cuda.Stream()
    for step in range(5):
        k.copy_(_rand((B, H, D), BF, 100 + step))
        v.copy_(_rand((B, H, D), BF, 200 + step))
        q.copy_(_rand((B, Hq, D), BF, 300 + step))
        slots.copy_(torch.tensor([int(table[b, n[b] // P]) * P + n[b] % P for b in range(B)], dtype=torch.int32))
        n = [x + 1 for x in n]
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            eager = gbe.attn_decode(q, cache, table, lens, 0.125)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager, out)
        want, tol = attn_ref.decode(q, cache, table, n, 0.125, True)
        attn_ref.assert_within(out, want, tol, f"step {step}")


def test_stream_argument():
    lens, Hq, H, D, P = [2000, 1000], 8, 2, 128, 64
    cache, table = _filled(lens, P, H, D, BF, BF, 101)
    q = _rand((2, Hq, D), BF, 103)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = gbe.attn_decode(q, cache, table, lens_t, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [gbe.attn_decode(q, cache, table, lens_t, 0.1, stream=side) for _ in range(4)]
    got.append(gbe.attn_decode(q, cache, table, lens_t, 0.1, stream=side.cuda_stream))
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g, want)


@pytest.mark.parametrize("kind", [BF, F8])
@pytest.mark.parametrize("D", [64, 128])
def test_a_large_batch_has_the_bits_of_its_rows_alone(kind, D):
    """Batches in which a CTA takes several chunks one after another; lengths of every residue."""
    B, Hq, H, P = 60, 16, 8, 64
    g = torch.Generator().manual_seed(5)
    lens = [8192, 0, 1, 511, 512, 513, 8191, 4097] + torch.randint(0, 8193, (B - 8,), generator=g).tolist()
    need = [-(-n // P) for n in lens]
    pages = sum(need) + 1
    cache = gbe.kv_cache(pages, H, P, D, kind)
    for t, seed in ((cache.k, 1), (cache.v, 2)):
        if kind == F8:  # codes of magnitude up to 30, no NaN
            t.view(torch.uint8).copy_(torch.randint(0, 96, t.shape, dtype=torch.uint8, device="cuda")
                                      | torch.randint(0, 2, t.shape, dtype=torch.uint8, device="cuda") << 7)
        else:
            t.copy_(_rand(t.shape, BF, seed))
    if kind == F8:
        for t in (cache.k_scale, cache.v_scale):
            t.copy_(torch.randint(121, 126, t.shape, dtype=torch.uint8, device="cuda"))
    table = torch.zeros(B, max(need), dtype=torch.int32)
    order = torch.randperm(pages, generator=g).tolist()
    for b, m in enumerate(need):
        for i in range(m):
            table[b, i] = order.pop()
    table = table.cuda()
    q = _rand((B, Hq, D), BF, 3)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    whole = gbe.attn_decode(q, cache, table, lens_t)
    for b in range(B):
        one = gbe.attn_decode(q[b:b + 1], cache, table[b:b + 1], lens_t[b:b + 1])
        assert torch.equal(one[0], whole[b]), (b, lens[b])
    for b in (0, 3, 7, 20):
        want, tol = attn_ref.decode(q[b:b + 1], cache, table[b:b + 1], lens[b:b + 1], 1.0 / math.sqrt(D), True)
        attn_ref.assert_within(whole[b:b + 1], want, tol, f"row {b}")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_e4m3_scales_far_apart(dtype, D):
    """Rows of v from 1e-9 to 1e9 in one sequence, the large ones with small weights, and rows of zeros; k likewise."""
    P, H, Hq, n = 16, 2, 8, 600
    cache = gbe.kv_cache(40, H, P, D, F8)
    g = torch.Generator(device="cuda").manual_seed(8)
    size = torch.rand(n, H, 1, generator=g, device="cuda") * 18.0 - 9.0
    size[::7] = -9.0
    size[5] = 9.0
    k, v = _rand((n, H, D), dtype, 1), (_rand((n, H, D), F32, 2) * 10.0 ** size).to(dtype)
    v[::50] = 0.0
    # a common direction that the tokens with large values are turned away from
    away = _rand((1, H, D), F32, 4)
    k = (k.float() - away * (size + 9.0) * 0.6).to(dtype)
    k[3] *= 1e-6
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    gbe.gbe_kv_write(k, v, slots, cache)
    table = torch.arange(38, dtype=torch.int32, device="cuda")[None]
    q = (_rand((1, Hq, D), F32, 3) * 0.3 + away.repeat_interleave(Hq // H, 1)).to(dtype)
    for m in (n, 16, 100):
        _check(q, cache, table, [m], 1.0 / math.sqrt(D), f"{m} tokens")


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("power", [-100, -60, 60, 100])
def test_e4m3_magnitudes_that_make_up_for_one_another(dtype, power):
    """q of 2^power and k of 2^-power, and the other way round: the logits are ordinary."""
    P, H, Hq, D, n = 16, 1, 4, 64, 200
    cache = gbe.kv_cache(13, H, P, D, F8)
    k, v = _rand((n, H, D), F32, 11), _rand((n, H, D), dtype, 12)
    gbe.gbe_kv_write((k * 2.0 ** -power).to(dtype), v, torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    table = torch.arange(13, dtype=torch.int32, device="cuda")[None]
    q = (_rand((1, Hq, D), F32, 13) * 2.0 ** power).to(dtype)
    _check(q, cache, table, [n], 0.125, f"2^{power}")


def test_a_workspace_allocated_for_another_stream_is_that_streams():
    """The memory is not one that work still queued on the current stream writes to."""
    lens, Hq, H, D, P = [6000, 3000], 8, 2, 128, 64
    cache, table = _filled(lens, P, H, D, BF, BF, 111)
    q = _rand((2, Hq, D), BF, 113)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = gbe.attn_decode(q, cache, table, lens_t, 0.1)
    n = gbe.attn_decode_workspace(2, Hq, cache, table.shape[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.zeros(1 << 28, device="cuda")
    for _ in range(3):
        for _ in range(20):
            big.add_(1.0)  # keeps the current stream busy
        scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
        for _ in range(50):
            scratch.fill_(0xFF)
        del scratch  # its memory is free for the next allocation on the current stream
        got = gbe.attn_decode(q, cache, table, lens_t, 0.1, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
