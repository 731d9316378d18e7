"""gbe_kv_write and gbe_kv_read on the GPU: bits of every cache type, strided
and unaligned rows, padding and bad slots, what is left untouched, special
values, offsets past 32 bits, graphs."""
import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
PAIRS = [(torch.float32, torch.float32), (torch.float32, F8), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, F8)]


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _sentinel(cache):
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(0x5A)


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


def _expect(cache, which, rows, slots):
    """The bytes of k or v and of its scales after the write, from their bytes before it."""
    x, s = getattr(cache, which), getattr(cache, which + "_scale")
    want, want_s = x.clone(), None if s is None else s.clone()
    P = cache.shape[2]
    keep = [(t, int(v)) for t, v in enumerate(slots.tolist()) if 0 <= v < cache.shape[0] * P]
    if s is None:
        for t, v in keep:
            want[v // P, :, v % P] = rows[t]
        return want, None
    codes, bytes_ = attn_ref.encode(rows)
    w8 = want.view(torch.uint8)
    for t, v in keep:
        w8[v // P, :, v % P] = codes[t].cuda()
        want_s[v // P, :, v % P] = bytes_[t].cuda()
    return want, want_s


def _check_write(cache, k, v, slots, bad=None):
    want = {w: _expect(cache, w, r, slots) for w, r in (("k", k), ("v", v))}
    gbe.gbe_kv_write(k, v, slots, cache, bad)
    for w, (x, s) in want.items():
        assert torch.equal(_bytes(getattr(cache, w)), _bytes(x)), w
        if s is not None:
            assert torch.equal(getattr(cache, w + "_scale"), s), w


@pytest.mark.parametrize("dtype,kind", PAIRS)
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 8, 1), (1, 8, 128, 64), (37, 3, 64, 16), (50, 2, 72, 48), (129, 5, 256, 7),
                                     (64, 1, 136, 100), (300, 8, 128, 64)])
def test_write_then_read(dtype, kind, T, H, D, P):
    pages = -(-T // P) + 2
    cache = gbe.kv_cache(pages, H, P, D, kind)
    _sentinel(cache)
    k, v = _rand((T, H, D), dtype, 1), _rand((T, H, D), dtype, 2, 30.0)
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32).cuda()
    _check_write(cache, k, v, slots)
    gk, gv = gbe.kv_read(cache, slots, dtype)
    for got, rows, w in ((gk, k, "k"), (gv, v, "v")):
        if kind == F8:
            at = slots.long()
            want = attn_ref.values(cache, w)[at // P, :, at % P]
            assert torch.equal(got.double(), want), w
            # one rounding to 4 significant bits, or half the least step
            assert bool(((got.double() - rows.double()).abs() <= rows.double().abs() * 2.0 ** -4
                         + rows.double().abs().amax(-1, keepdim=True) * 2.0 ** -17).all()), w
        else:
            assert torch.equal(got, rows), w


@pytest.mark.parametrize("dtype,kind", PAIRS)
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_slices_of_a_fused_buffer_padding_and_bad_slots(dtype, kind, pad):
    """k and v as columns of one buffer (pad = 1: rows off the 16-byte grid), some tokens not stored."""
    T, H, D, P, pages = 45, 3, 80, 16, 5
    fused = _rand((T, 4 * H * D + pad), dtype, 3)
    k = fused[:, H * D:2 * H * D].unflatten(1, (H, D))
    v = fused[:, 3 * H * D:4 * H * D].unflatten(1, (H, D))
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(5))[:T].to(torch.int32)
    slots[4], slots[10], slots[11], slots[30], slots[44] = -1, -2, pages * P, 2 ** 31 - 1, -2 ** 31
    slots = slots.cuda()
    cache = gbe.kv_cache(pages, H, P, D, kind)
    _sentinel(cache)
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    _check_write(cache, k, v, slots, bad)
    assert int(bad) == 4  # -1 is padding, not an error
    out = torch.full((T, 4 * H * D + pad), 7.0, dtype=dtype, device="cuda")
    ok, ov = out[:, :H * D].unflatten(1, (H, D)), out[:, H * D:2 * H * D].unflatten(1, (H, D))
    gbe.gbe_kv_read(ok, ov, slots, cache, bad)
    assert int(bad) == 8
    at = slots.long()
    gone = (at < 0) | (at >= pages * P)
    at = at.clamp(0, pages * P - 1)
    for got, w in ((ok, "k"), (ov, "v")):
        want = attn_ref.values(cache, w)[at // P, :, at % P]
        want[gone] = 0.0
        assert torch.equal(got.double(), want), w
    assert bool((out[:, 2 * H * D:] == 7.0).all()), "columns that are not k or v"


@pytest.mark.parametrize("dtype,kind", PAIRS)
def test_halves_of_one_page_buffer(dtype, kind):
    """k = kv[:, 0], v = kv[:, 1]: pages a stride apart, interleaved."""
    N, H, P, D, T = 6, 2, 16, 64, 40
    kv = torch.zeros((N, 2, H, P, D), dtype=kind, device="cuda")
    scales = [torch.zeros((N, H, P), dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == F8 else [None] * 2
    cache = gbe.KvCache(kv[:, 0], kv[:, 1], *scales)
    k, v = _rand((T, H, D), dtype, 6), _rand((T, H, D), dtype, 7)
    slots = torch.randperm(N * P, generator=torch.Generator().manual_seed(8))[:T].to(torch.int32).cuda()
    _check_write(cache, k, v, slots)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_e4m3_special_rows(dtype):
    """Zeros, signed zeros, infinities, NaN, the largest and the smallest numbers, ties and the borders of a scale."""
    D, H, P = 64, 1, 32
    big = torch.finfo(dtype).max
    rows = torch.zeros(20, H, D)
    rows[1] = -0.0
    rows[2, 0, 0] = float("inf")
    rows[2, 0, 1:4] = torch.tensor([1.0, -448.0, 3.0])
    rows[3, 0, :3] = torch.tensor([float("nan"), 2.0, float("-inf")])
    rows[4] = float("nan")
    rows[5, 0, :2] = torch.tensor([big, -big])
    rows[6, 0, :3] = torch.tensor([1e-38, -1e-40, 2.0 ** -126])
    rows[7, 0, :4] = torch.tensor([448.0, 464.0, 1.0, 2.0 ** -9])         # 464 is above 448: twice the scale
    rows[8, 0, :2] = torch.tensor([448.0, 2.0 ** -10])                    # half the least code: to even, 0
    rows[9, 0, :3] = torch.tensor([448.0, 3 * 2.0 ** -10, 5 * 2.0 ** -10])
    rows[10, 0, :17] = 256.0 + 16.0 * torch.arange(17)                    # ties between neighbours 32 apart
    rows[10, 0, 13:17] = 0.0
    rows[11, 0, :17] = 16.0 + torch.arange(17)
    for i in range(12, 20):
        rows[i] = torch.linspace(-3.0, 5.0, D) * 10.0 ** (i - 15)
    rows = rows.to(dtype).cuda()
    cache = gbe.kv_cache(2, H, P, D, F8)
    slots = torch.arange(20, dtype=torch.int32, device="cuda")
    _check_write(cache, rows, rows.flip(0).contiguous(), slots)
    k, _ = gbe.kv_read(cache, slots, dtype)
    k = k.float().cpu()
    assert bool((k[:2] == 0).all()) and bool(k[2, 0, 0].isnan()) and k[2, 0, 2] == -448.0
    assert bool(k[3, 0, 0].isnan()) and bool(k[3, 0, 2].isnan()) and k[3, 0, 1] == 2.0
    assert bool(k[4].isnan().all()) and bool(torch.isfinite(k[5]).all())
    # an untouched (zeroed) row stands for zeros
    z, _ = gbe.kv_read(cache, torch.tensor([40, 63], dtype=torch.int32, device="cuda"), dtype)
    assert bool((z == 0).all())


@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
def test_offsets_past_32_bits(kind):
    H, P, D, N = 8, 64, 128, 70000  # 4.6e9 elements in k and in v
    shape = (N, H, P, D)
    k, v = torch.empty(shape, dtype=kind, device="cuda"), torch.empty(shape, dtype=kind, device="cuda")
    s = [torch.empty(shape[:3], dtype=torch.uint8, device="cuda") for _ in range(2)] if kind == F8 else [None, None]
    cache = gbe.KvCache(k, v, *s)
    slots = torch.tensor([0, N * P - 1, 32768 * P, 32767 * P + 63, 65536 * P + 5], dtype=torch.int32, device="cuda")
    rows, more = _rand((5, H, D), torch.bfloat16, 9), _rand((5, H, D), torch.bfloat16, 10)
    gbe.gbe_kv_write(rows, more, slots, cache)
    at = slots.long()
    for x, sc, want in ((k, s[0], rows), (v, s[1], more)):
        if kind == F8:
            codes, bytes_ = attn_ref.encode(want)
            assert torch.equal(x.view(torch.uint8)[at // P, :, at % P].cpu(), codes)
            assert torch.equal(sc[at // P, :, at % P].cpu(), bytes_)
        else:
            assert torch.equal(x[at // P, :, at % P], want)
    gk, gv = gbe.kv_read(cache, slots)
    if kind != F8:
        assert torch.equal(gk, rows) and torch.equal(gv, more)
    # the same slot read twice
    gk2, _ = gbe.kv_read(cache, torch.cat([slots, slots]))
    assert torch.equal(gk2[:5], gk) and torch.equal(gk2[5:], gk)


def test_graph_replay_reads_the_slots_of_the_moment():
    H, P, D, T = 2, 16, 64, 8
    cache = gbe.kv_cache(8, H, P, D, F8)
    k, v = _rand((T, H, D), torch.bfloat16, 11), _rand((T, H, D), torch.bfloat16, 12)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    ok, ov = torch.empty_like(k), torch.empty_like(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gbe.gbe_kv_write(k, v, slots, cache)
        gbe.gbe_kv_read(ok, ov, slots, cache)
    for base in (0, 40, 100):
        slots.copy_(torch.arange(base, base + T, dtype=torch.int32))
        k.copy_(_rand((T, H, D), torch.bfloat16, 13 + base))
        g.replay()
        torch.cuda.synchronize()
        codes, bytes_ = attn_ref.encode(k)
        at = slots.long()
        assert torch.equal(cache.k.view(torch.uint8)[at // P, :, at % P].cpu(), codes)
        assert torch.equal(cache.k_scale[at // P, :, at % P].cpu(), bytes_)
        assert torch.equal(ok.double(), attn_ref.values(cache, "k")[at // P, :, at % P])


@pytest.mark.parametrize("kind", [torch.bfloat16, F8])
def test_many_rows(kind):
    """More rows than one wave of CTAs, every one checked through the inverse."""
    H, P, D, T = 8, 64, 128, 20000
    cache = gbe.kv_cache(-(-T // P), H, P, D, kind)
    k, v = _rand((T, H, D), torch.bfloat16, 14), _rand((T, H, D), torch.bfloat16, 15)
    slots = torch.randperm(T, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    gbe.gbe_kv_write(k, v, slots, cache)
    gk, gv = gbe.kv_read(cache, slots)
    if kind == F8:
        for got, want in ((gk, k), (gv, v)):
            codes, bytes_ = attn_ref.encode(want)
            y = codes.view(F8).double() * torch.exp2(bytes_.double() - 127.0)[..., None]
            assert torch.equal(got.cpu().double(), y)
    else:
        assert torch.equal(gk, k) and torch.equal(gv, v)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 1])
def test_a_cache_of_the_rows_type_holds_every_bit(dtype, pad):
    """Infinities, signed zeros and NaN of any payload, on and off the 16-byte grid."""
    T, H, D, P = 40, 2, 64, 16
    es = torch.empty((), dtype=dtype).element_size()
    raw = torch.randint(0, 256, (T, (2 * H * D + pad) * es), generator=torch.Generator().manual_seed(3),
                        dtype=torch.uint8).cuda().view(dtype)
    raw[:, ::7] = float("nan")
    raw.view(torch.uint8)[:, 1::13] = 0xFF
    k, v = raw[:, :H * D].unflatten(1, (H, D)), raw[:, H * D:2 * H * D].unflatten(1, (H, D))
    cache = gbe.kv_cache(4, H, P, D, dtype)
    slots = torch.randperm(4 * P, generator=torch.Generator().manual_seed(4))[:T].to(torch.int32).cuda()
    gbe.gbe_kv_write(k, v, slots, cache)
    out = torch.zeros_like(raw)
    ok, ov = out[:, :H * D].unflatten(1, (H, D)), out[:, H * D:2 * H * D].unflatten(1, (H, D))
    gbe.gbe_kv_read(ok, ov, slots, cache)
    assert torch.equal(_bytes(ok), _bytes(k)) and torch.equal(_bytes(ov), _bytes(v))


@pytest.mark.parametrize("H,P", [(7, 11), (1, 1), (12, 100), (64, 16), (3, 4096)])
def test_odd_heads_and_pages(H, P):
    """Counts that are no powers of two, and pages larger than the batch."""
    T, D = 333, 32
    pages = -(-T // P) + 1
    cache = gbe.kv_cache(pages, H, P, D, torch.bfloat16)
    k, v = _rand((T, H, D), torch.bfloat16, 21), _rand((T, H, D), torch.bfloat16, 22)
    slots = torch.randperm(pages * P, generator=torch.Generator().manual_seed(2))[:T].to(torch.int32).cuda()
    _check_write(cache, k, v, slots)
    gk, gv = gbe.kv_read(cache, slots)
    assert torch.equal(gk, k) and torch.equal(gv, v)
