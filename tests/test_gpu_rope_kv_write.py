"""gbe_rope_kv_write on the GPU: bit for bit what gbe_rope_qk followed by
gbe_kv_write leaves, in q_out and in every byte of the cache, and the
definition in 64 bits."""
import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import i32, rand

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
KINDS = [(F32, F32), (F32, F8), (BF, BF), (BF, F8)]


def _om(r):
    return (10000.0 ** (-torch.arange(r // 2, device="cuda").double() * 2 / max(r, 1))).float()


def _poisoned(n, H, P, D, kind):
    cache = gbe.kv_cache(n, H, P, D, kind)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).fill_(0x5A)
    if kind == F8:
        cache.k_scale.fill_(7)
        cache.v_scale.fill_(9)
    return cache


def _bytes(cache):
    return [t.view(torch.uint8) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]


def _both(q, k, v, pos, slots, cache, om, r, mu, layout, table=None, in_place=False):
    """(q_out, cache, bad) of the two calls, and of the one."""
    other = gbe.KvCache(*(None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
    bad = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    q2, k2 = q.clone(), k.clone()
    gbe.gbe_rope_qk(q2, q2, k2, k2, pos, om, r, mu, layout, table)
    gbe.gbe_kv_write(k2, v, slots, other, bad[0])
    span = (q.shape[0] - 1) * q.stride(0) + q.shape[1] * q.shape[2]
    qo = q if in_place else torch.full((span,), float("nan"), dtype=q.dtype, device="cuda").as_strided(q.shape, q.stride())
    gbe.gbe_rope_kv_write(q, qo, k, v, pos, slots, cache, om, r, mu, layout, table, bad[1])
    return (q2, other, bad[0]), (qo, cache, bad[1])


def _assert_same(two, one):
    assert torch.equal(two[0].contiguous().view(torch.uint8), one[0].contiguous().view(torch.uint8)), "q"
    for i, (x, y) in enumerate(zip(_bytes(two[1]), _bytes(one[1]))):
        assert torch.equal(x, y), ("k", "v", "k_scale", "v_scale")[i]
    assert int(two[2]) == int(one[2]), "bad slots"


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D,r", [(128, 128), (128, 64), (64, 32), (72, 72), (72, 36), (80, 80), (96, 48), (8, 8), (8, 2),
                                 (256, 256), (248, 48), (40, 0), (136, 130)])
def test_equals_the_two_calls(dtype, kind, layout, D, r):
    T, Hq, H, P = 37, 5, 2, 16
    q, k, v = rand((T, Hq, D), dtype, 1, 3.0), rand((T, H, D), dtype, 2, 3.0), rand((T, H, D), dtype, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(5 * P, generator=g, device="cuda")[:T].to(torch.int32)
    _assert_same(*_both(q, k, v, pos, slots, _poisoned(5, H, P, D, kind), _om(r), r, 1.25, layout))


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("T,Hq,H,P", [(1, 1, 1, 1), (1, 32, 8, 64), (2000, 32, 8, 64), (333, 7, 7, 48), (4097, 4, 1, 100),
                                      (65, 40, 1, 16), (130, 0, 3, 16), (3, 9, 130, 16)])
def test_head_counts_and_lengths(dtype, kind, T, Hq, H, P):
    """Slices of one fused projection, rotated in place."""
    D, r = 64, 64
    fused = rand((T, Hq + 2 * H, D), dtype, 11, 2.0)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
    n = -(-T // P) + 2
    g = torch.Generator(device="cuda").manual_seed(12)
    slots = torch.randperm(n * P, generator=g, device="cuda")[:T].to(torch.int32)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    cache = _poisoned(n, H, P, D, kind)
    if Hq == 0:
        other = gbe.KvCache(*(None if t is None else t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)))
        k2 = k.clone()
        gbe.gbe_rope_qk(None, None, k2, k2, pos, _om(r), r)
        gbe.gbe_kv_write(k2, v, slots, other)
        gbe.gbe_rope_kv_write(None, None, k, v, pos, slots, cache, _om(r), r)
        assert all(torch.equal(x, y) for x, y in zip(_bytes(other), _bytes(cache)))
        return
    before = fused.clone()
    _assert_same(*_both(q, k, v, pos, slots, cache, _om(r), r, 1.0, 0, in_place=True))
    assert torch.equal(fused[:, Hq:], before[:, Hq:]), "k and v are not changed"


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_padding_bad_slots_and_a_table_of_angles(dtype, kind):
    T, Hq, H, D, P, r = 40, 4, 2, 128, 16, 128
    q, k, v = rand((T, Hq, D), dtype, 21), rand((T, H, D), dtype, 22), rand((T, H, D), dtype, 23)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    slots[3], slots[9], slots[10], slots[11] = -1, -2, 4 * P, 2 ** 31 - 1
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3  # some past the table's end
    om = _om(r)
    table = gbe.rope_cos_sin(om, r, 60)
    two, one = _both(q, k, v, pos, slots, _poisoned(4, H, P, D, kind), om, r, 1.0, 0, table)
    _assert_same(two, one)
    assert int(one[2]) == 3
    plain = torch.empty_like(q)
    gbe.gbe_rope_kv_write(q, plain, k, v, pos, slots, one[1], om, r)
    assert torch.equal(plain, one[0]), "with and without the table"


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("r", [64, 36])
def test_infinities_nan_zeros_and_large_rows(dtype, kind, r):
    T, Hq, H, D, P = 24, 2, 2, 64, 16
    q, k, v = rand((T, Hq, D), dtype, 31), rand((T, H, D), dtype, 32), rand((T, H, D), dtype, 33)
    for x in (k, v):
        x[0, 0, 5] = float("inf")
        x[1, 0, 33] = float("nan")
        x[2] = 0.0
        x[3] = 1e30
        x[4, 1] = -3.3e38
        x[5] = 1e-40
        x[6, 0, :] = float("nan")
        x[7, 1, 63] = float("-inf")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    for layout in (0, 1):
        two, one = _both(q, k, v, pos, slots, _poisoned(3, H, P, D, kind), _om(r), r, 1.0, layout)
        # a NaN's bits are not part of the definition where two NaN meet in a sum
        for which in ("k", "v"):
            x, y = attn_ref.values(two[1], which), attn_ref.values(one[1], which)
            assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0)), which
        for x, y in zip(_bytes(two[1])[2:], _bytes(one[1])[2:]):
            assert torch.equal(x, y), "scales"


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_off_the_grid(dtype, kind):
    """Operands that begin off the 16-byte grid, or whose tokens do, give the same bits."""
    T, Hq, H, D, P, r = 19, 3, 2, 64, 16, 64
    wide = rand((T, (Hq + 2 * H) * D + 1), dtype, 41)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    slots = torch.arange(T, dtype=torch.int32, device="cuda")

    def cut(first, n): return wide[:, first * D + 1:(first + n) * D + 1].unflatten(1, (n, D))

    two, one = _both(cut(0, Hq), cut(Hq, H), cut(Hq + H, H), pos, slots, _poisoned(2, H, P, D, kind), _om(r), r, 1.0, 0)
    _assert_same(two, one)
    a = one[0].contiguous()
    cache = _poisoned(2, H, P, D, kind)
    out = torch.empty(T, Hq, D, dtype=dtype, device="cuda")
    gbe.gbe_rope_kv_write(cut(0, Hq).contiguous(), out, cut(Hq, H).contiguous(), cut(Hq + H, H).contiguous(), pos, slots,
                          cache, _om(r), r)
    assert torch.equal(a, out) and all(torch.equal(x, y) for x, y in zip(_bytes(cache), _bytes(one[1])))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_against_the_definition(dtype):
    """In 64 bits of the angle that is the f32 product: the cosine's and the sine's few ulp (2^-21), three roundings of
    sums and products, and the result's own."""
    T, Hq, H, D, P, r = 50, 2, 1, 128, 16, 128
    q, k, v = rand((T, Hq, D), dtype, 51), rand((T, H, D), dtype, 52), rand((T, H, D), dtype, 53)
    g = torch.Generator(device="cuda").manual_seed(54)
    pos = torch.randint(0, 1 << 17, (T,), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    cache, out, om = _poisoned(4, H, P, D, dtype), torch.empty_like(q), _om(r)
    gbe.gbe_rope_kv_write(q, out, k, v, pos, slots, cache, om, r)
    kk, vv = gbe.kv_read(cache, slots)
    assert torch.equal(vv, v)
    theta = (pos.float()[:, None] * om).double()[:, None]
    for x, y in ((q, out), (k, kk)):
        a, b = x.double()[..., :64], x.double()[..., 64:]
        want = torch.cat([a * theta.cos() - b * theta.sin(), a * theta.sin() + b * theta.cos()], -1)
        size = torch.hypot(a, b).repeat(1, 1, 2)
        step = 2.0 ** -8 if dtype == BF else 2.0 ** -24
        assert bool(((y.double() - want).abs() <= size * 2.0 ** -21 + want.abs() * step).all())


def test_captured_and_on_another_stream():
    T, Hq, H, D, P = 70, 8, 2, 128, 64
    q, k, v = rand((T, Hq, D), BF, 61), rand((T, H, D), BF, 62), rand((T, H, D), BF, 63)
    pos, slots, om = (torch.arange(T, dtype=torch.int32, device="cuda") for _ in range(2)), None, _om(D)
    pos, slots = pos
    want_q, want = torch.empty_like(q), _poisoned(2, H, P, D, F8)
    gbe.gbe_rope_kv_write(q, want_q, k, v, pos, slots, want, om, D)
    got_q, got = torch.empty_like(q), _poisoned(2, H, P, D, F8)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        gbe.gbe_rope_kv_write(q, got_q, k, v, pos, slots, got, om, D)
    for _ in range(2):
        got.k.view(torch.uint8).fill_(0x5A)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got_q, want_q) and all(torch.equal(x, y) for x, y in zip(_bytes(got), _bytes(want)))
    s = torch.cuda.Stream()
    got_q.zero_()
    s.wait_stream(torch.cuda.current_stream())
    gbe.gbe_rope_kv_write(q, got_q, k, v, pos, slots, got, om, D, stream=s)
    s.synchronize()
    assert torch.equal(got_q, want_q)


def test_outputs_stay_within_their_rows():
    """q_out's neighbours, and every slot that is not named, keep their bytes."""
    T, Hq, H, D, P = 33, 3, 2, 72, 16
    for dtype, kind in KINDS:
        wide = torch.full((T + 2, (Hq + 1) * D), 7.0, dtype=dtype, device="cuda")
        qo = wide[1:-1, :Hq * D].unflatten(1, (Hq, D))
        src = rand((T, (Hq + 1) * D), dtype, 71)
        q = src[:, :Hq * D].unflatten(1, (Hq, D))
        k, v = rand((T, H, D), dtype, 72), rand((T, H, D), dtype, 73)
        cache = _poisoned(6, H, P, D, kind)
        slots = torch.arange(1, 2 * T + 1, 2, dtype=torch.int32, device="cuda")
        gbe.gbe_rope_kv_write(q, qo, k, v, i32(list(range(T))), slots, cache, _om(64), 64)
        assert bool((wide[0] == 7).all()) and bool((wide[-1] == 7).all()) and bool((wide[:, Hq * D:] == 7).all())
        named = torch.zeros(6 * P, dtype=torch.bool, device="cuda")
        named[slots.long()] = True
        for t, fill in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (0x5A, 0x5A, 7, 9)):
            if t is None:
                continue
            t = t if t.dim() == 4 else t[..., None]
            rows = t.transpose(1, 2).reshape(6 * P, -1).view(torch.uint8)
            assert bool((rows[~named] == fill).all())
