"""gbe_attn_prompt on the GPU against the definition in 64 bits: types, head
layouts, packings of every shape, rows that no sequence holds, infinities and
NaN behind the mask, batch invariance, unaligned slices, graphs."""
import math

import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _qkv(T, Hq, H, D, dtype, seed, std=1.0, pad=0):
    """Columns of one fused buffer, `pad` elements off its start."""
    wide = _rand((T, (Hq + 2 * H) * D + pad), dtype, seed, std)
    return tuple(wide[:, pad + a * D:pad + z * D].unflatten(1, (z - a, D))
                 for a, z in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _check(q, k, v, starts, scale=None, what=""):
    scale = 1.0 / math.sqrt(q.shape[-1]) if scale is None else scale
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device="cuda")
    gbe.gbe_attn_prompt(q, k, v, out, _i32(starts), scale)
    want, tol, written = attn_ref.prompt(q, k, v, starts, scale, rounded=q.dtype == BF)
    attn_ref.assert_within(out[written], want[written], tol[written], what)
    assert bool((out[~written] == 3.0).all()), "rows of no sequence are left as they were"
    return out


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hq,H,D", [(1, 1, 8), (4, 1, 64), (6, 2, 72), (4, 4, 80), (8, 2, 128), (7, 1, 96), (2, 1, 256),
                                    (3, 1, 136), (5, 5, 120)])
@pytest.mark.parametrize("starts", [[0, 1], [0, 63, 64, 129, 129, 130, 386], [5, 6, 70, 300]])
def test_packings(dtype, Hq, H, D, starts):
    T = starts[-1] + (0 if starts[0] == 0 else 9)
    _check(*_qkv(T, Hq, H, D, dtype, 7), starts)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [2, 31, 64, 65, 127, 128, 129, 191, 255, 256, 257, 383, 384, 385, 511, 513, 640, 1025])
def test_lengths_around_the_tiles(dtype, n):
    _check(*_qkv(n, 4, 2, 128, dtype, n), [0, n])
    _check(*_qkv(n + 3, 2, 1, 64, dtype, n + 1), [3, n + 3])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_sequences(dtype):
    """More sequences than a warp has lanes, most of them short or empty."""
    lens = [(i * 37) % 50 if i % 3 else 0 for i in range(150)] + [200, 0, 1]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    _check(*_qkv(starts[-1] + 4, 4, 2, 64, dtype, 8), starts)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_sharp_flat_and_signed_logits(dtype):
    for std, scale in ((20.0, 0.125), (0.0, 0.125), (1.0, 0.0), (1.0, -0.5), (1e-3, 1e-6)):
        q, k, v = _qkv(300, 4, 2, 64, dtype, 9)
        _check((q * std).to(dtype), k, v, [0, 100, 300], scale, f"std {std} scale {scale}")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_growing_logits(dtype):
    """Every tile raises the running maximum, or lowers the logits far below it."""
    T = 900
    q, k, v = (x.contiguous() for x in _qkv(T, 2, 1, 128, dtype, 10))
    ramp = torch.linspace(-6.0, 6.0, T, device="cuda")[:, None, None]
    for sign in (1.0, -1.0):
        _check((q.abs() * 2).to(dtype), (k.abs() * sign * ramp).to(dtype), v, [0, T])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_what_is_masked_stays_where_it_is(dtype, D, what):
    """Bad numbers in k and v of later rows and of the next sequence: rows before them are as without them."""
    starts = [0, 200, 500]
    q, k, v = (x.contiguous() for x in _qkv(500, 4, 2, D, dtype, 11))
    clean = _check(q, k, v, starts)
    k2, v2 = k.clone(), v.clone()
    v2[150, 0, 3] = what       # within the first sequence
    v2[200:, 1] = what         # the whole second one, one head
    k2[170, 1] = float("nan")
    out = torch.empty_like(q)
    gbe.gbe_attn_prompt(q, k2, v2, out, _i32(starts), 1.0 / math.sqrt(D))
    want, tol, _ = attn_ref.prompt(q, k, v, starts, 1.0 / math.sqrt(D), dtype == BF)
    for rows, heads in ((slice(0, 150), slice(0, 2)), (slice(0, 170), slice(2, 4)), (slice(200, 500), slice(0, 2))):
        attn_ref.assert_within(out[rows, heads], want[rows, heads], tol[rows, heads], str(rows))
    assert torch.equal(out[:128], clean[:128]), "tiles without a bad number keep their bits"
    bad = out[150:200, 0:2]
    assert not bool(torch.isfinite(bad[..., 3]).any())
    rest = torch.arange(D, device="cuda") != 3
    attn_ref.assert_within(bad[..., rest], want[150:200, 0:2][..., rest], tol[150:200, 0:2][..., rest])
    assert bool(out[170:200, 2:4].isnan().all())
    assert not bool(torch.isfinite(out[200:, 2:4]).any())


@pytest.mark.parametrize("dtype", [F32, BF])
def test_a_sequence_has_the_same_bits_wherever_it_is_packed(dtype):
    n, Hq, H, D = 333, 4, 2, 128
    q, k, v = _qkv(n, Hq, H, D, dtype, 12)
    alone = gbe.attn_prompt(q, k, v, _i32([0, n]))
    for before, after in ((1, 0), (77, 200), (500, 3)):
        T = before + n + after
        pq, pk, pv = (x.contiguous() for x in _qkv(T, Hq, H, D, dtype, 13))
        for dst, src in ((pq, q), (pk, k), (pv, v)):
            dst[before:before + n] = src
        out = gbe.attn_prompt(pq, pk, pv, _i32([0, before, before + n, T]))
        assert torch.equal(out[before:before + n], alone), (before, after)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 72, 128])
def test_rows_off_the_16_byte_grid(dtype, D):
    q, k, v = _qkv(200, 4, 2, D, dtype, 14, pad=1)
    out = torch.full((200, 4 * D + 3), 3.0, dtype=dtype, device="cuda")
    o = out[:, 1:1 + 4 * D].unflatten(1, (4, D))
    gbe.gbe_attn_prompt(q, k, v, o, _i32([0, 90, 200]), 0.1)
    want, tol, _ = attn_ref.prompt(q, k, v, [0, 90, 200], 0.1, dtype == BF)
    attn_ref.assert_within(o, want, tol)
    assert bool((out[:, 0] == 3.0).all()) and bool((out[:, 1 + 4 * D:] == 3.0).all())


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("starts", [[-5, 40, 100], [0, 60, 1000], [0, 80, 40, 100], [100, 0], [2 ** 31 - 1, -2 ** 31]])
def test_starts_out_of_range_reach_no_other_memory(dtype, starts):
    """Entries outside [0, T] are brought into it, a sequence that ends before it begins is empty."""
    T, Hq, D = 100, 2, 64
    q, k, v = _qkv(T, Hq, 1, D, dtype, 15)
    raw = torch.full((T + 200, Hq, D), 3.0, dtype=dtype, device="cuda")
    gbe.gbe_attn_prompt(q, k, v, raw[100:100 + T], _i32(starts), 0.125)
    torch.cuda.synchronize()
    assert bool((raw[:100] == 3.0).all()) and bool((raw[100 + T:] == 3.0).all())


@pytest.mark.parametrize("dtype,T", [(F32, 2000), (BF, 5000)])
def test_a_long_prompt(dtype, T):
    """Llama-3-8B's heads; a sample of the heads against the definition."""
    Hq, H, D = 32, 8, 128
    q, k, v = _qkv(T, Hq, H, D, dtype, 16, 1.2)
    out = gbe.attn_prompt(q, k, v, _i32([0, T]))
    for h in (0, 13, 31):
        want, tol, _ = attn_ref.prompt(q[:, h:h + 1], k[:, h // 4:h // 4 + 1], v[:, h // 4:h // 4 + 1], [0, T],
                                       1.0 / math.sqrt(D), dtype == BF)
        attn_ref.assert_within(out[:, h:h + 1], want, tol, f"head {h}")


@pytest.mark.parametrize("dtype", [F32, BF])
def test_graph_replay_reads_the_starts_of_the_moment(dtype):
    T, Hq, H, D = 400, 4, 2, 128
    q, k, v = (x.contiguous() for x in _qkv(T, Hq, H, D, dtype, 17))
    starts, out = _i32([0, 400, 400]), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        gbe.gbe_attn_prompt(q, k, v, out, starts, 0.1)
    for s in ([0, 400, 400], [0, 1, 400], [0, 150, 300]):
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        q.copy_(_rand((T, Hq, D), dtype, s[1]))
        g.replay()
        torch.cuda.synchronize()
        want, tol, written = attn_ref.prompt(q, k, v, s, 0.1, dtype == BF)
        attn_ref.assert_within(out[written], want[written], tol[written], str(s))


def test_two_streams_at_once():
    a, b = _qkv(700, 8, 2, 128, BF, 18), _qkv(650, 8, 2, 128, BF, 19)
    want = [gbe.attn_prompt(*x, _i32([0, x[0].shape[0]])) for x in (a, b)]
    starts = [_i32([0, x[0].shape[0]]) for x in (a, b)]
    outs = [[torch.empty_like(x[0]) for _ in range(4)] for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(4):
        for j, x in enumerate((a, b)):
            gbe.gbe_attn_prompt(*x, outs[j][i], starts[j], 1.0 / math.sqrt(128), stream=streams[j])
    torch.cuda.synchronize()
    for j in range(2):
        for o in outs[j]:
            assert torch.equal(o, want[j])


@pytest.mark.parametrize("dtype,pad", [(F32, 0), (F32, 1), (BF, 1)])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_a_sequence_has_the_same_bits_in_a_large_call(dtype, pad, D):
    """Large calls may cut the rows otherwise than small ones (rows off the 16-byte grid: bf16 without tensor cores)."""
    n, Hq, H, before, T = 333, 8, 2, 4000, 5200
    q, k, v = _qkv(n, Hq, H, D, dtype, 31, pad=pad)
    alone = gbe.attn_prompt(q, k, v, _i32([0, n]))
    pq, pk, pv = _qkv(T, Hq, H, D, dtype, 32, pad=pad)
    for dst, src in ((pq, q), (pk, k), (pv, v)):
        dst[before:before + n] = src
    starts = [0, 150, before, before + n, T]
    out = gbe.attn_prompt(pq, pk, pv, _i32(starts))
    assert torch.equal(out[before:before + n], alone)
    part = slice(before + n, T)
    want, tol, _ = attn_ref.prompt(pq[part], pk[part], pv[part], [0, T - before - n], 1.0 / math.sqrt(D), False)
    attn_ref.assert_within(out[part], want, tol)
