"""What a call reads it leaves as it was: queries, keys, values, the cache, tables,
lengths, starts, slots and positions, copied before the call and compared after."""
import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe
from chunk_ref import filled, i32, rand

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
KINDS = [(F32, F32), (F32, F8), (BF, BF), (BF, F8)]


def _bytes(t):
    return t.contiguous().view(torch.uint8).clone()


def _held(call, *tensors):
    before = [_bytes(t) for t in tensors if t is not None]
    call()
    torch.cuda.synchronize()
    for i, (t, was) in enumerate(zip([t for t in tensors if t is not None], before)):
        assert torch.equal(_bytes(t), was), i


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_attention_over_the_cache(dtype, kind):
    new, lens, Hq, H, D, P = [9, 1, 40], [3000, 70, 200], 8, 2, 64, 16
    cache, table = filled(lens, P, H, D, dtype, kind, 1)
    table[2, 3] = -1
    q, starts, n = rand((50, Hq, D), dtype, 2), i32([0, 9, 10, 50]), i32(lens)
    held = q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, starts, n
    for window, sinks in ((0, 0), (50, 3)):
        _held(lambda: gbe.attn_chunk(q, cache, starts, table, n, 0.1, window, sinks), *held)
        _held(lambda: gbe.attn_decode_window(q[:3], cache, table, n, window, sinks, 0.1), *held)


@pytest.mark.parametrize("dtype,kind", [(F32, F32), (BF, BF)])
def test_attention_with_an_odd_value_among_the_attended(dtype, kind):
    for which, value in (("v", float("inf")), ("k", float("nan")), ("k", float("-inf"))):
        cache, table = filled([200], 16, 1, 64, dtype, kind, 72)
        getattr(cache, which)[int(table[0, 3]), 0, 2] = value
        q, starts, n = rand((2, 3, 64), dtype, 73), i32([0, 2]), i32([200])
        _held(lambda: gbe.attn_chunk(q, cache, starts, table, n, 0.1), q, cache.k, cache.v, table, starts, n)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompts(dtype):
    q, k, v = (rand((300, h, 64), dtype, 5 + i) for i, h in enumerate((4, 2, 2)))
    starts = i32([0, 130, 300])
    for window in (0, 40):
        _held(lambda: gbe.attn_prompt_window(q, k, v, starts, window, 2, 0.1), q, k, v, starts)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_append(dtype, kind):
    T, Hq, H, D = 33, 4, 2, 64
    q, k, v = (rand((T, h, D), dtype, 9 + i) for i, h in enumerate((Hq, H, H)))
    cache = gbe.kv_cache(5, H, 16, D, kind)
    om = (10000.0 ** (-torch.arange(D // 2, device="cuda").double() * 2 / D)).float()
    pos, slots, out = torch.arange(T, dtype=torch.int32, device="cuda"), i32([-1, *range(3, T + 2)]), torch.empty_like(q)
    _held(lambda: gbe.gbe_rope_kv_write(q, out, k, v, pos, slots, cache, om, D), q, k, v, pos, slots, om)
    # what no slot names: rows 0 to 2, and from T + 2 on
    for x in (cache.k, cache.v):
        assert bool((x[0, :, :3].view(torch.uint8) == 0).all()) and bool((x[3:].view(torch.uint8) == 0).all())
        assert bool((x[2, :, T + 2 - 32:].view(torch.uint8) == 0).all())
