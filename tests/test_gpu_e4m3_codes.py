"""e4m3 caches whose codes or scale bytes are unusual: rows with a scale byte
of 0 stand for zeros whatever their codes hold, NaN codes of other rows reach
what attends to them and nothing else."""
import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

F8, BF, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
P, H, Hq, N = 16, 2, 8, 600


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _cache(D, dtype, seed=1):
    """N stored tokens in pages 0, 1, 2, ...: slot t holds token t."""
    cache = gbe.kv_cache(40, H, P, D, F8)
    gbe.gbe_kv_write(_rand((N, H, D), dtype, seed), _rand((N, H, D), dtype, seed + 1),
                     torch.arange(N, dtype=torch.int32, device="cuda"), cache)
    return cache


def _copy(c):
    return gbe.KvCache(*(t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)))


def _empty_rows(cache, which, tokens, head, codes):
    """Scale byte 0 for those tokens' rows, and these codes in them."""
    x, s = getattr(cache, which).view(torch.uint8), getattr(cache, which + "_scale")
    for i, t in enumerate(tokens):
        x[t // P, head, t % P] = codes[i % len(codes)]
        s[t // P, head, t % P] = 0


CODES = [0x7F, 0xFF, 0x7E, 0xFE, 0x01, 0x80, 0x38]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 64, 72, 80, 128, 136, 256])
def test_rows_of_scale_byte_0_are_zeros(dtype, D):
    cache = _cache(D, dtype)
    clean = _copy(cache)
    for c, codes in ((cache, CODES), (clean, [0])):
        _empty_rows(c, "k", [0, 5, 17, 31, 32, 100, 511, 512, 599], 0, codes)
        _empty_rows(c, "v", [0, 6, 16, 17, 130, 513, 598], 0, codes)
        _empty_rows(c, "v", list(range(300, 340)), 1, codes)   # whole steps
        _empty_rows(c, "k", list(range(320, 400)), 1, codes)
    slots = torch.arange(N, dtype=torch.int32, device="cuda")
    for got, want in zip(gbe.kv_read(cache, slots, dtype), gbe.kv_read(clean, slots, dtype)):
        assert torch.equal(got, want)
    k, v = gbe.kv_read(cache, slots, dtype)
    assert bool((k[[0, 5, 599], 0] == 0).all()) and bool((v[300:340, 1] == 0).all())
    table = torch.arange(38, dtype=torch.int32, device="cuda")[None].repeat(4, 1)
    lens = [N, 1, 18, 340]
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = _rand((4, Hq, D), dtype, 7)
    got = gbe.attn_decode(q, cache, table, lens_t, 0.2)
    assert torch.equal(got, gbe.attn_decode(q, clean, table, lens_t, 0.2))
    want, tol = attn_ref.decode(q, clean, table, lens, 0.2, dtype == BF)
    attn_ref.assert_within(got, want, tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_cache_of_uninitialised_codes_and_zeroed_scales(dtype):
    """Every byte pattern as codes: nothing but zeros, and the mean of zeros."""
    D = 128
    cache = gbe.kv_cache(8, H, P, D, F8)
    for t in (cache.k, cache.v):
        t.view(torch.uint8).copy_(torch.arange(t.numel(), device="cuda").view(t.shape).to(torch.uint8))
    slots = torch.arange(8 * P, dtype=torch.int32, device="cuda")
    for x in gbe.kv_read(cache, slots, dtype):
        assert bool((x == 0).all())
    out = gbe.attn_decode(_rand((1, Hq, D), dtype, 3), cache, torch.arange(8, dtype=torch.int32, device="cuda")[None],
                          torch.tensor([100], dtype=torch.int32, device="cuda"))
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 72, 128, 256])
def test_nan_codes_in_attended_places(dtype, D):
    cache = _cache(D, dtype, 11)
    k8, v8 = cache.k.view(torch.uint8), cache.v.view(torch.uint8)
    k8[77 // P, 0, 77 % P, 5] = 0x7F       # a NaN logit: every entry of head 0's rows from 78 tokens on
    v8[200 // P, 1, 200 % P, 3] = 0xFF     # one entry of head 1's rows from 201 tokens on
    cache.v_scale[150 // P, 1, 150 % P] -= 30  # and a scale far below its neighbours'
    table = torch.arange(38, dtype=torch.int32, device="cuda")[None].repeat(4, 1)
    lens = [77, 78, 200, 600]
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = _rand((4, Hq, D), dtype, 13)
    got = gbe.attn_decode(q, cache, table, lens_t, 0.1)
    k8[77 // P, 0, 77 % P, 5] = 0
    v8[200 // P, 1, 200 % P, 3] = 0
    want, tol = attn_ref.decode(q, cache, table, lens, 0.1, dtype == BF)
    g = Hq // H
    attn_ref.assert_within(got[0], want[0], tol[0])
    assert bool(got[1:, :g].isnan().all())
    attn_ref.assert_within(got[1:3, g:], want[1:3, g:], tol[1:3, g:])
    assert bool(got[3, g:, 3].isnan().all())
    rest = torch.arange(D, device="cuda") != 3
    attn_ref.assert_within(got[3, g:][:, rest], want[3, g:][:, rest], tol[3, g:][:, rest])
