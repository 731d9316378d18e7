"""gbe_attn_prompt: a sequence's bits are its own, whatever the rows around it
hold -- infinities and NaN in the sequences before and behind it and in rows
that no sequence holds, at every length around the products' borders."""
import math

import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _same_bits(a, b):
    """Equal entries, NaN where the other has one."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(7.0, INF, -INF), b.nan_to_num(7.0, INF, -INF))


def _packed(x, before, after, what):
    T = before + x.shape[0] + after
    y = torch.full((T, *x.shape[1:]), what, dtype=x.dtype, device="cuda")
    y[before:before + x.shape[0]] = x
    return y


@pytest.mark.parametrize("dtype,D,Hq,H", [(BF, 128, 4, 2), (BF, 64, 4, 2), (BF, 72, 3, 1), (BF, 128, 2, 2), (BF, 136, 2, 1),
                                          (F32, 64, 4, 2), (F32, 128, 2, 1)])
@pytest.mark.parametrize("what", [NAN, INF, -INF])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 100, 112, 113, 127, 128, 129, 143, 255, 257, 300, 385])
def test_bad_rows_around_a_sequence(dtype, D, Hq, H, what, n):
    q, k, v = (_rand((n, h, D), dtype, i) for i, h in enumerate((Hq, H, H)))
    alone = gbe.attn_prompt(q, k, v, _i32([0, n]))
    want, tol, _ = attn_ref.prompt(q, k, v, [0, n], 1.0 / math.sqrt(D), dtype == BF)
    attn_ref.assert_within(alone, want, tol)
    for before, after in ((0, 1), (0, 130), (5, 9), (130, 0), (64, 200)):
        pq, pk, pv = (_packed(x, before, after, what) for x in (q, k, v))
        T = before + n + after
        # neighbours are sequences, and rows of none
        for starts in ([0, before, before + n, T], [before, before + n], [0, before, before + n, before + n]):
            out = torch.zeros_like(pq)
            gbe.gbe_attn_prompt(pq, pk, pv, out, _i32(starts), 1.0 / math.sqrt(D))
            assert torch.equal(out[before:before + n], alone), (before, after, starts)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("n", [20, 100, 200, 300])
def test_bad_rows_around_a_sequence_with_bad_rows_of_its_own(dtype, D, n):
    """Its own infinities and NaN, attended and masked, come out the same beside clean neighbours and bad ones."""
    Hq, H = 4, 2
    q, k, v = (_rand((n, h, D), dtype, 10 + i) for i, h in enumerate((Hq, H, H)))
    v[n // 2, 0, 3], v[n - 3, 1, 5], k[n // 3, 1, 2], q[n - 2, 0, 1] = NAN, INF, NAN, INF
    alone = gbe.attn_prompt(q, k, v, _i32([0, n]))
    assert bool(torch.isfinite(alone[:n // 3]).all()) and not bool(torch.isfinite(alone[n - 1]).all())
    for what in (0.5, NAN, INF):
        pq, pk, pv = (_packed(x, 40, 150, what) for x in (q, k, v))
        out = gbe.attn_prompt(pq, pk, pv, _i32([0, 40, 40 + n, 190 + n]))
        assert _same_bits(out[40:40 + n], alone), what


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences_between_bad_ones(dtype):
    """Every other sequence holds nothing but NaN; the others' bits are those of each alone."""
    Hq, H, D = 4, 2, 128
    lens = [1, 130, 7, 64, 33, 128, 250, 129, 16, 15, 17, 127, 400, 3, 96, 200, 1, 111]
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    q, k, v = (_rand((starts[-1], h, D), dtype, 20 + i) for i, h in enumerate((Hq, H, H)))
    for i in range(1, len(lens), 2):
        for x in (q, k, v):
            x[starts[i]:starts[i + 1]] = NAN
    out = gbe.attn_prompt(q, k, v, _i32(starts))
    for i in range(0, len(lens), 2):
        s = slice(starts[i], starts[i + 1])
        assert torch.equal(out[s], gbe.attn_prompt(q[s], k[s], v[s], _i32([0, lens[i]]))), lens[i]
        assert bool(torch.isfinite(out[s]).all())
    for i in range(1, len(lens), 2):
        assert bool(out[starts[i]:starts[i + 1]].isnan().all())
