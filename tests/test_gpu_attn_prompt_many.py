"""gbe_attn_prompt over thousands of packed sequences, most of them empty among
them: each one's bits are those that it has alone, rows of none are left as
they were, and the time to find the work does not grow with the square of
their number."""
import math

import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _lens(kind):
    g = torch.Generator().manual_seed(5)
    return {"ones": [1] * 3000, "short": torch.randint(0, 40, (2500,), generator=g).tolist(),
            "mixed": (torch.randint(0, 400, (129,), generator=g)).tolist() + [0] * 300 + [1200, 0, 1, 128, 129],
            "mostly empty": [n if i % 37 == 0 else 0 for i, n in enumerate(torch.randint(0, 90, (9000,),
                                                                                         generator=g).tolist())]}[kind]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,H,D", [(4, 2, 64), (3, 1, 128), (2, 2, 64), (7, 1, 72)])
@pytest.mark.parametrize("kind", ["ones", "short", "mixed", "mostly empty"])
def test_each_sequence_is_as_alone(dtype, Hq, H, D, kind):
    lens = _lens(kind)
    starts = [3]
    for n in lens:
        starts.append(starts[-1] + n)
    T = starts[-1] + 5
    q, k, v = (_rand((T, h, D), dtype, i) for i, h in enumerate((Hq, H, H)))
    out = torch.full_like(q, 9.0)
    scale = 1.0 / math.sqrt(D)
    gbe.gbe_attn_prompt(q, k, v, out, torch.tensor(starts, dtype=torch.int32, device="cuda"), scale)
    assert bool((out[:3] == 9.0).all()) and bool((out[T - 5:] == 9.0).all())
    # a hundred at a time: the few sequences' way of finding the work
    again = torch.full_like(q, 9.0)
    for b in range(0, len(lens), 100):
        part = torch.tensor(starts[b:b + 101], dtype=torch.int32, device="cuda")
        if starts[b] < starts[min(b + 100, len(lens))]:
            gbe.gbe_attn_prompt(q, k, v, again, part, scale)
    assert torch.equal(out, again)
    for b in [i for i, n in enumerate(lens) if n][::max(1, len(lens) // 40)]:
        s = slice(starts[b], starts[b + 1])
        want, tol, _ = attn_ref.prompt(q[s], k[s], v[s], [0, lens[b]], scale, dtype == BF)
        attn_ref.assert_within(out[s], want, tol, f"sequence {b} of {lens[b]}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n_seqs,T", [(1 << 20, 4096), (1 << 20, 1), (1 << 17, 1 << 17)])
def test_a_million_sequences(dtype, n_seqs, T):
    """One row to a sequence at most: its v.  Milliseconds; a search that walks the sequences for every piece of work
    would take minutes."""
    Hq, H, D = 4, 2, 64
    q, k, v = (_rand((T, h, D), dtype, i) for i, h in enumerate((Hq, H, H)))
    where = torch.randperm(n_seqs, generator=torch.Generator().manual_seed(6))[:T]
    size = torch.zeros(n_seqs + 1, dtype=torch.int64)
    size[where + 1] = 1
    starts = size.cumsum(0).to(torch.int32).cuda()
    gbe.attn_prompt(q[:1], k[:1], v[:1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    out = gbe.attn_prompt(q, k, v, starts)
    b.record()
    b.synchronize()
    assert torch.equal(out, v.repeat_interleave(Hq // H, 1))
    assert a.elapsed_time(b) < 500.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(dtype):
    """More than 2^31 entries of q and out, and as many bytes again behind column slices of one buffer."""
    Hq, H, D, n, seqs = 16, 1, 128, 400, 2700
    T = n * seqs
    wide = torch.empty((T, Hq + 2 * H, D), dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    for a in range(0, T, n * 100):  # (no temporaries of the whole)
        wide[a:a + n * 100] = torch.randn(wide[a:a + n * 100].shape, generator=g, device="cuda").to(dtype)
    q, k, v = wide[:, :Hq], wide[:, Hq:Hq + H], wide[:, Hq + H:]
    assert q.stride(0) * T > 2 ** 31
    starts = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    out = torch.full((T, Hq, D), 9.0, dtype=dtype, device="cuda")
    gbe.gbe_attn_prompt(q, k, v, out, starts, 0.1)
    one = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for b in (0, 1, seqs // 2, seqs - 800, seqs - 2, seqs - 1):
        s = slice(b * n, (b + 1) * n)
        assert torch.equal(out[s], gbe.attn_prompt(q[s], k[s], v[s], one, 0.1)), b
    s = slice(T - n, T)
    want, tol, _ = attn_ref.prompt(q[s], k[s], v[s], [0, n], 0.1, dtype == BF)
    attn_ref.assert_within(out[s], want, tol)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_starts_of_any_kind_reach_no_other_memory(dtype):
    """Hundreds of entries outside [0, T], going back and forth: nothing outside out is written."""
    T, Hq, H, D = 700, 3, 1, 64
    g = torch.Generator().manual_seed(8)
    q, k, v = (_rand((T, h, D), dtype, i) for i, h in enumerate((Hq, H, H)))
    for n in (129, 300, 1000):
        starts = torch.randint(-50, T + 50, (n + 1,), generator=g)
        starts[::17], starts[5::23] = 2 ** 31 - 1, -2 ** 31
        raw = torch.full((T + 400, Hq, D), 3.0, dtype=dtype, device="cuda")
        gbe.gbe_attn_prompt(q, k, v, raw[200:200 + T], starts.to(torch.int32).cuda(), 0.125)
        torch.cuda.synchronize()
        assert bool((raw[:200] == 3.0).all()) and bool((raw[200 + T:] == 3.0).all())
        assert bool(torch.isfinite(raw).all())
