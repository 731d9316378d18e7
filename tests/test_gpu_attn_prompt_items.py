"""gbe_attn_prompt on the tensor cores where a CTA takes many pieces of work,
some of two tiles and some of one: odd numbers of heads to a kv head, and
sequences of an odd number of row tiles, packed by the hundred.  Every row
against the same sequences in small calls, bit for bit, and against the
definition."""
import math

import pytest
import torch

import attn_ref
import elementwise_row_rmsnorm_gb300 as gbe

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _rand(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def _lens(kind):
    g = torch.Generator().manual_seed(9)
    return {"ones": [1] * 1500, "tiles": [[1, 130, 100, 257, 128, 300][i % 6] for i in range(120)],
            "any": torch.randint(1, 500, (128,), generator=g).tolist(),
            "short": torch.randint(1, 60, (900,), generator=g).tolist()}[kind]


@pytest.mark.parametrize("Hq,H,D", [(3, 1, 128), (5, 1, 64), (8, 8, 128), (7, 1, 64), (6, 2, 72), (21, 7, 128), (12, 4, 64)])
@pytest.mark.parametrize("kind", ["ones", "tiles", "any", "short"])
def test_many_items_of_one_and_two_tiles(Hq, H, D, kind):
    lens = _lens(kind)
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    q, k, v = (_rand((starts[-1], h, D), i) for i, h in enumerate((Hq, H, H)))
    scale = 1.0 / math.sqrt(D)
    where = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out = gbe.attn_prompt(q, k, v, where, scale)
    for _ in range(5):
        assert torch.equal(gbe.attn_prompt(q, k, v, where, scale), out), "the same bits every time"
    if kind == "ones":
        assert torch.equal(out, v.repeat_interleave(Hq // H, 1))
        return
    small = torch.empty_like(q)  # few enough sequences that a CTA has one piece of work
    per = 4
    for b in range(0, len(lens), per):
        part = slice(starts[b], starts[min(b + per, len(lens))])
        at = [s - starts[b] for s in starts[b:b + per + 1]]
        for h in range(H):
            hs = slice(h * Hq // H, (h + 1) * Hq // H)
            small[part, hs] = gbe.attn_prompt(q[part, hs], k[part, h:h + 1], v[part, h:h + 1],
                                              torch.tensor(at, dtype=torch.int32, device="cuda"), scale)
    assert torch.equal(out, small)
    for b in range(0, len(lens), max(1, len(lens) // 12)):
        s = slice(starts[b], starts[b + 1])
        want, tol, _ = attn_ref.prompt(q[s], k[s], v[s], [0, lens[b]], scale, True)
        attn_ref.assert_within(out[s], want, tol, f"sequence {b} of {lens[b]}")
