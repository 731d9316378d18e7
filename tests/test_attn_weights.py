"""The bits that decode keeps of a softmax weight, where they show: values that
cancel, so that an entry is small beside the terms that it is the sum of and
its own rounding hides nothing.

Tolerance.  q and k hold small whole numbers, eight of them not zero, and the
scale is a power of two, so that sums of q k are exact in every order.  What is
left, relative to A = sum_j p_j |v_j|:

    weights   over a bf16 cache each is two bf16 numbers: the first cut off, so
              that less than 2^-7 of the weight is left (8 significant bits),
              the second rounded, 2^-8 of that: 2^-15.  Over an e4m3 cache
              each is one f16 number, 11 significant bits: 2^-11 (weights here
              stay far above its smallest normal one).  Over an f32 cache
              they are f32: 0.
    base 2    with L = log2(e) * scale * sum_d |q_d k_d| at most: log2(e), its
              product with the scale and that with the sum are rounded, 3 * 2^-24 L,
              and the difference to the maximum, 2^-24 * 2 L; for f32 queries the
              factor goes into q, and eight products and four sums of theirs
              are rounded, 12 * 2^-24 L.  Times ln 2 in the weight, and as much
              again in the sum that normalises it.
    2^-20     the exponential (2 ulp of ex2.approx) and the rescalings
    n 2^-24   the sums, of weights and of products, in f32, twice

and the result is rounded once, half a step of its type: 2^-8 |out| in bf16,
2^-24 |out| in f32."""
import math

import pytest
import torch

import elementwise_row_rmsnorm_gb300 as gbe

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SCALE = 0.25
WEIGHTS = {BF: 2.0 ** -15, F8: 2.0 ** -11, F32: 0.0}


def _cut(x, bits):
    """x of 64 bits, to `bits` significant ones, towards zero."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.trunc(m * 2.0 ** bits) / 2.0 ** bits, e)


def _round(x, bits):
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 2.0 ** bits) / 2.0 ** bits, e)


def _case(dtype, kind, n, D, heads, seed):
    """q [heads, D], k, v [n, D] in 64 bits, exact in `dtype` and in the cache's type: for every head a run of D / heads
    entries of v that nearly cancels, by way of the heaviest token."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-2, 3, (heads, D), generator=g).double()
    k = torch.randint(-1, 2, (n, D), generator=g).double()
    q[:, 8:] = 0.0  # logits of |16| * SCALE at most
    p = torch.softmax(q @ k.T * SCALE, -1)
    narrow = 4 if kind == F8 else 8 if dtype == BF or kind == BF else 24
    v = _round(torch.rand(n, D, generator=g, dtype=torch.float64) + 1.0, narrow) * torch.where(
        torch.rand(n, D, generator=g) < 0.5, 1.0, -1.0)
    for d in range(D):
        h = d * heads // D
        last = int(p[h].argmax())
        rest = (p[h] @ v[:, d]) - p[h, last] * v[last, d]
        v[last, d] = _round(-rest / p[h, last], narrow)
    if kind == F8:  # as values of a row with one power-of-two scale: codes of 4 bits down to 2^-6 of 2^8
        v = torch.where(v.abs() < 2.0 ** -8, 0.0, v)
    return q, k, v, p


def _bound(q, k, v, p, dtype, kind):
    n = k.shape[0]
    L = float((q.abs() @ k.abs().T).max()) * SCALE / math.log(2.0)
    base2 = 2.0 * math.log(2.0) * 2.0 ** -24 * L * (5 if dtype == BF else 17)
    rel = WEIGHTS[kind if dtype == BF else F32] + base2 + 2.0 ** -20 + 2 * n * 2.0 ** -24
    return (p @ v.abs()) * rel + (p @ v).abs() * (2.0 ** -8 if dtype == BF else 2.0 ** -24)


CASES = [(BF, BF), (BF, F8), (F32, F32), (F32, F8)]
SIZES = [(8, 64, 4), (40, 128, 8), (16, 72, 2), (700, 128, 4), (24, 256, 8)]


def _model(q, k, v, p, kind, loss):
    """The result with weights of `kind` as documented, or with less of them."""
    w = p / p.amax(-1, keepdim=True)
    if loss == "one bf16":
        w = _round(w, 8)
    elif loss == "cut":
        w = _cut(w, 8)
    elif kind == BF:
        first = _cut(w, 8)
        w = first + _round(w - first, 8)
    elif kind == F8:
        w = _round(w, 11)
    return w @ v / (p / p.amax(-1, keepdim=True)).sum(-1, keepdim=True)


@pytest.mark.parametrize("n,D,heads", SIZES)
@pytest.mark.parametrize("kind", [BF, F8])
def test_the_bound_tells_fewer_bits(kind, n, D, heads):
    """On the CPU: weights as documented are within the bound (their own part of it alone), the second bf16 left out
    or a bf16 in place of an f16 is not (of hundreds of tokens the roundings of f16 and bf16 both average out)."""
    q, k, v, p = _case(BF, kind, n, D, heads, 3)
    want, tol = p @ v, _bound(q, k, v, p, BF, kind)
    good = (_model(q, k, v, p, kind, None) - want).abs()
    assert bool((good <= (p @ v.abs()) * WEIGHTS[kind] * (1 + 1e-9)).all())
    for loss in ("one bf16", "cut") if kind == BF or n < 100 else ():
        bad = _model(q, k, v, p, kind, loss)
        bad = _round(bad, 8)  # stored as bf16
        assert bool(((bad - want).abs() > tol).any()), loss


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,kind", CASES)
@pytest.mark.parametrize("n,D,heads", SIZES)
def test_weights_keep_their_bits(dtype, kind, n, D, heads):
    for seed in range(3, 11):
        q, k, v, p = _case(dtype, kind, n, D, heads, seed)
        P = 16
        cache = gbe.kv_cache(-(-n // P), 1, P, D, kind)
        slots = torch.arange(n, dtype=torch.int32, device="cuda")
        kk, vv = (x[:, None].to(dtype).cuda() for x in (k, v))
        gbe.gbe_kv_write(kk, vv, slots, cache)
        back = gbe.kv_read(cache, slots, dtype)
        assert torch.equal(back[0], kk)
        v = back[1][:, 0].double().cpu()  # what the cache holds (of 8 bits: rows of one scale)
        table = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda")[None]
        got = gbe.attn_decode(q[None].to(dtype).cuda(), cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                              SCALE)[0].double().cpu()
        want, tol = p @ v, _bound(q, k, v, p, dtype, kind)
        err = (got - want).abs()
        assert bool((err <= tol).all()), (seed, float((err / tol).max()))
