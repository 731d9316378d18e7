"""The paged cache and attention evaluated in 64 bits, and how far a result
may be from it.

Tolerances.  With p the weights and v the values of one row, write
A = sum_j p_j |v_j| for an output entry.  The computed weights differ from the
exact ones by a relative

    2 * delta  from the logits: every product sum of D terms is within
               (D + 4) u * scale * sum_d |q_d k_d| of the exact one (f32
               accumulation, u = 2^-24, and the roundings of the scale and of
               the exponential's argument), in the weight and in the sum that
               normalises it; doubled once more for the change to base 2;
    2^-20      from the exponential (2 ulp of ex2.approx) and the rescalings;
    n u        from adding n terms in f32, in the sum and in the output;
    2^-8       where weights are rounded to bf16 before the product

and the result is rounded once: 2^-8 |out| in bf16, 2^-24 |out| in f32.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24


def e4m3_values() -> torch.Tensor:
    """The 127 non-negative e4m3 numbers in code order (0 .. 448)."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def encode(x: torch.Tensor):
    """(codes uint8, scale bytes uint8) of rows x[..., D], by search in the table of e4m3 numbers."""
    x = x.detach().cpu().double()
    finite = torch.isfinite(x)
    largest = torch.where(finite, x.abs(), 0.0).amax(-1)
    e = torch.full(largest.shape, -126, dtype=torch.int64)
    for k in range(-126, 122):  # the least power that brings the largest to 448
        e = torch.where(largest > 448.0 * 2.0 ** k, k + 1, e)
    y = torch.where(finite, x, 0.0).abs() / torch.exp2(e.double())[..., None]
    y = torch.where((e == 120)[..., None], y.clamp(max=240.0), y)  # 256 * 2^120 is past f32's range
    table = e4m3_values()
    hi = torch.searchsorted(table, y.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = table[hi] - y, y - table[lo]
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(y == table[hi], hi, code)
    code = code + torch.where(torch.signbit(x), 128, 0)
    code = torch.where(finite, code, 127)
    return code.to(torch.uint8), (e + 127).to(torch.uint8)


def values(cache, which: str) -> torch.Tensor:
    """k or v of a KvCache in 64 bits, [n_pages, Hkv, page_size, D] on its device."""
    x = getattr(cache, which)
    s = getattr(cache, which + "_scale")
    y = x.double()
    if s is not None:
        y = y * torch.where(s == 0, 0.0, torch.exp2(s.double() - 127.0))[..., None]
    return y


def _attend(q, k, v, scale, rounded, out_round):
    """q [m, D], k, v [n, D] in 64 bits, all attended: (out, tolerance)."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        return z, z
    logits = q @ k.T * scale
    p = torch.softmax(logits, -1)
    out = p @ v
    spread = abs(scale) * (q.abs() @ k.abs().T).amax(-1, keepdim=True)
    rel = 4 * (q.shape[1] + 4) * U * spread + k.shape[0] * U + 2.0 ** -20 + (2.0 ** -8 if rounded else 0.0)
    return out, (p @ v.abs()) * rel + out.abs() * out_round + 1e-30


def decode(q, cache, table, lens, scale, rounded=False):
    """(out, tolerance) of gbe_attn_decode, [B, Hq, D] in 64 bits."""
    N, H, P, D = cache.shape
    B, Hq, _ = q.shape
    k, v = values(cache, "k"), values(cache, "v")
    group = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    step = 2.0 ** -8 if q.dtype == torch.bfloat16 else U
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * P)
        t = torch.arange(n, device=q.device)
        page = table[b].long()[t // P] if n else t
        good = (page >= 0) & (page < N)
        page, row = page[good], (t % P)[good]
        for h in range(H):
            kk, vv = k[page, h, row], v[page, h, row]
            hs = slice(h * group, (h + 1) * group)
            out[b, hs], tol[b, hs] = _attend(q[b, hs].double(), kk, vv, scale, rounded, step)
    return out, tol


def prompt(q, k, v, starts, scale, rounded=False):
    """(out, tolerance, written) of gbe_attn_prompt; written: which rows it covers."""
    T, Hq, D = q.shape
    group = Hq // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    written = torch.zeros(T, dtype=torch.bool, device=q.device)
    step = 2.0 ** -8 if q.dtype == torch.bfloat16 else U
    starts = [min(max(int(s), 0), T) for s in starts]
    for a, z in zip(starts, starts[1:]):
        if z <= a:
            continue
        written[a:z] = True
        n = z - a
        later = torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1)
        for h in range(Hq):
            qq, kk, vv = q[a:z, h].double(), k[a:z, h // group].double(), v[a:z, h // group].double()
            s = (qq @ kk.T * scale).masked_fill(later, -math.inf)
            p = torch.softmax(s, -1)
            spread = (abs(scale) * (qq.abs() @ kk.abs().T)).masked_fill(later, 0.0).amax(-1, keepdim=True)
            rel = 4 * (D + 4) * U * spread + n * U + 2.0 ** -20 + (2.0 ** -8 if rounded else 0.0)
            o = p @ vv
            out[a:z, h], tol[a:z, h] = o, (p @ vv.abs()) * rel + o.abs() * step + 1e-30
    return out, tol, written


def assert_within(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} entries off; first at {i}: got {float(got[i])}, "
                             f"want {float(want[i])} within {float(tol[i])}; worst ratio "
                             f"{float((err / tol.clamp_min(1e-300)).nan_to_num(1e300).max())}")


def make_table(lens, page, n_pages, seed, spare=0):
    """int32 [B, max_pages] of distinct pages in random order; entries past a sequence's last page are garbage."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // page) for n in lens]
    order = torch.randperm(n_pages, generator=g).tolist()
    assert sum(need) <= n_pages
    table = torch.full((len(lens), max(1, max(need) + spare)), 1 << 30, dtype=torch.int32)
    table[:, ::2] = -9
    for b, m in enumerate(need):
        for i in range(m):
            table[b, i] = order.pop()
    return table
