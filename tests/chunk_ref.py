"""Attention of new rows behind a cached prefix, and under a sliding window,
evaluated in 64 bits; how far a result may be from it is derived in attn_ref.
(Splits that are joined add at most one rounding of a sum of n terms each, and
there are fewer of them than terms: n u covers them.)"""
from __future__ import annotations

import math

import torch

import attn_ref
from attn_ref import U


def sees(places, n, window, sinks, device="cpu"):
    """[m, n]: whether a row at each of the places sees each of the keys."""
    p = torch.as_tensor(places, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    ok = j <= p
    if window:
        ok = ok & ((j > p - window) | (j < sinks))
    return ok


def masked(q, k, v, ok, scale, rounded, step):
    """(out, tolerance) of rows q [m, D] that see the keys [n, D] where ok [m, n]; a row that sees none is zeros."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64, device=q.device)
        return z, z
    any_ = ok.any(-1, keepdim=True)
    k, v = torch.where(ok.any(0)[:, None], k, 0.0), torch.where(ok.any(0)[:, None], v, 0.0)
    s = (q @ k.T * scale).masked_fill(~ok, -math.inf)
    p = torch.where(any_, torch.softmax(torch.where(any_, s, 0.0), -1), 0.0)
    spread = (abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~ok, 0.0).amax(-1, keepdim=True)
    rel = 4 * (q.shape[1] + 4) * U * spread + k.shape[0] * U + 2.0 ** -20 + (2.0 ** -8 if rounded else 0.0)
    out = p @ v
    return out, (p @ v.abs()) * rel + out.abs() * step + 1e-30


def chunk(q, cache, starts, table, lens, scale, window=0, sinks=0, rounded=False):
    """(out, tolerance, written) of gbe_attn_chunk, [T, Hq, D] in 64 bits; written: which rows it covers."""
    N, H, P, D = cache.shape
    T, Hq, _ = q.shape
    kv = attn_ref.values(cache, "k"), attn_ref.values(cache, "v")
    group = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    written = torch.zeros(T, dtype=torch.bool, device=q.device)
    step = 2.0 ** -8 if q.dtype == torch.bfloat16 else U
    starts = [min(max(int(s), 0), T) for s in starts]
    for b, (a, z) in enumerate(zip(starts, starts[1:])):
        if z <= a:
            continue
        written[a:z] = True
        n = min(max(int(lens[b]), 0), table.shape[1] * P)
        t = torch.arange(n, device=q.device)
        page = table[b].long()[t // P] if n else t
        good = (page >= 0) & (page < N)
        ok = sees(range(n - (z - a), n), n, window, sinks, q.device)[:, good].repeat_interleave(group, 0)
        page, row = page[good], (t % P)[good]
        for h in range(H):
            hs = slice(h * group, (h + 1) * group)
            o, e = masked(q[a:z, hs].reshape(-1, D).double(), kv[0][page, h, row], kv[1][page, h, row], ok, scale,
                          rounded, step)
            out[a:z, hs], tol[a:z, hs] = o.view(z - a, group, D), e.view(z - a, group, D)
    return out, tol, written


def decode(q, cache, table, lens, scale, window, sinks):
    """(out, tolerance) of gbe_attn_decode_window; bf16 queries: weights of 8 bits at least."""
    B = q.shape[0]
    out, tol, _ = chunk(q, cache, range(B + 1), table, [max(int(n), 0) for n in lens], scale, window, sinks,
                        q.dtype == torch.bfloat16)
    return out, tol


def prompt(q, k, v, starts, scale, window, sinks, rounded=False):
    """(out, tolerance, written) of gbe_attn_prompt_window."""
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
        ok = sees(range(z - a), z - a, window, sinks, q.device)
        for h in range(Hq):
            out[a:z, h], tol[a:z, h] = masked(q[a:z, h].double(), k[a:z, h // group].double(),
                                              v[a:z, h // group].double(), ok, scale, rounded, step)
    return out, tol, written


def rand(shape, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(counts, first=0):
    at = [first]
    for n in counts:
        at.append(at[-1] + n)
    return at


def filled(lens, P, H, D, dtype, kind, seed, spare_pages=3, spare_cols=0, std=1.0):
    """A cache whose live tokens are random and whose every other byte is NaN, and its table."""
    import elementwise_row_rmsnorm_gb300 as gbe
    pages = sum(-(-n // P) for n in lens) + spare_pages
    cache = gbe.kv_cache(pages, H, P, D, kind)
    if kind == torch.float8_e4m3fn:
        cache.k.view(torch.uint8).fill_(0x7F)
        cache.v.view(torch.uint8).fill_(0xFF)
        cache.k_scale.fill_(254)
        cache.v_scale.fill_(254)
    else:
        cache.k.fill_(float("nan"))
        cache.v.fill_(float("nan"))
    table = attn_ref.make_table(lens, P, pages, seed, spare_cols)
    slots = [int(table[b, t // P]) * P + t % P for b, n in enumerate(lens) for t in range(n)]
    if slots:
        gbe.gbe_kv_write(rand((len(slots), H, D), dtype, seed, std), rand((len(slots), H, D), dtype, seed + 1),
                         i32(slots), cache)
    return cache, table.cuda()
