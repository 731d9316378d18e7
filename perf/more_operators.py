"""The operators that serve tokens behind a cached prefix, as cases to be timed and compared:

  append  q and k rotated by their positions, q returned, k and v stored into
          a paged cache as they are or as e4m3 with a power-of-two scale a row
  chunk   attention of the new tokens of each sequence over the paged cache
          that holds its prefix and them, with or without a sliding window
  decode  attention of one new token per sequence over the cache under a
          sliding window, a few first tokens (sinks) staying visible
  prompt  causal attention over packed prompts under such a window

``listed()`` names the cases, ``draw()`` makes more of the same ranges,
``prepare()`` makes a case's inputs on the GPU, ``run()`` passes once through
the operator -- in elementary torch operations in 32 bits, or, where ``own`` is
true, by the library's entry points -- and ``exact()`` evaluates the definition
in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---- the cases -------------------------------------------------------------------

def listed():
    return [
        # a decode step of 64 sequences: one token each rotated and stored, bound by the launch
        {"name": "append-64-bf16", "op": "append", "dtype": "bf16", "cache": "bf16", "tokens": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "r": 128, "layout": 0},
        # a prefill of 8192 tokens from the fused projection's output into 8 bits (read back to be compared)
        {"name": "append-8192-e4m3", "op": "append", "dtype": "bf16", "cache": "e4m3", "tokens": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "page": 64, "r": 128, "layout": 0},
        # f32 storage, an odd count of tokens, small pages, interleaved pairs over half of each head
        {"name": "append-1333-f32", "op": "append", "dtype": "f32", "cache": "f32", "tokens": 1333, "Hq": 14, "Hkv": 2,
         "D": 64, "page": 16, "r": 32, "layout": 1},
        # one long prompt's next 2048 tokens behind 30720 cached ones: bound by the products
        {"name": "chunk-2048+30720-bf16", "op": "chunk", "dtype": "bf16", "cache": "bf16", "B": 1, "new": 2048,
         "cached": 30720, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": False, "window": 0, "sinks": 0},
        # a mixed batch: 24 sequences with 1 to 200 new tokens behind up to 8000 cached ones
        {"name": "chunk-24x200+8000-bf16", "op": "chunk", "dtype": "bf16", "cache": "bf16", "B": 24, "new": 200,
         "cached": 8000, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": True, "window": 0, "sinks": 0},
        # 64 users' drafts of 5 tokens to be verified over an 8-bit cache: bound by the cache's bytes
        {"name": "chunk-64x5+8000-e4m3", "op": "chunk", "dtype": "bf16", "cache": "e4m3", "B": 64, "new": 5,
         "cached": 8000, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": False, "window": 0, "sinks": 0},
        # one user's question of 33 tokens behind a very long document: few rows, so the length has to be split
        {"name": "chunk-33+131072-bf16", "op": "chunk", "dtype": "bf16", "cache": "bf16", "B": 1, "new": 33,
         "cached": 131072, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": False, "window": 0, "sinks": 0},
        # f32 storage, small pages, 7 query heads to a kv head, a window
        {"name": "chunk-5x100+900-f32", "op": "chunk", "dtype": "f32", "cache": "f32", "B": 5, "new": 100,
         "cached": 900, "Hq": 14, "Hkv": 2, "D": 64, "page": 16, "ragged": True, "window": 500, "sinks": 4},
        # a decode step of 64 sequences of 0 to 8192 tokens, of which a layer sees the last 1024 and the first 4
        {"name": "decode-64x8192-w1024-bf16", "op": "decode", "dtype": "bf16", "cache": "bf16", "B": 64,
         "longest": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": True, "window": 1024, "sinks": 4},
        # one user far into a long conversation, an 8-bit cache
        {"name": "decode-1x131072-w4096-e4m3", "op": "decode", "dtype": "bf16", "cache": "e4m3", "B": 1,
         "longest": 131072, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "ragged": False, "window": 4096, "sinks": 16},
        # the long prefill of a windowed layer
        {"name": "prompt-8192-w1024-bf16", "op": "prompt", "dtype": "bf16", "B": 1, "longest": 8192, "Hq": 32,
         "Hkv": 8, "D": 128, "ragged": False, "window": 1024, "sinks": 4},
        # three packed prompts in f32, an odd window
        {"name": "prompt-3x1000-w129-f32", "op": "prompt", "dtype": "f32", "B": 3, "longest": 1000, "Hq": 8, "Hkv": 8,
         "D": 64, "ragged": True, "window": 129, "sinks": 1},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "chunk", "chunk", "decode", "prompt"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "D": rng.choice([64, 72, 80, 96, 128])}
    Hkv = rng.choice([1, 2, 4, 5, 8])
    case |= {"Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8])}
    if op != "prompt":
        case["cache"] = rng.choice([case["dtype"], "e4m3"])
        case["page"] = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        case |= {"tokens": _log(rng, 64, 8192), "layout": rng.choice([0, 1]),
                 "r": case["D"] // rng.choice([1, 1, 2]) // 2 * 2}
        while case["tokens"] * case["Hq"] * case["D"] > 2 ** 25:
            case["tokens"] //= 2
        return case
    case["ragged"] = rng.random() < 0.7
    case |= {"window": _log(rng, 16, 8192), "sinks": rng.choice([0, 1, 4, 16, 100])}
    if op == "chunk":
        if rng.random() < 0.6:
            case |= {"window": 0, "sinks": 0}
        case |= {"B": _log(rng, 1, 64), "new": _log(rng, 1, 2048), "cached": _log(rng, 50, 131072)}
        while case["B"] * case["Hq"] * case["new"] * (case["new"] + case["cached"]) > 2 ** 30:
            side = "B" if case["B"] > 1 and rng.random() < 0.4 else max("new", "cached", key=case.get)
            case[side] //= 2
        while case["B"] * (case["new"] + case["cached"]) * Hkv * case["D"] > 2 ** 27:
            case["cached"] //= 2
    elif op == "decode":
        case |= {"B": _log(rng, 1, 64), "longest": _log(rng, 100, 131072)}
        while case["B"] * case["longest"] * Hkv * case["D"] > 2 ** 27:
            case["longest"] //= 2
    else:
        case |= {"Hq": min(case["Hq"], 4 * Hkv), "B": _log(rng, 1, 16),
                 "longest": _log(rng, 60, 4096 if case["dtype"] == "bf16" else 1500)}
        while case["B"] * case["Hq"] * case["longest"] ** 2 > 2 ** 29:
            case["longest"] //= 2
    return case


def _spread(n, most, first):
    """n whole numbers between `first` and most (golden-section steps), the first one the largest."""
    got = [first + int((most - first) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]
    got[0] = most
    return got


def _lengths(case):
    """(new tokens, tokens in all) of each sequence.  Ragged: spread over the range; a ragged decode batch of 8 or more
    also holds an empty slot, a ragged batch of chunks of 8 or more a sequence without new tokens."""
    B = case["B"]
    if case["op"] == "chunk":
        new, cached = [case["new"]] * B, [case["cached"]] * B
        if case["ragged"]:
            new, cached = _spread(B, case["new"], 1), _spread(B, case["cached"], 0)[::-1]
            if B >= 8:
                new[3], new[5], cached[6] = 1, 0, 0
        return new, [a + b for a, b in zip(new, cached)]
    lens = [case["longest"]] * B
    if case["ragged"]:
        lens = _spread(B, case["longest"], 1)
        if B >= 8:
            lens[3] = 1
            if case["op"] == "decode":
                lens[5] = 0
    return [min(n, 1) for n in lens] if case["op"] == "decode" else lens, lens


def _seen(first, last, window, sinks):
    """(pairs of a row and a key that it sees, keys that any row sees) for rows at positions first .. last."""
    if last < first:
        return 0, 0
    if not window:
        return sum(range(first + 1, last + 2)), last + 1
    pairs = 0
    for p in range(first, last + 1):
        low = max(0, p - window + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, first - window + 1)
    return pairs, last + 1 - low + min(sinks, low)


def work(case):
    D, Hq, Hkv, es = case["D"], case["Hq"], case["Hkv"], SIZE[case["dtype"]]
    row = 0
    if case["op"] != "prompt":  # one token of the cache: k and v, with a scale byte for each head of an 8-bit one
        row = 2 * Hkv * (D * SIZE[case["cache"]] + (1 if case["cache"] == "e4m3" else 0))
    if case["op"] == "append":
        n = case["tokens"]
        moved = n * ((2 * Hq + 2 * Hkv) * D * es + 8 + row) + 2 * case["r"]
        if case["cache"] == "e4m3":  # read back
            moved += n * (row + 2 * Hkv * D * es)
        return {"bytes": moved, "flops": 3 * n * (Hq + Hkv) * case["r"]}
    new, lens = _lengths(case)
    pairs, keys = zip(*(_seen(n - m, n - 1, case["window"], case["sinks"]) for m, n in zip(new, lens)))
    small = 8 * case["B"]
    if case["op"] == "prompt":
        return {"bytes": sum(lens) * (2 * Hq + 2 * Hkv) * D * es + small, "flops": 4 * D * Hq * sum(pairs)}
    small += sum(4 * -(-n // case["page"]) for n in keys)
    return {"bytes": sum(keys) * row + 2 * (sum(new) if case["op"] == "chunk" else case["B"]) * Hq * D * es + small,
            "flops": 4 * D * Hq * sum(pairs)}


# ---- inputs ----------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _power(e):
    """2^e of whole e, -126 <= e <= 127, in 32 bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x):
    """e4m3 codes and scale bytes of rows x[..., D]: the scale is the least power of two, 2^(byte - 127), that brings
    the row's largest magnitude to 448 or below."""
    mantissa, exponent = torch.frexp(x.float().abs().amax(-1))
    e = (exponent - torch.where(mantissa > 0.875, 8, 9)).clamp(-126, 126)
    e = torch.where(mantissa == 0, -126, e)
    codes = (x.float() * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _cache(case, g, pages, filled):
    """k, v, k_scale, v_scale of a paged cache [pages, Hkv, page, D]; the scales are None unless it holds e4m3."""
    shape = (pages, case["Hkv"], case["page"], case["D"])
    kind = TYPES[case["cache"]]
    got = []
    for channels in (0.5, 0.0):  # keys have a few loud channels, values none
        if filled:
            x = _normal(g, *shape) * torch.exp(channels * _normal(g, case["Hkv"], 1, case["D"]))
            x = x.to(TYPES[case["dtype"]])
        else:
            x = torch.zeros(shape, device="cuda")
        got.append(_encode(x) if case["cache"] == "e4m3" else (x.to(kind), None))
        del x
    (k, ks), (v, vs) = got
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def _starts(counts):
    starts = torch.zeros(len(counts) + 1, dtype=torch.int64)
    starts[1:] = torch.tensor(counts).cumsum(0)
    return starts.to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, Hq, Hkv, kind = case["D"], case["Hq"], case["Hkv"], TYPES[case["dtype"]]
    state = {"case": case, "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "append":
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + 3
        # the tokens fill whole pages in the order in which a pool handed them out
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        state["slots"] = (order[t // page] * page + t % page).to(torch.int32)
        state["pos"] = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
        state["inv_freq"] = (500000.0 ** (-torch.arange(case["r"] // 2, device="cuda").double() * 2 / case["r"])).float()
        state["cache"] = _cache(case, g, pages, False)
        fused = (_normal(g, n, Hq + 2 * Hkv, D) * 1.5).to(kind)
        state["q"], state["k"], state["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        state["q_out"] = torch.zeros_like(fused)[:, :Hq]
        return state
    new, lens = _lengths(case)
    state["starts"] = _starts(new)
    state["longest"], state["most_new"] = max(lens), max(new)
    if case["op"] == "prompt":
        fused = (_normal(g, sum(lens), Hq + 2 * Hkv, D) * 1.2).to(kind)
        state["q"], state["k"], state["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
        return state
    need = [-(-n // case["page"]) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    state["table"] = table
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    state["cache"] = _cache(case, g, pages, True)
    state["q"] = (_normal(g, len(lens) if case["op"] == "decode" else sum(new), Hq, D) * 1.5).to(kind)
    return state


# ---- one pass --------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "chunk": _chunk, "decode": _decode, "prompt": _prompt}[state["case"]["op"]](state)


def _run_own(state):
    import elementwise_row_rmsnorm_gb300 as gbe
    case = state["case"]
    window, sinks = case.get("window"), case.get("sinks")
    if case["op"] == "prompt":
        return gbe.attn_prompt_window(state["q"], state["k"], state["v"], state["starts"], window, sinks, state["scale"])
    c = state["cache"]
    cache = gbe.KvCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    if case["op"] == "append":
        gbe.gbe_rope_kv_write(state["q"], state["q_out"], state["k"], state["v"], state["pos"], state["slots"], cache,
                              state["inv_freq"], case["r"], 1.0, case["layout"])
        if c["k_scale"] is None:
            return state["q_out"], c["k"], c["v"]
        return state["q_out"], *gbe.kv_read(cache, state["slots"], state["q"].dtype)
    if case["op"] == "chunk":
        return gbe.attn_chunk(state["q"], cache, state["starts"], state["table"], state["lens"], state["scale"], window,
                              sinks)
    return gbe.attn_decode_window(state["q"], cache, state["table"], state["lens"], window, sinks, state["scale"])


def _angles(state):
    """[T, r/2] in 64 bits: by definition the product of position and frequency in 32."""
    return (state["pos"].float()[:, None] * state["inv_freq"]).double()


def _rotated(state, x):
    """x [T, H, D] turned by its positions' angles; in 32 bits, not rounded."""
    case, r = state["case"], state["case"]["r"]
    theta = _angles(state)
    cos, sin = theta.cos().float()[:, None], theta.sin().float()[:, None]
    y = x.float()
    if case["layout"] == 0:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, y[..., r:]], -1)
    a, b = y[..., 0:r:2], y[..., 1:r:2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(2), y[..., r:]], -1)


def _append(state):
    case, c = state["case"], state["cache"]
    kind = state["q"].dtype
    p, row = state["slots"].long() // case["page"], state["slots"].long() % case["page"]
    state["q_out"].copy_(_rotated(state, state["q"]).to(kind))
    k, v = _rotated(state, state["k"]).to(kind), state["v"]
    if c["k_scale"] is None:
        c["k"][p, :, row], c["v"][p, :, row] = k, v
        return state["q_out"], c["k"], c["v"]
    back = []
    for name, x in (("k", k), ("v", v)):
        codes, scale = _encode(x)
        c[name].view(torch.uint8)[p, :, row] = codes.view(torch.uint8)
        c[name + "_scale"][p, :, row] = scale
        codes = c[name].view(torch.uint8)[p, :, row].view(torch.float8_e4m3fn)
        back.append(_widen(codes, c[name + "_scale"][p, :, row]).to(kind))
    return state["q_out"], *back


def _widen(x, scale):
    return x.float() if scale is None else x.float() * _power(scale[..., None].int() - 127)


def _paged(x, scale, table):
    """[B, Hkv, tokens, D] in 32 bits of the pages that a table lists."""
    at = table.long()
    if scale is None:
        y = x[at].float()
    else:
        y = _widen(x.view(torch.uint8)[at].view(torch.float8_e4m3fn), scale[at])
    return y.transpose(1, 2).flatten(2, 3)


def _visible(p, j, case):
    """Whether a row at position p sees key j."""
    seen = j <= p
    if case["window"]:
        seen &= (j > p - case["window"]) | (j < case["sinks"])
    return seen


def _softmax_(s, seen):
    """Weights over the last axis, in place, and their sums; a row that sees nothing gets zeros."""
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    s -= torch.where(m == -math.inf, 0.0, m)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    return s, torch.where(total == 0, 1.0, total)


def _chunk(state):
    case, c, q = state["case"], state["cache"], state["q"]
    starts, lens, n = state["starts"].long(), state["lens"].long(), state["most_new"]
    k, v = _paged(c["k"], c["k_scale"], state["table"]), _paged(c["v"], c["v_scale"], state["table"])
    T, Hq, D = q.shape
    B, Hkv, L = k.shape[:3]
    i = torch.arange(n, device=q.device)
    at = starts[:-1, None] + i
    there = at < starts[1:, None]
    qs = q[at.clamp(max=T - 1)].float().reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    s = (qs.reshape(B, Hkv, -1, D) @ k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, n, L)
    s *= state["scale"]
    p = (lens - (starts[1:] - starts[:-1]))[:, None] + i
    w, total = _softmax_(s, _visible(p[:, :, None], torch.arange(L, device=q.device), case)[:, None, None])
    out = (w.view(B, Hkv, -1, L) @ v).view(B, Hkv, Hq // Hkv, n, D) / total
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)[there].to(q.dtype)


def _decode(state):
    case, c, q = state["case"], state["cache"], state["q"]
    k, v = _paged(c["k"], c["k_scale"], state["table"]), _paged(c["v"], c["v_scale"], state["table"])
    B, Hq, D = q.shape
    p = (state["lens"] - 1)[:, None, None, None]
    s = q.float().reshape(B, k.shape[1], Hq // k.shape[1], D) @ k.transpose(2, 3) * state["scale"]
    w, total = _softmax_(s, _visible(p, torch.arange(k.shape[2], device=q.device), case))
    return (w @ v / total).reshape(B, Hq, D).to(q.dtype)


def _prompt(state):
    q, k, v, starts, n = state["q"], state["k"], state["v"], state["starts"].long(), state["longest"]
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    step = torch.arange(n, device=q.device)
    at = starts[:-1, None] + step
    there = at < starts[1:, None]
    at = at.clamp(max=T - 1)
    B = at.shape[0]
    qs = q[at].float().reshape(B, n, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4)
    ks = k[at].float().permute(0, 2, 3, 1)[:, :, None]
    vs = v[at].float().transpose(1, 2)[:, :, None]
    s = qs @ ks
    s *= state["scale"]
    w, total = _softmax_(s, _visible(step[:, None], step, state["case"]))
    out = (w @ vs / total).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return out[there].to(q.dtype)


# ---- the definition in 64 bits -----------------------------------------------------

def _round_e4m3(y):
    """The e4m3 number nearest to y, ties to the even code; |y| <= 448."""
    top = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20)))
    unit = torch.exp2(top.clamp_min(-6.0) - 3.0)
    return torch.round(y / unit) * unit


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(state)
    q = state["q"].double()
    out = torch.zeros_like(q)
    new, lens = _lengths(case)
    group, at = case["Hq"] // case["Hkv"], 0
    for b, (m, n) in enumerate(zip(new, lens)):
        if m == 0:
            at += 1 if case["op"] == "decode" else 0
            continue
        i = torch.arange(n - m, n, device="cuda")[:, None]
        j = torch.arange(n, device="cuda")[None]
        hidden = j > i
        if case["window"]:
            hidden |= (i - j >= case["window"]) & (j >= case["sinks"])
        for h in range(case["Hkv"]):
            k, v = _exact_rows(state, b, h, at, n)
            logits = q[at:at + m, h * group:(h + 1) * group].transpose(0, 1) @ k.T * state["scale"]
            w = torch.softmax(logits.masked_fill_(hidden, -math.inf), -1)
            out[at:at + m, h * group:(h + 1) * group] = (w @ v).transpose(0, 1)
        at += m
    return out


def _exact_rows(state, b, h, at, n):
    """k and v [n, D] of kv head h of sequence b, whose rows begin at row `at` of the packed buffers."""
    case = state["case"]
    if case["op"] == "prompt":
        return state["k"][at:at + n, h].double(), state["v"][at:at + n, h].double()
    c, t = state["cache"], torch.arange(n, device="cuda")
    page, row = state["table"][b, t // case["page"]].long(), t % case["page"]
    got = []
    for name in ("k", "v"):
        if c[name + "_scale"] is None:
            got.append(c[name][page, h, row].double())
        else:
            codes = c[name].view(torch.uint8)[page, h, row].view(torch.float8_e4m3fn).double()
            got.append(codes * torch.exp2(c[name + "_scale"][page, h, row].double() - 127.0)[:, None])
    return got


def _exact_append(state):
    case, r = state["case"], state["case"]["r"]
    # pair i turns as a complex number does that is multiplied by exp(i theta)
    theta = (state["pos"].float()[:, None] * state["inv_freq"]).double()
    turn = torch.polar(torch.ones_like(theta), theta)[:, None]
    turned = []
    for x in (state["q"].double(), state["k"].double()):
        first, second = (x[..., :r // 2], x[..., r // 2:r]) if case["layout"] == 0 else (x[..., 0:r:2], x[..., 1:r:2])
        z = torch.complex(first.contiguous(), second.contiguous()) * turn
        y = x.clone()
        if case["layout"] == 0:
            y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
        else:
            y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
        turned.append(y)
    q, k = turned
    v = state["v"].double()
    c, slots = state["cache"], state["slots"].long()
    got = []
    for name, rows in (("k", k), ("v", v)):
        if c[name + "_scale"] is not None and name == "k":
            got.append(None)  # next to a border between two codes the last bit of a cosine decides, and the step is 2^-4
        elif c[name + "_scale"] is not None:  # what the cache stands for
            largest = rows.abs().amax(-1)
            e = torch.ceil(torch.log2(largest / 448.0)).clamp(-126, 127)
            e = torch.where(largest > 448.0 * torch.exp2(e), e + 1, e)
            e = torch.where(largest <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-126, 127)[..., None]
            got.append(_round_e4m3(rows / torch.exp2(e)) * torch.exp2(e))
        else:
            token = torch.zeros(c[name].shape[0] * case["page"], case["Hkv"], case["D"], dtype=torch.float64,
                                device="cuda")
            token[slots] = rows
            got.append(token.view(-1, case["page"], case["Hkv"], case["D"]).transpose(1, 2).contiguous())
    return q, *got
