"""The serving operators around attention, as cases to be timed and compared:

  write   k and v rows of new tokens into a paged cache, stored as they are or
          as e4m3 with one power-of-two scale per token and head
  read    cached rows gathered back, widened to the model's type
  decode  attention of one new token per sequence over the paged cache
  prompt  causal attention over packed prompts, with grouped heads

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
        # a decode step of 64 sequences stores one token each (8 kv heads of 128): bound by the launch
        {"name": "write-64-bf16", "op": "write", "dtype": "bf16", "cache": "bf16", "tokens": 64, "Hkv": 8, "D": 128,
         "page": 64},
        # a prefill of 8192 tokens stored in 8 bits, k and v columns of the fused projection's output
        {"name": "write-8192-e4m3", "op": "write", "dtype": "bf16", "cache": "e4m3", "tokens": 8192, "Hkv": 8,
         "D": 128, "page": 64},
        # one short prompt's cache copied out, an odd count of tokens and small pages
        {"name": "read-333-bf16", "op": "read", "dtype": "bf16", "cache": "bf16", "tokens": 333, "Hkv": 8, "D": 128,
         "page": 16},
        # a long shared prefix in 8 bits widened for reuse by a prompt
        {"name": "read-65536-e4m3", "op": "read", "dtype": "bf16", "cache": "e4m3", "tokens": 65536, "Hkv": 8,
         "D": 128, "page": 64},
        # one user, a short chat: latency
        {"name": "decode-1x500-bf16", "op": "decode", "dtype": "bf16", "cache": "bf16", "B": 1, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "longest": 500, "ragged": False},
        # the ordinary decode step: 64 sequences of 0 to 8192 tokens
        {"name": "decode-64x8192-bf16", "op": "decode", "dtype": "bf16", "cache": "bf16", "B": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "longest": 8192, "ragged": True},
        # the same step over an 8-bit cache, every sequence full
        {"name": "decode-64x8192-e4m3", "op": "decode", "dtype": "bf16", "cache": "e4m3", "B": 64, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "longest": 8192, "ragged": False},
        # two users with very long contexts: few rows, so the length has to be split
        {"name": "decode-2x131072-bf16", "op": "decode", "dtype": "bf16", "cache": "bf16", "B": 2, "Hq": 32, "Hkv": 8,
         "D": 128, "page": 64, "longest": 131072, "ragged": False},
        # f32 storage, an odd batch, small pages, 7 query heads to a kv head
        {"name": "decode-17x2000-f32", "op": "decode", "dtype": "f32", "cache": "f32", "B": 17, "Hq": 14, "Hkv": 2,
         "D": 64, "page": 16, "longest": 2000, "ragged": True},
        # a packed batch of short prompts of 1 to 500 tokens
        {"name": "prompt-12x500-bf16", "op": "prompt", "dtype": "bf16", "B": 12, "Hq": 32, "Hkv": 8, "D": 128,
         "longest": 500, "ragged": True},
        # the long prefill: one prompt of 8192 tokens
        {"name": "prompt-1x8192-bf16", "op": "prompt", "dtype": "bf16", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "longest": 8192, "ragged": False},
        # f32 storage, heads of 64, three packed prompts
        {"name": "prompt-3x1000-f32", "op": "prompt", "dtype": "f32", "B": 3, "Hq": 8, "Hkv": 8, "D": 64,
         "longest": 1000, "ragged": True},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "decode", "decode", "prompt", "prompt"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "D": rng.choice([64, 72, 80, 96, 128])}
    Hkv = rng.choice([1, 2, 4, 5, 8])
    if op != "prompt":
        case["cache"] = rng.choice([case["dtype"], "e4m3"])
        case["page"] = rng.choice([16, 32, 48, 64, 128])
    if op in ("write", "read"):
        case |= {"tokens": _log(rng, 64, 8192 if op == "write" else 32768), "Hkv": Hkv}
        return case
    case |= {"Hkv": Hkv, "Hq": Hkv * rng.choice([1, 2, 3, 4, 7, 8])}
    if op == "decode":
        case["B"] = _log(rng, 1, 64)
        case["longest"] = _log(rng, 100, 131072)
        while case["B"] * case["longest"] * Hkv * case["D"] > 2 ** 27:
            case["longest"] //= 2
    else:
        case["Hq"] = min(case["Hq"], 4 * Hkv)
        case["B"] = _log(rng, 1, 16)
        case["longest"] = _log(rng, 60, 4096 if case["dtype"] == "bf16" else 1500)
        while case["B"] * case["Hq"] * case["longest"] ** 2 > 2 ** 29:
            case["longest"] //= 2
    case["ragged"] = rng.random() < 0.7
    return case


def _lengths(case):
    """The sequences' lengths: all the longest, or spread between 1 and it (golden-section steps), the first one the
    longest; a ragged decode batch of 8 or more also holds an empty slot, as a padded batch does."""
    B, n = case["B"], case["longest"]
    if not case["ragged"]:
        return [n] * B
    got = [1 + int((n - 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(B)]
    got[0] = n
    if B >= 8:
        got[3] = 1
        if case["op"] == "decode":
            got[5] = 0
    return got


def work(case):
    D, Hkv, es = case["D"], case["Hkv"], SIZE[case["dtype"]]
    row = 0
    if case["op"] != "prompt":  # one token of the cache: k and v, with a scale byte for each head of an 8-bit one
        row = 2 * Hkv * (D * SIZE[case["cache"]] + (1 if case["cache"] == "e4m3" else 0))
    if case["op"] in ("write", "read"):
        n = case["tokens"]
        return {"bytes": n * (2 * Hkv * D * es + 4 + row), "flops": 0}
    lens, Hq = _lengths(case), case["Hq"]
    if case["op"] == "decode":
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": sum(lens) * row + 2 * case["B"] * Hq * D * es + 4 * (pages + case["B"]),
                "flops": 4 * D * Hq * sum(lens)}
    return {"bytes": sum(lens) * (2 * Hq + 2 * Hkv) * D * es + 4 * (case["B"] + 1),
            "flops": 4 * D * Hq * sum(n * (n + 1) // 2 for n in lens)}


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, Hkv, kind = case["D"], case["Hkv"], TYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("write", "read"):
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + 3
        # the tokens fill whole pages in the order in which a pool handed them out
        order = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        state["slots"] = (order[t // page] * page + t % page).to(torch.int32)
        state["cache"] = _cache(case, g, pages, case["op"] == "read")
        if case["op"] == "write":
            fused = (_normal(g, n, 4 * Hkv, D) * 1.5).to(kind)  # [q | k | v] of the projection, 2 q heads a kv head
            state["k_new"], state["v_new"] = fused[:, 2 * Hkv:3 * Hkv], fused[:, 3 * Hkv:]
        return state
    lens, Hq = _lengths(case), case["Hq"]
    state["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "decode":
        need = [-(-n // case["page"]) for n in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        wide = max(1, max(need))
        table = torch.zeros(len(lens), wide, dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = order[at:at + m]
            at += m
        state["table"] = table
        state["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        state["cache"] = _cache(case, g, pages, True)
        state["q"] = (_normal(g, len(lens), Hq, D) * 1.5).to(kind)
        return state
    fused = (_normal(g, sum(lens), Hq + 2 * Hkv, D) * 1.2).to(kind)
    state["q"], state["k"], state["v"] = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    starts = torch.zeros(len(lens) + 1, dtype=torch.int64)
    starts[1:] = torch.tensor(lens).cumsum(0)
    state["starts"] = starts.to(torch.int32).cuda()
    state["longest"] = max(lens)
    return state


# ---- one pass --------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"write": _write, "read": _read, "decode": _decode, "prompt": _prompt}[state["case"]["op"]](state)


def _run_own(state):
    import elementwise_row_rmsnorm_gb300 as gbe
    op = state["case"]["op"]
    if op == "prompt":
        return gbe.attn_prompt(state["q"], state["k"], state["v"], state["starts"], state["scale"])
    c = state["cache"]
    cache = gbe.KvCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    if op == "write":
        gbe.gbe_kv_write(state["k_new"], state["v_new"], state["slots"], cache)
        return c
    if op == "read":
        return gbe.kv_read(cache, state["slots"], TYPES[state["case"]["dtype"]])
    return gbe.attn_decode(state["q"], cache, state["table"], state["lens"], state["scale"])


def _write(state):
    c, page = state["cache"], state["case"]["page"]
    p, r = state["slots"].long() // page, state["slots"].long() % page
    if c["k_scale"] is None:
        c["k"][p, :, r] = state["k_new"].to(c["k"].dtype)
        c["v"][p, :, r] = state["v_new"].to(c["v"].dtype)
        return c
    codes, scale = _encode(state["k_new"])
    c["k"].view(torch.uint8)[p, :, r] = codes.view(torch.uint8)
    c["k_scale"][p, :, r] = scale
    codes, scale = _encode(state["v_new"])
    c["v"].view(torch.uint8)[p, :, r] = codes.view(torch.uint8)
    c["v_scale"][p, :, r] = scale
    return c


def _widen(x, scale):
    return x.float() if scale is None else x.float() * _power(scale[..., None].int() - 127)


def _read(state):
    c, page = state["cache"], state["case"]["page"]
    p, r = state["slots"].long() // page, state["slots"].long() % page
    kind = TYPES[state["case"]["dtype"]]
    if c["k_scale"] is None:
        return c["k"][p, :, r].to(kind), c["v"][p, :, r].to(kind)
    k = _widen(c["k"].view(torch.uint8)[p, :, r].view(torch.float8_e4m3fn), c["k_scale"][p, :, r])
    v = _widen(c["v"].view(torch.uint8)[p, :, r].view(torch.float8_e4m3fn), c["v_scale"][p, :, r])
    return k.to(kind), v.to(kind)


def _paged(x, scale, table):
    """[B, Hkv, tokens, D] in 32 bits of the pages that a table lists."""
    at = table.long()
    if scale is None:
        y = x[at].float()
    else:
        y = _widen(x.view(torch.uint8)[at].view(torch.float8_e4m3fn), scale[at])
    return y.transpose(1, 2).flatten(2, 3)


def _decode(state):
    c, q = state["cache"], state["q"]
    k, v = _paged(c["k"], c["k_scale"], state["table"]), _paged(c["v"], c["v_scale"], state["table"])
    B, Hq, D = q.shape
    there = torch.arange(k.shape[2], device=q.device) < state["lens"][:, None]
    there = there[:, None, None, :]
    s = q.float().reshape(B, k.shape[1], Hq // k.shape[1], D) @ k.transpose(2, 3) * state["scale"]
    s = torch.where(there, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = w.sum(-1, keepdim=True)
    out = w @ v / torch.where(total == 0, 1.0, total)
    return out.reshape(B, Hq, D).to(q.dtype)


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
    s.masked_fill_(step > step[:, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    out = (s @ vs / total).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return out[there].to(q.dtype)


# ---- the definition in 64 bits -----------------------------------------------------

def _round_e4m3(y):
    """The e4m3 number nearest to y, ties to the even code; |y| <= 448."""
    top = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20)))
    unit = torch.exp2(top.clamp_min(-6.0) - 3.0)
    return torch.round(y / unit) * unit


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(state)
    c = state["cache"]
    page = case["page"]
    if case["op"] == "write":
        out = {}
        for name in ("k", "v"):
            rows = state[name + "_new"].double()
            values = torch.zeros(c[name].shape, dtype=torch.float64, device="cuda")
            token = values.transpose(1, 2).reshape(-1, case["Hkv"], case["D"])  # [slot, head, D]
            if c[name + "_scale"] is None:
                token[state["slots"].long()] = rows
                out[name + "_scale"] = None
            else:
                largest = rows.abs().amax(-1)
                e = torch.ceil(torch.log2(largest / 448.0)).clamp(-126, 127)
                e = torch.where(largest > 448.0 * torch.exp2(e), e + 1, e)
                e = torch.where(largest <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-126, 127)
                token[state["slots"].long()] = _round_e4m3(rows / torch.exp2(e)[..., None])
                out[name + "_scale"] = None
            out[name] = token.reshape(-1, page, case["Hkv"], case["D"]).transpose(1, 2).contiguous()
        return out
    if case["op"] == "read":
        got = []
        for name in ("k", "v"):
            token = c[name].double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])[state["slots"].long()]
            if c[name + "_scale"] is not None:
                bytes_ = c[name + "_scale"].transpose(1, 2).reshape(-1, case["Hkv"])[state["slots"].long()]
                token = token * torch.exp2(bytes_.double() - 127.0)[..., None]
            got.append(token)
        return tuple(got)
    q = state["q"].double()
    group = case["Hq"] // case["Hkv"]
    out = torch.zeros_like(q)
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        at = state["table"][b, :-(-n // page)].long()
        kv = []
        for name in ("k", "v"):
            x = c[name].view(torch.uint8)[at].view(c[name].dtype).double() if c[name + "_scale"] is not None \
                else c[name][at].double()
            if c[name + "_scale"] is not None:
                x = x * torch.exp2(c[name + "_scale"][at].double() - 127.0)[..., None]
            kv.append(x.transpose(0, 1).reshape(case["Hkv"], -1, case["D"])[:, :n])
        for h in range(case["Hkv"]):
            logits = q[b, h * group:(h + 1) * group] @ kv[0][h].T * state["scale"]
            out[b, h * group:(h + 1) * group] = torch.softmax(logits, -1) @ kv[1][h]
    return out


def _exact_prompt(state):
    q, k, v = state["q"], state["k"], state["v"]
    group = q.shape[1] // k.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    starts = state["starts"].tolist()
    for a, z in zip(starts, starts[1:]):
        later = torch.ones(z - a, z - a, dtype=torch.bool, device="cuda").triu(1)
        for h in range(q.shape[1]):
            logits = q[a:z, h].double() @ k[a:z, h // group].double().T * state["scale"]
            out[a:z, h] = torch.softmax(logits.masked_fill(later, -math.inf), -1) @ v[a:z, h // group].double()
    return out
