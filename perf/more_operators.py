"""Cases of the operators on a key/value cache that is held in 4 or 8 bits: writing new tokens' keys and values into it,
reading a context back, and attention of new tokens over it.

A row of the cache (one token, one key/value head) holds `dim` codes c of 4 or 8 bits and, for every 32 of them, a step d and
a base m in fp16: a value stands as d c + m.  Codes come first (two to a byte in 4 bits, the lower element in the lower half),
then the dim/32 steps, then the dim/32 bases; a row is padded to a multiple of 16 bytes.

Head layouts are those of the decode workloads in qgemv_inputs/workloads.py: 16 query and 8 key/value heads of 128
(0.6b-class), 32 and 8 heads of 128 (4b-class).  Page sizes, context lengths and batch sizes are generic.  With ``own`` false,
run() computes the operators in elementary torch operations in 32 bits; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
TYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
BLOCK = 32  # elements that share a step and a base
LARGEST = 65504.0


def listed():
    return [
        # one decode token of the 4b-class model on its way into a 4-bit cache, read back as the step's other consumers see it
        dict(name="write-one-token", op="write", bits=4, tokens=1, kv_heads=8, dim=128, page=16, source=F32, type=BF16,
             skipped=0, order="token"),
        # a mixed step: 61 tokens into an 8-bit cache; every 9th is padding of a fixed-size batch and leaves the cache as it was
        dict(name="write-61-tokens", op="write", bits=8, tokens=61, kv_heads=8, dim=128, page=64, source=F16, type=F16,
             skipped=9, order="head"),
        # a long prompt into a 4-bit cache
        dict(name="write-prompt", op="write", bits=4, tokens=16000, kv_heads=8, dim=128, page=64, source=BF16, type=BF16,
             skipped=0, order="token"),
        # a short chat's context, read back to be moved to another pool
        dict(name="read-short", op="read", bits=4, seqs=1, ctx=777, kv_heads=8, dim=128, page=16, type=BF16, first=0,
             order="token", mix=1),
        # the ends of 16 uneven contexts in 8 bits, read back for a program that continues in 16
        dict(name="read-batch", op="read", bits=8, seqs=16, ctx=8001, kv_heads=8, dim=128, page=32, type=F16, first=500,
             order="head", mix=2),
        # the whole of one very long context
        dict(name="read-long", op="read", bits=4, seqs=1, ctx=100003, kv_heads=8, dim=128, page=64, type=BF16, first=0,
             order="token", mix=3),
        # the smallest decode step: one sequence, one new token, a short chat
        dict(name="decode4-short", op="attention", bits=4, seqs=1, new=1, ctx=777, heads=32, kv_heads=8, dim=128, page=16,
             type=BF16, window=0, lse=False, idle=0, order="token", mix=4),
        # one sequence with a very long context: the keys have to be split over the whole GPU
        dict(name="decode4-long", op="attention", bits=4, seqs=1, new=1, ctx=100003, heads=32, kv_heads=8, dim=128, page=64,
             type=BF16, window=0, lse=False, idle=0, order="head", mix=5),
        # the usual serving step: 48 sequences of uneven length, one new token each
        dict(name="decode4-batch", op="attention", bits=4, seqs=48, new=1, ctx=16384, heads=32, kv_heads=8, dim=128, page=16,
             type=BF16, window=0, lse=False, idle=0, order="token", mix=6),
        # drafted tokens to be verified: 16 sequences of up to 5 new tokens, fp16, 0.6b-class heads, 8 bits; three idle slots of
        # a fixed-size batch whose rows see nothing; log-sum-exp wanted for a merge with another part
        dict(name="verify8-drafts", op="attention", bits=8, seqs=16, new=5, ctx=4000, heads=16, kv_heads=8, dim=128, page=32,
             type=F16, window=0, lse=True, idle=3, order="token", mix=7),
        # 33 sequences over an 8-bit cache in a layer with a window of 1024
        dict(name="decode8-window", op="attention", bits=8, seqs=33, new=1, ctx=16384, heads=32, kv_heads=8, dim=128, page=16,
             type=F16, window=1024, lse=False, idle=0, order="token", mix=8),
        # a chunk of a long prompt over what is in the cache already
        dict(name="chunk4-2000-of-24000", op="attention", bits=4, seqs=1, new=2000, ctx=24000, heads=32, kv_heads=8, dim=128,
             page=64, type=BF16, window=0, lse=False, idle=0, order="token", mix=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads = rng.choice([(16, 8), (32, 8)])
    op = rng.choice(["write", "read", "attention", "attention"])
    c = dict(op=op, bits=rng.choice([4, 4, 8]), kv_heads=kv_heads, dim=rng.choice([128, 128, 64, 96, 256]),
             page=rng.choice([16, 32, 64]), type=rng.choice([BF16, F16]), order=rng.choice(["token", "head"]))
    if op == "write":
        c.update(tokens=_log_int(rng, 1, 8000), source=rng.choice([F32, c["type"]]), skipped=rng.choice([0, 0, 7]))
        return c
    mix = rng.randrange(1 << 30)
    if op == "read":
        ctx = _log_int(rng, 16, 100003)
        c.update(seqs=_log_int(rng, 1, max(1, min(48, 100003 // ctx))), ctx=ctx,
                 first=rng.choice([0, rng.randrange(1, ctx)]), mix=mix)
        return c
    c.update(heads=heads, window=rng.choice([0, 0, 1024]), mix=mix)
    if rng.random() < 0.7:  # decode and drafts
        new = rng.choice([1, 1, _log_int(rng, 2, 16)])
        ctx = _log_int(rng, 16, 100003)
        seqs = _log_int(rng, 1, max(1, min(48, 24 * 16384 // (ctx * new))))
        c.update(seqs=seqs, new=new, ctx=ctx, lse=rng.choice([False, True]), idle=rng.choice([0, seqs // 4]))
        return c
    new = _log_int(rng, 17, 3001)
    ctx = _log_int(rng, new, max(new, min(24000, 18000000 // new)))
    c.update(seqs=rng.choice([1, 1, 2]), new=new, ctx=ctx, lse=False, idle=0)
    return c


# ---------------------------------------------------------------------------------------------------- sizes

def _lengths(case):
    """New tokens and context of each sequence: the first has the case's, the others fewer, idle ones no context."""
    r = random.Random(case["mix"])
    new, ctx = [], []
    most = case.get("new", 1)
    for b in range(case["seqs"]):
        n = most if b == 0 else r.randint(max(1, most // 2), most)
        c = case["ctx"] if b == 0 else max(n, int(case["ctx"] * math.exp(-r.random() * math.log(8.0))))
        if b >= case["seqs"] - case.get("idle", 0):
            n, c = 1, 0
        new.append(n)
        ctx.append(c)
    return new, ctx


def _firsts(case, ctx):
    """First token that is read of each context: the case's, or less where a context is as short."""
    return [min(case["first"], c // 2) for c in ctx]


def _row(case):
    """Bytes that a row of the cache holds."""
    return case["dim"] * case["bits"] // 8 + case["dim"] // BLOCK * 4


def _pitch(case):
    return -(-_row(case) // 16) * 16


def work(case):
    token = case["kv_heads"] * case["dim"]
    if case["op"] == "write":
        t = case["tokens"]
        live = t - (t // case["skipped"] if case["skipped"] else 0)
        size = 4 if case["source"] == F32 else 2
        # the tokens, their rows in the cache, and the values read back
        return {"bytes": 2 * (t * token * size + live * case["kv_heads"] * _row(case) + t * token * 2) + 8 * t,
                "flops": 2 * 6 * t * token}
    new, ctx = _lengths(case)
    if case["op"] == "read":
        t = sum(c - f for c, f in zip(ctx, _firsts(case, ctx)))
        return {"bytes": 2 * t * (case["kv_heads"] * _row(case) + token * 2), "flops": 2 * 2 * t * token}
    seen, keys = 0, 0  # pairs of a query and a key it sees; keys that some query sees
    for n, c in zip(new, ctx):
        w = case["window"] or c
        if not c:
            continue
        seen += sum(min(w, c - n + j + 1) for j in range(n))
        keys += min(c, w + n - 1)
    return {"bytes": 2 * sum(new) * case["heads"] * case["dim"] * 2 + 2 * keys * case["kv_heads"] * _row(case)
            + (4 * sum(new) * case["heads"] if case["lse"] else 0),
            "flops": 4 * seen * case["heads"] * case["dim"]}


# ------------------------------------------------------------------------------------------- rows of a cache

def _half_toward(x, up):
    """x (32 bits, within fp16's range) as the nearest fp16 that is not below (up) or not above it."""
    h = x.to(torch.float16)
    bits = h.view(torch.int16).to(torch.int32) & 0xFFFF
    negative = bits >= 0x8000
    off = h.float() < x if up else h.float() > x
    # one step: away from zero on its own side, towards it on the other, over zero to the smallest of the other sign
    away = negative != up
    zero = (bits & 0x7FFF) == 0
    step = torch.where(zero, torch.full_like(bits, 1 if up else 0x8001), torch.where(away, bits + 1, bits - 1))
    bits = torch.where(off, step, bits)
    return torch.where(bits >= 0x8000, bits - 0x10000, bits).to(torch.int16).view(torch.float16)


def _pack(x, bits):
    """Rows of a cache, uint8 [..., bytes], of the values x [..., dim]: per block, the base is its least value rounded down
    to fp16, the step what the largest needs, rounded up; the codes are rounded to the nearest (every step in 32 bits)."""
    top = (1 << bits) - 1
    x = x.float().clamp(-LARGEST, LARGEST).unflatten(-1, (-1, BLOCK))
    base = _half_toward(x.amin(-1), False)
    span = x.amax(-1) - base.float()
    step = _half_toward(span / torch.full_like(span[..., :1], top), True)
    rate = torch.where(step == 0, 0.0, 1.0 / step.float())
    code = torch.round((x - base.float()[..., None]) * rate[..., None]).clamp_(max=top).to(torch.uint8).flatten(-2)
    if bits == 4:
        code = code[..., 0::2] | (code[..., 1::2] << 4)
    row = torch.cat([code, step.contiguous().view(torch.uint8), base.contiguous().view(torch.uint8)], -1)
    return torch.nn.functional.pad(row, (0, -row.shape[-1] % 16))


def _values(rows, bits, dim):
    """The values that rows of a cache stand for, in 32 bits."""
    n, blocks = dim * bits // 8, dim // BLOCK
    code = rows[..., :n]
    if bits == 4:
        code = torch.stack([code & 15, code >> 4], -1).flatten(-2)
    scale = rows[..., n:n + 4 * blocks].contiguous().view(torch.float16).float()
    value = code.float().unflatten(-1, (blocks, BLOCK)) * scale[..., :blocks, None] + scale[..., blocks:, None]
    return value.flatten(-2)


# --------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _keys(g, tokens, heads, dim):
    """Keys as a layer has them: a few channels of every head lie far from zero."""
    x = torch.randn(tokens, heads, dim, generator=g, device="cuda")
    far = 5.0 * torch.randn(heads, dim, generator=g, device="cuda")
    return x.add_(torch.where(torch.rand(heads, dim, generator=g, device="cuda") < 0.04, far, 0.0))


def _ordered(rows, order):
    """The same [pages, page size, heads, bytes], laid out a page's tokens or a page's heads first."""
    return rows if order == "token" else rows.transpose(1, 2).contiguous().transpose(1, 2)


def _library_cache(s):
    import quantized_weight_gemv_quantize_gb300 as qg
    return qg.packed_cache({4: "Q4", 8: "Q8"}[s["case"]["bits"]], s["k_cache"], s["v_cache"], s["case"]["dim"])


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "op": case["op"]}
    {"write": _prepare_write, "read": _prepare_read, "attention": _prepare_attention}[case["op"]](s, case, g)
    return s


def _prepare_write(s, case, g):
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    s["k"] = _keys(g, t, h, d).to(TYPES[case["source"]])
    s["v"] = torch.randn(t, h, d, generator=g, device="cuda").to(TYPES[case["source"]])
    pages = -(-t // page)
    order = torch.randperm(pages + 2, generator=g, device="cuda")  # of the two left over one holds what padding tokens write here
    i = torch.arange(t, device="cuda")
    s["slots"] = order[i // page] * page + i % page
    if case["skipped"]:
        s["slots"][case["skipped"] - 1::case["skipped"]] = -1
    s["spare"] = order[pages]
    for name in ("k_cache", "v_cache"):  # an older sequence's rows
        old = _pack(torch.randn(pages + 2, page, h, d, generator=g, device="cuda"), case["bits"])
        s[name] = _ordered(old, case["order"])
    s["table"] = order[None, :pages].to(torch.int32).contiguous()
    s["start"] = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    s["first"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["k_out"], s["v_out"] = (torch.empty(t, h, d, dtype=TYPES[case["type"]], device="cuda") for _ in range(2))
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        cache = _library_cache(s)
        s["write"] = qg.cache_write_args(s["k"], s["v"], cache, s["slots"])
        s["read"] = qg.cache_read_args(cache, s["table"], s["start"], s["k_out"], s["v_out"], first=s["first"])


def _prepare_contexts(s, case, g, ctx):
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    need = [-(-c // page) for c in ctx]
    total = sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(ctx), max(1, max(need)), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    s["table"] = order[table.long().cuda()].contiguous()
    keys = _keys(g, total * page, h, d).view(total, page, h, d)
    keys[s["table"][:, 0].long(), 0] *= 2.0  # the first token draws attention
    s["k_cache"] = _ordered(_pack(keys, case["bits"]), case["order"])
    del keys
    s["v_cache"] = _ordered(_pack(torch.randn(total, page, h, d, generator=g, device="cuda"), case["bits"]), case["order"])


def _starts(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def _prepare_read(s, case, g):
    _, ctx = _lengths(case)
    _prepare_contexts(s, case, g, ctx)
    first = _firsts(case, ctx)
    s["start"] = _starts([c - f for c, f in zip(ctx, first)])
    s["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
    t = sum(ctx) - sum(first)
    s["k_out"], s["v_out"] = (torch.empty(t, case["kv_heads"], case["dim"], dtype=TYPES[case["type"]], device="cuda")
                              for _ in range(2))
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        s["read"] = qg.cache_read_args(_library_cache(s), s["table"], s["start"], s["k_out"], s["v_out"], first=s["first"])


def _prepare_attention(s, case, g):
    new, ctx = _lengths(case)
    h, kh, d, kind = case["heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]
    _prepare_contexts(s, case, g, ctx)
    s["q"] = (1.5 * torch.randn(sum(new), h, d, generator=g, device="cuda")).to(kind)
    s["q_start"] = _starts(new)
    s["kv_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["max_new"], s["max_ctx"] = max(new), max(ctx)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(sum(new), h, dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        cache = _library_cache(s)
        nbytes = qg.qgemv_attn_scratch_bytes(len(new), sum(new), h, kh, d, s["max_new"], s["max_ctx"], cache=cache)
        s["scratch"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        s["args"] = qg.attn_args(s["q"], cache, s["table"], s["q_start"], s["kv_len"], s["out"], s["scratch"],
                                 max_q=s["max_new"], max_kv=s["max_ctx"], scale=s["scale"], window=case["window"],
                                 lse=s["lse"])


# ------------------------------------------------------------------------------------------------- one pass

def run(state):
    return {"write": _write, "read": _read, "attention": _attention}[state["op"]](state)


def _write(s):
    """New tokens into the cache, and their context read back: the values that the codes stand for."""
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_cache_write(s["write"])
        qg.qgemv_cache_read(s["read"])
        return {"k": s["k_out"], "v": s["v_out"]}
    case = s["case"]
    page = case["page"]
    at = torch.where(s["slots"] < 0, s["spare"] * page, s["slots"])
    for cache, x in (("k_cache", "k"), ("v_cache", "v")):
        s[cache][at // page, at % page] = _pack(s[x], case["bits"])
    return _read(s)


def _read(s):
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_cache_read(s["read"])
        return {"k": s["k_out"], "v": s["v_out"]}
    case = s["case"]
    row = torch.arange(s["k_out"].shape[0], device="cuda")
    seq = torch.searchsorted(s["start"][1:].long(), row, right=True)
    token = s["first"].long()[seq] + row - s["start"].long()[seq]
    where = s["table"].long()[seq, token // case["page"]], token % case["page"]
    s["k_out"].copy_(_values(s["k_cache"][where], case["bits"], case["dim"]))
    s["v_out"].copy_(_values(s["v_cache"][where], case["bits"], case["dim"]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _attention(s):
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_attn(s["args"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    case = s["case"]
    h, kh, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    b, n, length = s["kv_len"].numel(), s["max_new"], max(1, s["max_ctx"])
    t = torch.arange(length, device="cuda")
    where = s["table"].long()[:, t // page], t % page  # [b, length]
    keys = _values(s["k_cache"][where], case["bits"], d).permute(0, 2, 3, 1)  # [b, kh, d, length]
    values = _values(s["v_cache"][where], case["bits"], d).permute(0, 2, 1, 3)  # [b, kh, length, d]
    start, count = s["q_start"][:-1].long(), (s["q_start"][1:] - s["q_start"][:-1]).long()
    j = torch.arange(n, device="cuda")
    row = (start[:, None] + j).clamp(max=s["q"].shape[0] - 1)  # [b, n]
    q = s["q"][row].float().view(b, n, kh, h // kh, d).permute(0, 2, 3, 1, 4).reshape(b, kh, h // kh * n, d)
    score = (q @ keys).mul_(s["scale"]).view(b, kh, h // kh, n, length)
    at = (s["kv_len"].long() - count)[:, None] + j  # position of each new token
    sees = (t <= at[..., None]) & (t < s["kv_len"].long()[:, None, None])
    if case["window"]:
        sees &= t > at[..., None] - case["window"]
    score = score.masked_fill_(~sees[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, kh, -1, length) @ values).view(b, kh, h // kh, n, d) / torch.where(total == 0, 1.0, total)
    token = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(s["q_start"][1:].long(), token, right=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(b, n, h, d)[seq, token - start[seq]].to(TYPES[case["type"]])
    if s["lse"] is None:
        return {"out": out}
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, n, h)[seq, token - start[seq]]
    return {"out": out, "lse": lse}


# --------------------------------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "attention": _exact_attention}[case["op"]](case, s)


def _exact_scale(case, rows, nth):
    """Steps (nth 0) or bases (nth 1) of rows, in 64 bits, from the bytes' bits."""
    blocks = case["dim"] // BLOCK
    at = case["dim"] * case["bits"] // 8 + 2 * blocks * nth
    raw = rows[..., at:at + 2 * blocks].long()
    bits = raw[..., 0::2] + 256 * raw[..., 1::2]
    exponent, fraction = (bits >> 10) & 31, (bits & 1023).double()
    size = torch.where(exponent == 0, fraction * 2.0 ** -24, (1024 + fraction) * torch.exp2((exponent - 25).double()))
    return torch.where(bits >= 32768, -size, size)


def _exact_values(case, rows):
    d, b = case["dim"], case["bits"]
    i = torch.arange(d, device="cuda")
    code = (rows[..., i * b // 8].long() >> (i * b % 8)) & ((1 << b) - 1)
    return code.double() * _exact_scale(case, rows, 0)[..., i // BLOCK] + _exact_scale(case, rows, 1)[..., i // BLOCK]


def _exact_half(x, up):
    """The fp16 at or next to each x (64 bits) on the asked side."""
    x = x.double()
    unit = torch.exp2(torch.clamp(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))), min=-14.0) - 10.0)
    return (torch.ceil(x / unit) if up else torch.floor(x / unit)) * unit


def _exact_write(case, s):
    """The definition's roundings of differences, quotients and products to 32 bits, the rest in 64."""
    out = {}
    slot = s["slots"]
    page = s["table"][0].long().repeat_interleave(case["page"])[:case["tokens"]]
    token = torch.arange(case["tokens"], device="cuda") % case["page"]
    for name in ("k", "v"):
        x = s[name].double().clamp(-LARGEST, LARGEST).unflatten(-1, (-1, BLOCK))
        base = _exact_half(x.min(-1).values, False)
        span = (x.max(-1).values - base).float().double()
        top = 2.0 ** case["bits"] - 1
        step = _exact_half((span / top).float(), True)
        rate = torch.where(step > 0, 1.0 / step, 0.0).float().double()
        code = torch.round(((x - base[..., None]).float().double() * rate[..., None]).float()).double().clamp(max=top)
        fresh = (code * step[..., None] + base[..., None]).flatten(-2)
        out[name] = torch.where((slot >= 0)[:, None, None], fresh, _exact_values(case, s[name + "_cache"][page, token]))
    return out


def _exact_read(case, s):
    _, ctx = _lengths(case)
    parts = {"k": [], "v": []}
    for b, (c, f) in enumerate(zip(ctx, _firsts(case, ctx))):
        pages = s["table"][b, :-(-c // case["page"])].long()
        for name in parts:
            parts[name].append(_exact_values(case, s[name + "_cache"][pages].flatten(0, 1)[f:c]))
    return {name: torch.cat(v) for name, v in parts.items()}


def _exact_attention(case, s):
    new, ctx = _lengths(case)
    if work(case)["flops"] > 8e12:
        return None
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, c) in enumerate(zip(new, ctx)):
        if c:
            pages = s["table"][b, :-(-c // case["page"])].long()
            place = torch.arange(c - n, c, device="cuda")
            t = torch.arange(c, device="cuda")
            hidden = t[None, :] > place[:, None]
            if case["window"]:
                hidden |= t[None, :] <= place[:, None] - case["window"]
            for kv in range(case["kv_heads"]):
                k = _exact_values(case, s["k_cache"][pages, :, kv].flatten(0, 1)[:c])
                v = _exact_values(case, s["v_cache"][pages, :, kv].flatten(0, 1)[:c])
                for head in range(kv * group, (kv + 1) * group):
                    a = torch.einsum("nd,cd->nc", s["q"][first:first + n, head].double(), k) / math.sqrt(case["dim"])
                    a.masked_fill_(hidden, -math.inf)
                    lse[first:first + n, head] = torch.logsumexp(a, 1)
                    out[first:first + n, head] = torch.softmax(a, 1) @ v
        first += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
