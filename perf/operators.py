"""Cases of the operators that stand between the library's GEMVs in a serving step: rotary positions with the
write into a paged cache, attention of new tokens over that cache, and sampling from the lm_head's logits.

Head layouts and the vocabulary are those of the decode workloads in qgemv_inputs/workloads.py: 16 query and 8
key/value heads of 128 (0.6b-class), 32 and 8 heads of 128 (4b-class), 151936 logits.  Page sizes, context
lengths and batch sizes are generic.  With ``own`` false, run() computes the operators in elementary torch
operations in 32 bits; with ``own`` true it calls the library.
"""
import math
import random

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
TYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
MASS = float(2 ** 42)  # sampling: the whole number that stands for a weight of exp(0)


def listed():
    return [
        # one decode token of the 4b-class model: the fp32 qkv row of the GEMV, rotated and put into the cache
        dict(name="rope-one-token", op="rope", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="none", source=F32, type=BF16, page=16, longest=4096, skipped=0),
        # a mixed step of the 0.6b-class model: 61 tokens, half of each head rotated in interleaved pairs, linear
        # scaling, fp16; every 9th token is padding of a fixed-size batch (no slot in the cache)
        dict(name="rope-61-tokens", op="rope", tokens=61, heads=16, kv_heads=8, dim=128, rot=64, layout="interleaved",
             scaling="linear", source=F16, type=F16, page=64, longest=20000, skipped=9),
        # a long prompt of the 4b-class model, frequencies scaled by parts for positions up to 131072
        dict(name="rope-prompt", op="rope", tokens=16000, heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             scaling="parts", source=BF16, type=BF16, page=64, longest=131072, skipped=0),
        # the smallest decode step: one sequence, one new token, a short chat
        dict(name="decode-short", op="attention", seqs=1, new=1, ctx=777, heads=32, kv_heads=8, dim=128, page=16,
             type=BF16, window=0, lse=False, idle=0, mix=1),
        # one sequence with a very long context: the keys have to be split over the whole GPU
        dict(name="decode-long", op="attention", seqs=1, new=1, ctx=100003, heads=32, kv_heads=8, dim=128, page=64,
             type=BF16, window=0, lse=False, idle=0, mix=2),
        # the usual serving step: 48 sequences of uneven length, one new token each
        dict(name="decode-batch", op="attention", seqs=48, new=1, ctx=16384, heads=32, kv_heads=8, dim=128, page=16,
             type=BF16, window=0, lse=False, idle=0, mix=3),
        # drafted tokens to be verified: 16 sequences of up to 5 new tokens, fp16, 0.6b-class heads; three idle
        # slots of a fixed-size batch whose rows see nothing; log-sum-exp wanted for a merge with another part
        dict(name="verify-drafts", op="attention", seqs=16, new=5, ctx=4000, heads=16, kv_heads=8, dim=128, page=32,
             type=F16, window=0, lse=True, idle=3, mix=4),
        # a chunk of a long prompt over what is in the cache already
        dict(name="chunk-2000-of-24000", op="attention", seqs=1, new=2000, ctx=24000, heads=32, kv_heads=8, dim=128,
             page=64, type=BF16, window=0, lse=False, idle=0, mix=5),
        # two whole prompts of uneven length
        dict(name="prompts", op="attention", seqs=2, new=6001, ctx=6001, heads=32, kv_heads=8, dim=128, page=64,
             type=BF16, window=0, lse=False, idle=0, mix=6),
        # one row of logits as the lm_head GEMV leaves them
        dict(name="sample-one-row", op="sample", rows=1, vocab=151936, type=F32, top_k=50, top_p=0.95, min_p=0.0,
             masked=0.0),
        # a batch of 16 rows with a settings mix: greedy rows, unfiltered rows, all filters; a grammar's mask on some
        dict(name="sample-16-rows", op="sample", rows=16, vocab=151936, type=F32, top_k=-1, top_p=0.9, min_p=0.05,
             masked=0.9),
        # a large batch of bf16 logits, nucleus only
        dict(name="sample-320-rows", op="sample", rows=320, vocab=151936, type=BF16, top_k=0, top_p=0.9, min_p=0.0,
             masked=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads, kv_heads = rng.choice([(16, 8), (32, 8)])
    kind = rng.choice([BF16, F16])
    op = rng.choice(["rope", "attention", "attention", "sample"])
    if op == "rope":
        return dict(op=op, tokens=_log_int(rng, 1, 16000), heads=heads, kv_heads=kv_heads, dim=128,
                    rot=rng.choice([32, 64, 96, 128]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "parts"]), source=rng.choice([F32, kind]), type=kind,
                    page=rng.choice([16, 32, 64]), longest=_log_int(rng, 2000, 131072),
                    skipped=rng.choice([0, 0, 7]))
    if op == "sample":
        return dict(op=op, rows=_log_int(rng, 1, 320), vocab=rng.choice([151936, _log_int(rng, 1000, 151936)]),
                    type=rng.choice([F32, BF16, F16]), top_k=rng.choice([-1, 0, _log_int(rng, 1, 1000)]),
                    top_p=rng.choice([1.0, 0.9, 0.95]), min_p=rng.choice([0.0, 0.02]),
                    masked=rng.choice([0.0, 0.5, 0.98]))
    page, mix = rng.choice([16, 32, 64]), rng.randrange(1 << 30)
    if rng.random() < 0.6:  # decode and drafts
        new = rng.choice([1, 1, _log_int(rng, 2, 16)])
        ctx = _log_int(rng, 16, 100003)
        seqs = _log_int(rng, 1, max(1, min(48, 48 * 16384 // (ctx * new))))
        return dict(op=op, seqs=seqs, new=new, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=128, page=page, type=kind,
                    window=rng.choice([0, 0, 1024]), lse=rng.choice([False, True]),
                    idle=rng.choice([0, seqs // 4]), mix=mix)
    new = _log_int(rng, 17, 6001)
    ctx = _log_int(rng, new, max(new, min(24000, 36000000 // new)))
    return dict(op=op, seqs=rng.choice([1, 1, 2]), new=new, ctx=ctx, heads=heads, kv_heads=kv_heads, dim=128, page=page,
                type=kind, window=rng.choice([0, 0, 1024]), lse=False, idle=0, mix=mix)


# ---------------------------------------------------------------------------------------------------- sizes

def _lengths(case):
    """New tokens and context of each sequence: the first has the case's, the others fewer, idle ones no context."""
    r = random.Random(case["mix"])
    new, ctx = [], []
    for b in range(case["seqs"]):
        n = case["new"] if b == 0 else r.randint(max(1, case["new"] // 2), case["new"])
        c = case["ctx"] if b == 0 else max(n, int(case["ctx"] * math.exp(-r.random() * math.log(8.0))))
        if b >= case["seqs"] - case["idle"]:
            n, c = 1, 0
        new.append(n)
        ctx.append(c)
    return new, ctx


def work(case):
    size = 4 if case.get("source", case["type"]) == F32 else 2
    if case["op"] == "rope":
        t, rows, keys = case["tokens"], case["heads"] + 2 * case["kv_heads"], case["heads"] + case["kv_heads"]
        live = t - (t // case["skipped"] if case["skipped"] else 0)
        return {"bytes": t * rows * case["dim"] * size + t * case["heads"] * case["dim"] * 2
                + live * 2 * case["kv_heads"] * case["dim"] * 2 + t * 12 + case["rot"] * 4,
                "flops": 3 * t * keys * case["rot"]}
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * (4 if case["type"] == F32 else 2) + 28),
                "flops": 4 * case["rows"] * case["vocab"]}
    new, ctx = _lengths(case)
    seen, keys = 0, 0  # pairs of a query and a key it sees; keys that some query sees
    for n, c in zip(new, ctx):
        w = case["window"] or c
        if not c:
            continue
        seen += sum(min(w, c - n + j + 1) for j in range(n))
        keys += min(c, w + n - 1)
    token = case["heads"] * case["dim"] * 2
    return {"bytes": 2 * sum(new) * token + 2 * keys * case["kv_heads"] * case["dim"] * 2
            + (4 * sum(new) * case["heads"] if case["lse"] else 0),
            "flops": 4 * seen * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------------------------------- inputs

def _inverse_frequencies(case):
    """Radians a position of each rotated pair, in 64 bits."""
    r = case["rot"]
    f = [10000.0 ** (-2.0 * i / r) if case["scaling"] == "none" else 1e6 ** (-2.0 * i / r) for i in range(r // 2)]
    if case["scaling"] == "linear":
        f = [x / 4.0 for x in f]
    if case["scaling"] == "parts":  # slow pairs are interpolated by 4, fast ones kept, a ramp between
        def pair(turns):
            return r * math.log(32768.0 / (turns * 2 * math.pi)) / (2 * math.log(1e6))
        lo, hi = max(0, math.floor(pair(32.0))), min(r - 1, math.ceil(pair(1.0)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo))) for i in range(r // 2)]
        f = [x / 4.0 * g + x * (1.0 - g) for x, g in zip(f, ramp)]
    return f


def _magnitude(case):
    return 0.1 * math.log(4.0) + 1.0 if case["scaling"] == "parts" else 1.0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "op": case["op"]}
    {"rope": _prepare_rope, "attention": _prepare_attention, "sample": _prepare_sample}[case["op"]](s, case, g)
    return s


def _prepare_rope(s, case, g):
    t, h, kh, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    qkv = torch.randn(t, (h + 2 * kh) * d, generator=g, device="cuda").to(TYPES[case["source"]])
    s["q"] = qkv[:, :h * d].view(t, h, d)
    s["k"] = qkv[:, h * d:(h + kh) * d].view(t, kh, d)
    s["v"] = qkv[:, (h + kh) * d:].view(t, kh, d)
    start = int(torch.randint(0, max(1, case["longest"] - t), (1,), generator=g, device="cuda"))
    s["positions"] = (start + torch.arange(t, device="cuda")).to(torch.int32)
    pages = -(-t // page) + 2
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    slots = order[i // page] * page + i % page
    if case["skipped"]:
        slots[case["skipped"] - 1::case["skipped"]] = -1
    s["slots"] = slots
    s["freqs"] = torch.tensor([int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in _inverse_frequencies(case)],
                              dtype=torch.int64, device="cuda")
    s["k_cache"] = torch.zeros(pages, page, kh, d, dtype=TYPES[case["type"]], device="cuda")
    s["v_cache"] = torch.zeros_like(s["k_cache"])
    s["q_out"] = torch.empty(t, h, d, dtype=TYPES[case["type"]], device="cuda")
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        s["args"] = qg.rope_args(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["q_out"],
                                 cache=qg.kv_cache(s["k_cache"], s["v_cache"]), slots=s["slots"], rot_dim=case["rot"],
                                 layout=case["layout"], mscale=_magnitude(case))


def _prepare_attention(s, case, g):
    new, ctx = _lengths(case)
    h, kh, d, page, kind = case["heads"], case["kv_heads"], case["dim"], case["page"], TYPES[case["type"]]
    need = [-(-c // page) for c in ctx]
    most, total = max(1, max(need)), sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(new), most, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    table = order[table.long().cuda()]
    s["k_cache"] = torch.randn(total, page, kh, d, generator=g, device="cuda", dtype=torch.float32).to(kind)
    s["v_cache"] = torch.randn(total, page, kh, d, generator=g, device="cuda", dtype=torch.float32).to(kind)
    s["k_cache"][table[:, 0].long(), 0] *= 2.0  # the first token draws attention
    s["q"] = (1.5 * torch.randn(sum(new), h, d, generator=g, device="cuda")).to(kind)
    s["table"] = table.contiguous()
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    s["kv_len"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s["max_new"], s["max_ctx"] = max(new), max(ctx)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(sum(new), h, dtype=torch.float32, device="cuda") if case["lse"] else None
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        nbytes = qg.qgemv_attn_scratch_bytes(len(new), sum(new), h, kh, d, s["max_new"], s["max_ctx"])
        s["scratch"] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        s["args"] = qg.attn_args(s["q"], qg.kv_cache(s["k_cache"], s["v_cache"]), s["table"], s["q_start"], s["kv_len"],
                                 s["out"], s["scratch"], max_q=s["max_new"], max_kv=s["max_ctx"], scale=s["scale"],
                                 window=case["window"], lse=s["lse"])


def _prepare_sample(s, case, g):
    m, n = case["rows"], case["vocab"]
    x = torch.randn(m, n, generator=g, device="cuda") * 2.5
    # a few candidates stand out, as a trained lm_head's do
    hot = torch.randint(0, n, (m, 24), generator=g, device="cuda")
    x.scatter_add_(1, hot, 8.0 + 2.0 * torch.randn(m, 24, generator=g, device="cuda"))
    if case["masked"]:  # every third row has a mask that leaves a share of the vocabulary
        gone = torch.rand(m, n, generator=g, device="cuda") < case["masked"]
        gone[1::3] = False
        gone[2::3] = False
        x = x.masked_fill(gone, float("-inf"))
    s["logits"] = x.to(TYPES[case["type"]])
    i = torch.arange(m, device="cuda")
    s["temperature"] = 0.6 + 0.1 * (i % 7).float()
    k, p, low = case["top_k"], case["top_p"], case["min_p"]
    if k < 0:  # each row has its own settings
        s["temperature"] = torch.where(i % 5 == 4, 0.0, s["temperature"])
        s["top_k"] = torch.where(i % 4 == 0, 0, 20 + 37 * i).to(torch.int32)
        s["top_p"] = torch.where(i % 3 == 0, 1.0, p).float()
        s["min_p"] = torch.where(i % 2 == 0, 0.0, low).float()
    else:
        s["top_k"] = torch.full((m,), k, dtype=torch.int32, device="cuda")
        s["top_p"] = torch.full((m,), p, dtype=torch.float32, device="cuda")
        s["min_p"] = torch.full((m,), low, dtype=torch.float32, device="cuda")
    s["u"] = torch.rand(m, generator=g, device="cuda")
    s["token"] = torch.empty(m, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(m, dtype=torch.float32, device="cuda")


# ------------------------------------------------------------------------------------------------- one pass

def run(state):
    return {"rope": _rope, "attention": _attention, "sample": _sample}[state["op"]](state)


def _rope(s):
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_rope(s["args"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    case = s["case"]
    r, kind = case["rot"], TYPES[case["type"]]
    turns = (s["positions"].long()[:, None] * s["freqs"][None, :]) >> 32  # the whole turns wrap away
    angle = turns.float() * (2.0 * math.pi / 2.0 ** 32)
    c, n = (torch.cos(angle) * _magnitude(case))[:, None], (torch.sin(angle) * _magnitude(case))[:, None]

    def turned(x):
        x = x.float()
        if case["layout"] == "half":
            a, b = x[..., :r // 2], x[..., r // 2:r]
            return torch.cat([a * c - b * n, b * c + a * n, x[..., r:]], -1)
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        return torch.cat([torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2), x[..., r:]], -1)

    s["q_out"].copy_(turned(s["q"]).to(kind))
    # tokens without a slot go to a row past the cache's, which is dropped
    kc, vc = s["k_cache"].view(-1, *s["k"].shape[1:]), s["v_cache"].view(-1, *s["v"].shape[1:])
    at = torch.where(s["slots"] < 0, kc.shape[0], s["slots"])
    for cache, x in ((kc, turned(s["k"])), (vc, s["v"].float())):
        wide = torch.cat([cache, cache[:1]])
        wide[at] = x.to(kind)
        cache.copy_(wide[:-1])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attention(s):
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_attn(s["args"])
        return {"out": s["out"]} if s["lse"] is None else {"out": s["out"], "lse": s["lse"]}
    case = s["case"]
    h, kh, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    b, n, length = s["kv_len"].numel(), s["max_new"], max(1, s["max_ctx"])
    t = torch.arange(length, device="cuda")
    slot = s["table"].long()[:, t // page] * page + t % page  # [b, length]
    keys = s["k_cache"].view(-1, kh, d)[slot].float().permute(0, 2, 3, 1)  # [b, kh, d, length]
    values = s["v_cache"].view(-1, kh, d)[slot].float().permute(0, 2, 1, 3)  # [b, kh, length, d]
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


def _sample(s):
    if own:
        import quantized_weight_gemv_quantize_gb300 as qg
        qg.qgemv_sample(s["logits"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], s["token"], s["prob"])
        return {"token": s["token"], "prob": s["prob"]}
    x = s["logits"].float()
    n = x.shape[1]
    greedy = s["temperature"] <= 0
    rate = 1.0 / torch.where(greedy, 1.0, s["temperature"])
    e = torch.exp((x - x.amax(-1, keepdim=True)) * rate[:, None])
    weight = (e * MASS).to(torch.int64)  # whole numbers: their sums do not depend on the order
    _, order = torch.sort(x, dim=-1, descending=True, stable=True)
    sorted_weight = weight.gather(1, order)
    k = torch.where(greedy, 1, torch.where(s["top_k"] > 0, s["top_k"], n))
    rank = torch.arange(n, device="cuda")[None, :]
    keep = rank < k[:, None]
    before = torch.cumsum(sorted_weight, 1) - sorted_weight
    total = torch.where(keep, sorted_weight, 0).sum(1)
    keep &= (before.double() < (s["top_p"].double() * total.double())[:, None]) | (s["top_p"] >= 1)[:, None]
    keep &= e.gather(1, order) >= s["min_p"][:, None]
    keep |= rank == 0
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    reach = torch.cumsum(torch.where(kept, weight, 0), 1)
    total = reach[:, -1]
    target = torch.minimum((s["u"].double() * total.double()).to(torch.int64), total - 1)
    token = (reach <= target[:, None]).sum(1)
    prob = e.gather(1, token[:, None]).squeeze(1) / (total.float() / MASS)
    return {"token": token.to(torch.int32), "prob": prob}


# --------------------------------------------------------------------------------------- in 64 bits, apart

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attention": _exact_attention, "sample": _exact_sample}[case["op"]](case, s)


def _exact_rope(case, s):
    f = torch.tensor(_inverse_frequencies(case), dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full((), _magnitude(case), dtype=torch.float64, device="cuda"),
                    s["positions"].double()[:, None, None] * f)
    r = case["rot"]

    def turned(x):
        x = x.double().clone()
        if case["layout"] == "half":
            y = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * z
            x[..., :r // 2], x[..., r // 2:r] = y.real, y.imag
        else:
            y = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * z
            x[..., 0:r:2], x[..., 1:r:2] = y.real, y.imag
        return x

    out = {"q": turned(s["q"])}
    live = (s["slots"] >= 0).nonzero().squeeze(1)
    for name, x in (("k_cache", turned(s["k"])), ("v_cache", s["v"].double())):
        cache = s[name].double()
        cache[s["slots"][live] // case["page"], s["slots"][live] % case["page"]] = x[live]
        out[name] = cache
    return out


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
            for head in range(case["heads"]):
                k = s["k_cache"][pages, :, head // group].flatten(0, 1)[:c].double()
                v = s["v_cache"][pages, :, head // group].flatten(0, 1)[:c].double()
                a = torch.einsum("nd,cd->nc", s["q"][first:first + n, head].double(), k) / math.sqrt(case["dim"])
                a.masked_fill_(hidden, -math.inf)
                lse[first:first + n, head] = torch.logsumexp(a, 1)
                out[first:first + n, head] = torch.softmax(a, 1) @ v
        first += n
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def _exact_sample(case, s):
    x = s["logits"].double()
    prob = torch.empty(case["rows"], dtype=torch.float64, device="cuda")
    for i in range(case["rows"]):
        t, k, p, low = (float(s[name][i]) for name in ("temperature", "top_k", "top_p", "min_p"))
        if t <= 0:
            prob[i] = 1.0
            continue
        q = torch.softmax(x[i] / t, 0)
        _, order = torch.sort(q, descending=True, stable=True)
        order = order[:int(k)] if k > 0 else order
        d = q[order] / q[order].sum()
        if p < 1:
            order = order[(torch.cumsum(d, 0) - d < p) | (torch.arange(d.numel(), device="cuda") == 0)]
        order = order[q[order] >= low * q[order[0]]]
        order, _ = torch.sort(order)
        d = q[order] / q[order].sum()
        at = torch.searchsorted(torch.cumsum(d, 0), s["u"][i:i + 1].double(), right=True)
        prob[i] = d[at.clamp(max=d.numel() - 1)].squeeze()
    return {"token": None, "prob": prob}
