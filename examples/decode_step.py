"""A decode step from the library's parts: quantize, qkv GEMVs, rotary positions with the cache write, attention over the paged
cache, o GEMV, lm_head GEMV, sampling; captured as one CUDA graph and replayed.

The "model" is one attention sublayer of the 0.6b-class shapes (16 query and 8 key/value heads of 128) between an embedding and
an lm_head, with random weights: it shows the calls, their order and their buffers, not a language.

    python examples/decode_step.py [--seqs 4] [--prompt 100] [--steps 32] [--cache bf16|Q8|Q4]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import qgemv_inputs as gen  # noqa: E402
import quantized_weight_gemv_quantize_gb300 as qg  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, VOCAB, PAGE = 1024, 16, 8, 128, 151936, 32


class Decoder:
    """Weights, cache and buffers of `seqs` sequences of at most `longest` tokens.  seqs * new <= 16: the GEMVs' rows."""

    def __init__(self, seqs, longest, seed=0, kind="bf16"):
        def weight(fmt, n, k, tag):
            return torch.from_numpy(gen.weights(fmt, n, k, gen.derive(seed, tag))).cuda()

        self.seqs, self.longest = seqs, longest
        self.wq, self.wk, self.wv = (weight("Q4_K", n * DIM, HIDDEN, i) for i, n in enumerate((HEADS, KV_HEADS, KV_HEADS)))
        self.wo, self.head = weight("Q4_K", HIDDEN, HEADS * DIM, 3), weight("Q8_0", VOCAB, HIDDEN, 4)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda")
        pages = -(-longest // PAGE)
        packed = kind != "bf16"
        row = (qg.qgemv_cache_row_bytes(kind, DIM), torch.uint8) if packed else (DIM, torch.bfloat16)
        self.k_cache = torch.zeros(seqs * pages, PAGE, KV_HEADS, row[0], dtype=row[1], device="cuda")
        self.v_cache = torch.zeros_like(self.k_cache)
        self.cache = qg.packed_cache(kind, self.k_cache, self.v_cache, DIM) if packed else qg.kv_cache(self.k_cache, self.v_cache)
        self.table = torch.randperm(seqs * pages, generator=g, device="cuda").to(torch.int32).view(seqs, pages)
        freqs, self.mscale = qg.qgemv_rope_freqs(DIM, 1e6)
        self.freqs = freqs.cuda()
        self.kv_len = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        need = qg.qgemv_attn_scratch_bytes(seqs, 16, HEADS, KV_HEADS, DIM, 16 // seqs, longest, self.cache)  # of every smaller call too
        self.scratch = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.buffers = {}

    def block(self, new):
        """Buffers and argument records of a call with `new` tokens a sequence, made once."""
        if new in self.buffers:
            return self.buffers[new]
        m = self.seqs * new
        f32 = lambda *n: torch.empty(*n, device="cuda")  # noqa: E731
        b = dict(m=m, x=f32(m, HIDDEN), q=f32(m, HEADS, DIM), k=f32(m, KV_HEADS, DIM), v=f32(m, KV_HEADS, DIM), y=f32(m, HIDDEN),
                 rotated=torch.empty(m, HEADS, DIM, dtype=torch.bfloat16, device="cuda"),
                 positions=torch.empty(m, dtype=torch.int32, device="cuda"),
                 slots=torch.empty(m, dtype=torch.int64, device="cuda"),
                 xq=torch.empty(qg.qgemv_act_bytes(m, HEADS * DIM), dtype=torch.uint8, device="cuda"))
        b["out"] = torch.empty_like(b["rotated"])
        b["starts"] = torch.arange(0, m + 1, new, dtype=torch.int32, device="cuda")
        b["qkv"] = qg.mats_array([(self.wq, b["q"], HEADS * DIM), (self.wk, b["k"], KV_HEADS * DIM), (self.wv, b["v"], KV_HEADS * DIM)])
        b["rope"] = qg.rope_args(b["q"], b["k"], b["v"], b["positions"], self.freqs, b["rotated"], cache=self.cache,
                                 slots=b["slots"], mscale=self.mscale)
        b["attn"] = qg.attn_args(b["rotated"], self.cache, self.table, b["starts"], self.kv_len, b["out"], self.scratch,
                                 max_q=new, max_kv=self.longest, scale=DIM ** -0.5)
        self.buffers[new] = b
        return b

    def attend(self, tokens, new, flags=0):
        """The sublayer on `new` tokens a sequence (int [seqs * new], a sequence's together); returns its fp32 output rows."""
        b = self.block(new)
        m = b["m"]
        # places of the new tokens, on the device: nothing here depends on the host's knowledge of the lengths
        at = (self.kv_len[:, None] + torch.arange(new, device="cuda", dtype=torch.int32)).long()
        b["positions"].copy_(at.flatten())
        b["slots"].copy_((self.table.gather(1, at // PAGE).long() * PAGE + at % PAGE).flatten())
        self.kv_len += new
        torch.index_select(self.embedding, 0, tokens, out=b["x"])
        qg.qgemv_multi("Q4_K", b["qkv"], "f32", b["x"], m, HIDDEN, flags=flags)
        qg.qgemv_rope(b["rope"], flags)
        qg.qgemv_attn(b["attn"], flags)
        qg.qgemv_quantize_act_typed("bf16", b["out"], m, HEADS * DIM, b["xq"], flags)
        qg.qgemv_ex("Q4_K", self.wo, b["xq"], b["y"], m, HIDDEN, HEADS * DIM, flags)
        y = b["y"]
        y.mul_(0.3 * y.square().mean(-1, keepdim=True).add_(1e-6).rsqrt_())  # (the random weights' output, to a third of the input's size)
        return y.add_(b["x"])

    def prompt(self, tokens):
        """Puts all but the last of each sequence's tokens [seqs, n] through the sublayer, as many at a time as the GEMVs take."""
        step = 16 // self.seqs
        for i in range(0, tokens.shape[1] - 1, step):
            part = tokens[:, i:min(i + step, tokens.shape[1] - 1)]
            self.attend(part.flatten(), part.shape[1])

    def sampler(self, temperature=0.8, top_k=50, top_p=0.95):
        s, full = self.seqs, torch.full
        self.hq = torch.empty(qg.qgemv_act_bytes(s, HIDDEN), dtype=torch.uint8, device="cuda")
        self.logits = torch.empty(s, VOCAB, device="cuda")
        self.settings = (full((s,), temperature, device="cuda"), full((s,), top_k, dtype=torch.int32, device="cuda"),
                         full((s,), top_p, device="cuda"), None)
        self.u = torch.empty(s, device="cuda")
        self.token = torch.empty(s, dtype=torch.int32, device="cuda")
        self.prob = torch.empty(s, device="cuda")

    def step(self, flags=0):
        """One token for every sequence: from self.token to self.token."""
        y = self.attend(self.token, 1, flags)
        qg.qgemv_quantize_act_ex(y, self.seqs, HIDDEN, self.hq, flags)
        qg.qgemv_ex("Q8_0", self.head, self.hq, self.logits, self.seqs, VOCAB, HIDDEN, flags)
        qg.qgemv_sample(self.logits, *self.settings, self.u, self.token, self.prob, flags)


def generate(seqs, prompt, steps, seed=0, graph=True, kind="bf16"):
    """The sampled tokens [steps, seqs], their probabilities, and the time of a step in microseconds."""
    d = Decoder(seqs, prompt + steps, seed, kind)
    d.sampler()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    tokens = torch.randint(0, VOCAB, (seqs, prompt), generator=g, device="cuda", dtype=torch.int32)
    u = torch.rand(steps, seqs, generator=g, device="cuda")
    d.prompt(tokens)
    last, length = tokens[:, -1].contiguous(), d.kv_len.clone()
    d.token.copy_(last), d.u.copy_(u[0])
    d.step()  # every kernel has been launched once before the capture
    run = d.step
    if graph:
        c = torch.cuda.CUDAGraph()
        with torch.cuda.graph(c):
            d.step(qg.QGEMV_FLAG_PDL)
        run = c.replay
    d.token.copy_(last), d.kv_len.copy_(length)
    out, prob = torch.empty(steps, seqs, dtype=torch.int32, device="cuda"), torch.empty(steps, seqs, device="cuda")
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(steps):
        d.u.copy_(u[i])
        run()
        out[i].copy_(d.token), prob[i].copy_(d.prob)
    torch.cuda.synchronize()
    return out, prob, (time.perf_counter() - t) / steps * 1e6


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=100)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--cache", choices=("bf16", "Q8", "Q4"), default="bf16")
    a = p.parse_args()
    if not 1 <= a.seqs <= 16 or a.prompt < 1 or a.steps < 1:
        p.error("1 to 16 sequences, at least one token and one step")
    qg.build()
    for graph in (False, True):
        out, prob, us = generate(a.seqs, a.prompt, a.steps, graph=graph, kind=a.cache)
        print(f"{'one graph a step' if graph else 'call by call'}: {us:.1f} us a step; sequence 0: {out[:8, 0].tolist()} ...")
    sys.exit(1 if qg.qgemv_device_error() else 0)
