"""The operators between the GEMVs on the GPU, against their formulas in 64 bits (numpy).

Tolerances, from the arithmetic:
 - a value is rounded once to its type: u |ref| with u = 2^-8 (bf16), 2^-11 (f16), 2^-24 (fp32), plus the smallest step of f16;
 - rotary positions: fp32 products and sines of an angle good to 2^-24 of a half turn: 16 * 2^-24 (|a| + |b|);
 - attention: a score is an fp32 sum of products that are exact in fp32, off by at most D = 2^-20 scale max|q||k|; then a
   probability is off by e^(2D) and its rounding to 16 bits, and the output by that share of A = sum p |v|:
   u |ref| + (u + 4 D + 2^-18) A;  lse is off by D + 2^-20 max(1, |lse|);
 - sampling: masses are off by the 2 ulp of expf and the fp32 of (x - max) / T, a few 2^-24 of the exponent: shares of the
   whole are good to EPS = 1e-5 at the logits used here, so a token has to hold u within EPS of its interval.
"""
import math

import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.build()
    qg.lib()
    qg.qgemv_device_error(reset=True)
    yield
    assert qg.qgemv_device_error() == 0


@pytest.fixture(params=["16-row", "128-row"])
def kernel(request):
    """Attention by one kernel or the other, whatever the planner would take (heads beyond 128 go to the first)."""
    qg.qgemv_tune_attn(1 if request.param == "16-row" else 2)
    yield request.param
    qg.qgemv_tune_attn(0)


def rnd(rng, shape, dtype, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)) * scale).to(dtype).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol):
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (float((err - tol).max()), np.unravel_index(np.argmax(err - tol), err.shape))


# ------------------------------------------------------------------------------------------------- rotary positions

def turned(x, pos, freqs, rot, layout, ms):
    """x [T, H, D] fp64, in 64 bits; the angle from the whole-number turn table, exactly."""
    t = np.array([[((int(p) * int(f)) % 2 ** 64) / 2.0 ** 64 for f in freqs] for p in pos]) * 2 * math.pi
    c, s = (np.cos(t) * ms)[:, None], (np.sin(t) * ms)[:, None]
    y, m = x.copy(), np.zeros_like(x)
    i, j = (np.arange(rot // 2), np.arange(rot // 2, rot)) if layout == "half" else (np.arange(0, rot, 2), np.arange(1, rot, 2))
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    m[..., i] = m[..., j] = (np.abs(x[..., i]) + np.abs(x[..., j])) * abs(ms)
    return y, m


ROPE = [
    # tokens, heads, kv heads, dim, rot, layout, input, output, cache, page
    (1, 32, 8, 128, 128, "half", torch.float32, torch.bfloat16, torch.bfloat16, 16),
    (61, 16, 8, 128, 64, "interleaved", torch.float16, torch.float16, torch.float16, 64),
    (7, 5, 1, 64, 64, "half", torch.bfloat16, torch.float32, torch.float16, 1),
    (33, 3, 3, 80, 20, "half", torch.float32, torch.float32, torch.bfloat16, 7),        # pairs that split no 16-byte piece
    (33, 3, 3, 80, 20, "interleaved", torch.bfloat16, torch.bfloat16, torch.bfloat16, 7),
    (9, 1, 1, 8, 2, "half", torch.float16, torch.float16, torch.float16, 3),
    (300, 4, 2, 256, 256, "half", torch.float32, torch.float16, torch.bfloat16, 5),
    (5, 4, 2, 256, 254, "interleaved", torch.float32, torch.float16, torch.bfloat16, 5),
    (2500, 2, 1, 96, 96, "half", torch.bfloat16, torch.bfloat16, torch.bfloat16, 32),
]


@pytest.mark.parametrize("T,H,KH,D,rot,layout,xt,ot,ct,page", ROPE)
def test_rope_and_append(T, H, KH, D, rot, layout, xt, ot, ct, page):
    rng = np.random.default_rng(T * 131 + rot)
    qkv = rnd(rng, (T, (H + 2 * KH) * D), xt)  # slices of one row, as a merged GEMV writes them
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, KH * D, KH * D], 1))
    pos = rng.integers(-5, 1 << 20, T).astype(np.int32)
    pos[0] = 0
    if T > 4:
        pos[1:4] = (2 ** 31 - 1, -2 ** 31, 1)
    freqs, ms = qg.qgemv_rope_freqs(rot, 10000.0, "parts" if rot > 32 else "none", 4.0, trained=4096.0)
    pages = -(-T // page) + 1
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2::5] = -1
    kc = torch.full((pages, page, KH, D), 3.0, dtype=ct, device="cuda")
    vc = torch.full_like(kc, 5.0)
    qo, ko = (torch.empty(T, n, D, dtype=ot, device="cuda") for n in (H, KH))
    a = qg.rope_args(q, k, v, torch.from_numpy(pos).cuda(), freqs.cuda(), qo, ko, qg.kv_cache(kc, vc),
                     torch.from_numpy(slots).cuda(), rot, layout, ms)
    qg.qgemv_route_reset()
    qg.qgemv_rope(a)
    assert qg.qgemv_route_counts()[qg.ROUTE_ROPE] == 1
    table = [int(x) % 2 ** 64 for x in freqs.tolist()]
    for x, y in ((q, qo), (k, ko)):
        ref, m = turned(f64(x), pos, table, rot, layout, ms)
        close(y, ref, U[ot] * np.abs(ref) + TINY[ot] + 16 * 2.0 ** -24 * m)
    ref, m = turned(f64(k), pos, table, rot, layout, ms)
    live = slots >= 0
    flat = lambda t: t.flatten(0, 1)  # noqa: E731
    close(flat(kc)[slots[live]], ref[live], (U[ct] * np.abs(ref) + TINY[ct] + 16 * 2.0 ** -24 * m)[live])
    assert torch.equal(flat(vc)[slots[live]], v[torch.from_numpy(live).cuda()].to(ct))
    rest = np.setdiff1d(np.arange(pages * page), slots[live])
    assert bool((flat(kc)[rest] == 3.0).all()) and bool((flat(vc)[rest] == 5.0).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("order", ["page-token-head", "page-head-token"])
def test_rope_in_place_and_cache_orders(layout, order):
    rng = np.random.default_rng(5)
    T, H, KH, D, page = 19, 8, 2, 64, 4
    qkv = rnd(rng, (T, (H + 2 * KH) * D), torch.bfloat16)
    before = qkv.clone()
    cut = lambda t: [s.unflatten(1, (-1, D)) for s in t.split([H * D, KH * D, KH * D], 1)]  # noqa: E731
    q, k, v = cut(qkv)
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device="cuda")
    freqs, _ = qg.qgemv_rope_freqs(D)
    shape = (8, page, KH, D) if order == "page-token-head" else (8, KH, page, D)
    kc, vc = (torch.zeros(2, *shape, dtype=torch.bfloat16, device="cuda").select(0, i) for i in (0, 1))
    if order == "page-head-token":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    slots = torch.arange(T, dtype=torch.int64, device="cuda") + 2
    qg.qgemv_rope(qg.rope_args(q, k, v, pos, freqs.cuda(), q, k, qg.kv_cache(kc, vc), slots, layout=layout))
    q0, k0, v0 = cut(before)
    for x, y in ((q0, q), (k0, k)):
        ref, m = turned(f64(x), pos.cpu().numpy(), freqs.tolist(), D, layout, 1.0)
        close(y, ref, U[torch.bfloat16] * np.abs(ref) + 16 * 2.0 ** -24 * m)
    assert torch.equal(v, v0)
    at = (slots // page, slots % page)
    assert torch.equal(kc[at], k) and torch.equal(vc[at], v0)
    # a single operand each: queries only, keys only
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    qg.qgemv_rope(qg.rope_args(q0, None, None, pos, freqs.cuda(), qo, layout=layout))
    qg.qgemv_rope(qg.rope_args(None, k0, None, pos, freqs.cuda(), None, ko, layout=layout))
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_rope_slot_beyond_the_cache_is_skipped_and_reported():
    rng = np.random.default_rng(6)
    q, k, v = (rnd(rng, (3, 2, 16), torch.bfloat16) for _ in range(3))
    kc = torch.zeros(2, 4, 2, 16, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    slots = torch.tensor([1, 8, 2 ** 62], dtype=torch.int64, device="cuda")
    freqs, _ = qg.qgemv_rope_freqs(16)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    qg.qgemv_rope(qg.rope_args(q, k, v, pos, freqs.cuda(), torch.empty_like(q), cache=qg.kv_cache(kc, vc), slots=slots))
    assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
    assert torch.equal(kc[0, 1], k[0]) and int((kc != 0).any(-1).sum()) == 2 and int((vc != 0).any(-1).sum()) == 2


# -------------------------------------------------------------------------------------------------------- attention

class Step:
    """A batch: sequences with `new[b]` new tokens over contexts of `ctx[b]` tokens in shuffled pages."""

    def __init__(self, seed, new, ctx, H, KH, D, page, dtype, order="token-head", junk=float("nan"), scale=None):
        rng = np.random.default_rng(seed)
        self.new, self.ctx, self.H, self.KH, self.D, self.page, self.dtype = new, ctx, H, KH, D, page, dtype
        need = [-(-c // page) for c in ctx]
        total = sum(need) + 2
        shape = (total, page, KH, D) if order == "token-head" else (total, KH, page, D)
        self.kc, self.vc = (torch.full(shape, junk, dtype=dtype, device="cuda") for _ in range(2))
        if order != "token-head":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        perm = rng.permutation(total).astype(np.int32)
        table = np.full((len(ctx), max([1] + need)), 2 ** 30, np.int32)  # entries that no context reaches
        at = 0
        self.k, self.v = [], []
        for b, c in enumerate(ctx):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            k, v = rnd(rng, (c, KH, D), dtype), rnd(rng, (c, KH, D), dtype)
            self.k.append(k), self.v.append(v)
            t = np.arange(c)
            where = (torch.from_numpy(table[b, t // page].astype(np.int64)).cuda(), torch.from_numpy(t % page).cuda())
            self.kc[where], self.vc[where] = k, v
        self.table = torch.from_numpy(table).cuda()
        self.q = rnd(rng, (sum(new), H, D), dtype, 1.5)
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale

    def args(self, causal=True, window=0, lse=True, scratch=None, q=None, out=None, max_q=None, max_kv=None):
        max_q, max_kv = max(self.new) if max_q is None else max_q, max(self.ctx) if max_kv is None else max_kv
        q = self.q if q is None else q
        self.out = torch.full_like(q.contiguous(), 7.0) if out is None else out
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        n = qg.qgemv_attn_scratch_bytes(len(self.new), q.shape[0], self.H, self.KH, self.D, max_q, max_kv)
        self.scratch = torch.zeros(n, dtype=torch.uint8, device="cuda") if scratch is None else scratch
        return qg.attn_args(q, qg.kv_cache(self.kc, self.vc), self.table, self.starts, self.lens, self.out, self.scratch, max_q,
                            max_kv, self.scale, causal, window, self.lse)

    def check(self, causal=True, window=0):
        out, lse, first, u = f64(self.out), None if self.lse is None else f64(self.lse), 0, U[self.dtype]
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            q, k, v = f64(self.q[first:first + n]), f64(self.k[b]), f64(self.v[b])
            pos = c - n + np.arange(n)
            t = np.arange(c)
            sees = np.ones((n, c), bool)
            if causal or window:
                sees &= t[None] <= pos[:, None]
            if window:
                sees &= t[None] > pos[:, None] - window
            for h in range(self.H):
                kh, vh, qh = k[:, h // (self.H // self.KH)], v[:, h // (self.H // self.KH)], q[:, h]
                s = np.where(sees, self.scale * (qh @ kh.T), -np.inf)
                top = s.max(1, initial=-np.inf, keepdims=True)
                top = np.where(np.isinf(top), 0.0, top)
                p = np.exp(s - top)
                l = p.sum(1, keepdims=True)
                p = p / np.where(l == 0, 1, l)
                ref, A = p @ vh, p @ np.abs(vh)
                off = 2.0 ** -20 * abs(self.scale) * (np.linalg.norm(qh, axis=1) * np.linalg.norm(kh, axis=1).max(initial=0.0))[:, None]
                tol = u * np.abs(ref) + (u + 4 * off + 2.0 ** -18) * A + TINY[self.dtype]
                err = np.abs(out[first:first + n, h] - ref)
                assert np.all(err <= tol), (b, h, float((err - tol).max()), np.unravel_index((err - tol).argmax(), err.shape))
                if lse is not None:
                    with np.errstate(divide="ignore"):
                        want = np.where(l[:, 0] > 0, top[:, 0] + np.log(l[:, 0]), -np.inf)
                    got = lse[first:first + n, h]
                    empty = np.isinf(want)
                    assert np.array_equal(np.isneginf(got), empty)
                    got, want, off = got[~empty], want[~empty], off[~empty, 0]
                    assert np.all(np.abs(got - want) <= off + 2.0 ** -20 * np.maximum(1, np.abs(want)))
            first += n


B16, H16 = torch.bfloat16, torch.float16
ATTN = [
    # new tokens, contexts, heads, kv heads, dim, page, type
    ([1], [1], 1, 1, 8, 1, B16),
    ([1], [777], 32, 8, 128, 16, B16),
    ([1], [5000], 16, 8, 128, 64, H16),
    ([1, 1, 1, 1], [1, 16, 17, 2000], 4, 4, 64, 16, B16),
    ([1, 1, 1], [0, 33, 0], 8, 2, 128, 16, B16),               # idle slots: rows that see nothing
    ([3, 1, 5], [2, 0, 5], 6, 2, 64, 7, H16),                  # fewer cached than new: the first tokens see nothing
    ([5, 4, 0, 3], [4000, 130, 50, 3], 16, 8, 128, 32, H16),   # drafts; a sequence without new tokens
    ([2, 7], [300, 129], 5, 1, 40, 33, B16),                   # odd sizes: dim inside a padded tile, one kv head for five
    ([4], [1000], 12, 4, 80, 16, H16),
    ([3], [260], 8, 4, 192, 5, B16),
    ([6, 1], [515, 64], 8, 2, 256, 64, H16),
    ([16], [16], 8, 8, 128, 16, B16),
    ([17, 40], [17, 300], 8, 2, 128, 16, B16),
    ([129], [1000], 4, 1, 128, 16, H16),
    ([333, 64], [333, 500], 6, 2, 64, 64, B16),
    ([65], [700], 3, 1, 96, 16, B16),
    ([130], [400], 2, 1, 256, 16, B16),
    ([700], [1900], 4, 2, 128, 128, B16),
]


@pytest.mark.parametrize("mask", [dict(), dict(window=100), dict(window=1), dict(causal=False)], ids=str)
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention(case, mask, kernel):
    new, ctx, H, KH, D, page, dtype = ATTN[case]
    s = Step(case, new, ctx, H, KH, D, page, dtype)
    qg.qgemv_attn(s.args(**mask))
    s.check(**mask)
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("case", ["few tiles", "more tiles than blocks", "idle", "long heads", "no context"])
def test_attention_many_sequences(case, kernel):
    """The division of the work over one wave of blocks: more sequences than a warp's 32, with and without rows, idle ones, more row
    tiles than blocks (a block then has the end of one, whole ones and the start of another)."""
    rng = np.random.default_rng(99)
    if case == "few tiles":
        new, ctx, H, KH, D = [1] * 40, rng.integers(1, 900, 40).tolist(), 4, 2, 64
    elif case == "more tiles than blocks":
        new, ctx, H, KH, D = rng.integers(0, 6, 90).tolist(), rng.integers(5, 700, 90).tolist(), 8, 8, 64
    elif case == "idle":
        new, ctx, H, KH, D = [1] * 70, [0] * 33 + [100] + [0] * 35 + [1], 8, 2, 64
    elif case == "long heads":
        new, ctx, H, KH, D = [3, 0, 50, 1], [2000, 10, 60, 1], 4, 2, 192
    else:
        new, ctx, H, KH, D = [150, 33, 2], [0, 20, 0], 4, 1, 64  # the 128-row kernel, row tiles that see nothing
    s = Step(40, new, ctx, H, KH, D, 16, B16)
    for mask in (dict(), dict(window=64)):
        qg.qgemv_attn(s.args(**mask))
        s.check(**mask)
        first = s.out.clone()
        qg.qgemv_attn(s.args(**mask))
        assert torch.equal(first, s.out)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("D,page,dtype", [(128, 64, B16), (64, 5, H16)])
def test_attention_blocks_that_take_many_parts(D, page, dtype, kernel):
    """More parts of row tiles than blocks: ones with one row and with two full tiles, without rows, without keys, with a few keys and with
    many, after one another in a block; three times with one scratch."""
    rng = np.random.default_rng(7)
    new = [int(x) for x in rng.choice([0, 1, 20, 100, 130, 300], 60)]
    ctx = [int(x) for x in rng.choice([0, 1, 60, 128, 400, 700, 1500], 60)]
    s = Step(61, new, ctx, 8, 4, D, page, dtype)
    for mask in (dict(), dict(causal=False), dict(window=150)):
        qg.qgemv_attn(s.args(**mask))
        s.check(**mask)
        first, scratch = s.out.clone(), s.scratch
        for _ in range(3):
            qg.qgemv_attn(s.args(scratch=scratch, **mask), qg.QGEMV_FLAG_PDL)
            assert torch.equal(first, s.out)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("mask", [dict(), dict(window=1100)], ids=str)
def test_attention_whole_row_tiles_before_cut_ones(mask):
    """160 row tiles: the 152 that fill a wave of blocks are left whole, the others' contexts are cut into parts."""
    s = Step(62, [1250], [2100], 32, 32, 64, 16, B16)
    qg.qgemv_route_reset()
    qg.qgemv_attn(s.args(**mask))
    assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_TILES] == 1
    s.check(**mask)
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("flags", [0, qg.QGEMV_FLAG_PDL])
def test_attention_takes_the_kernel_that_the_sizes_ask_for(flags):
    for new, ctx, route in ((1, 9000, qg.ROUTE_ATTN_ROWS), (8, 9000, qg.ROUTE_ATTN_ROWS), (40, 40, qg.ROUTE_ATTN_ROWS), (500, 9000, qg.ROUTE_ATTN_TILES)):
        s = Step(42, [new], [ctx], 8, 2, 128, 64, B16)
        a = s.args(lse=False)
        qg.qgemv_route_reset()
        qg.qgemv_attn(a, flags)
        assert qg.qgemv_route_counts()[route] == 1
        s.check()


@pytest.mark.parametrize("flags", [0, qg.QGEMV_FLAG_PDL])
def test_attention_of_a_chunk_in_a_graph(flags):
    s = Step(41, [500], [9000], 8, 2, 128, 64, B16)  # parts, joined by the second kernel
    a = s.args()
    qg.qgemv_route_reset()
    qg.qgemv_attn(a)
    assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_TILES] == 1
    s.check()
    want = (s.out.clone(), s.lse.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            qg.qgemv_attn(a, flags)
    s.out.fill_(0), s.lse.fill_(0)
    g.replay(), g.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1])


@pytest.mark.parametrize("new,ctx", [([1], [3000]), ([4, 200], [900, 700])])
def test_attention_orders_and_strides(new, ctx, kernel):
    s = Step(21, new, ctx, 8, 2, 128, 16, B16, order="head-token")
    wide = torch.full((s.q.shape[0], 3, 8, 128 + 8), float("nan"), dtype=B16, device="cuda")
    wide[:, 1, :, :128] = s.q
    target = torch.full((8, s.q.shape[0], 128), float("nan"), dtype=B16, device="cuda").transpose(0, 1)
    qg.qgemv_attn(s.args(q=wide[:, 1, :, :128], out=target))
    s.check()


@pytest.mark.parametrize("new,ctx,loose", [([1, 1], [900, 40], 40000), ([150, 20], [900, 40], 5000)])
def test_attention_loose_bounds_shared_scratch_and_repeats(new, ctx, loose, kernel):
    s = Step(22, new, ctx, 8, 2, 128, 16, B16)
    n = max(qg.qgemv_attn_scratch_bytes(2, sum(new), 8, 2, 128, a, b) for a, b in ((max(new), loose), (max(new) + 70, max(ctx))))
    scratch = torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")  # only the head has to start as zeros
    scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD] = 0
    outs = []
    for kw in (dict(max_kv=loose), dict(max_q=max(new) + 70), dict(max_kv=loose), dict()):
        qg.qgemv_attn(s.args(scratch=scratch, **kw))
        s.check()
        outs.append((s.out, s.lse))
        assert int(scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
    assert torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1])


@pytest.mark.parametrize("new", [1, 200])
def test_attention_large_scores_and_softmax_range(new, kernel):
    # scores of hundreds: the running maximum moves far, most probabilities vanish
    s = Step(23, [new], [1500], 8, 2, 128, 16, B16, scale=2.0)
    s.check_args = s.args()
    qg.qgemv_attn(s.check_args)
    s.check()
    # growing keys: the maximum rises all along the context
    s = Step(24, [new], [1500], 4, 1, 128, 16, B16)
    ramp = torch.linspace(0.01, 3.0, 1500, device="cuda")[:, None, None]
    s.k[0] = (s.q[-1, 0].float() * ramp * 0.2).to(B16).expand(1500, 1, 128).contiguous()
    t = torch.arange(1500, device="cuda")
    s.kc[s.table[0, t // 16].long(), t % 16] = s.k[0]
    qg.qgemv_attn(s.args())
    s.check()


def test_attention_bad_page_is_masked_and_reported(kernel):
    for new in (1, 150):
        s = Step(25, [new], [400], 4, 2, 128, 16, B16)
        s.table[0, 3], s.table[0, 7] = -1, 2 ** 30
        qg.qgemv_attn(s.args(causal=False))
        assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
        gone = np.r_[48:64, 112:128]
        keep = torch.from_numpy(np.setdiff1d(np.arange(400), gone)).cuda()
        s.k[0], s.v[0], s.ctx = s.k[0][keep], s.v[0][keep], [keep.numel()]
        s.check(causal=False)


def test_attention_tokens_beyond_the_bounds_are_left_alone(kernel):
    s = Step(26, [3, 2], [50, 60], 4, 2, 64, 16, B16)
    qg.qgemv_attn(s.args(max_q=2, causal=False))
    assert bool((s.out[2] == 7.0).all()) and bool((s.lse[2] == 7.0).all()) and not bool((s.out[[0, 1, 3, 4]] == 7.0).any())
    # a context longer than the table's row is read as far as the row goes
    s = Step(27, [1], [50], 4, 2, 64, 16, B16)
    s.table = s.table[:, :2].contiguous()
    qg.qgemv_attn(s.args(causal=False, max_kv=50))
    s.k[0], s.v[0], s.ctx = s.k[0][:32], s.v[0][:32], [32]
    s.check(causal=False)


@pytest.mark.parametrize("new", [1, 140])
def test_attention_offsets_past_32_bits(new, kernel):
    # pages 2^31 elements apart in one allocation: element offsets to 2^33
    free = torch.cuda.mem_get_info()[0]
    assert free > 40 << 30
    big = torch.empty((1 << 33) + (1 << 20), dtype=B16, device="cuda")
    KH, D, page, pages = 2, 128, 16, 5
    kc = big.as_strided((pages, page, KH, D), (1 << 31, KH * D, D, 1))
    vc = big.as_strided((pages, page, KH, D), (1 << 31, KH * D, D, 1), 1 << 19)
    s = Step(28, [new], [min(5 * page, 72)], 4, KH, D, page, B16)
    at = torch.tensor([4, 0, 3, 1, 2], device="cuda")
    for b in range(5):
        c = slice(b * page, min(72, (b + 1) * page))
        kc[at[b], :c.stop - c.start], vc[at[b], :c.stop - c.start] = s.k[0][c], s.v[0][c]
    s.kc, s.vc, s.table = kc, vc, at[None].to(torch.int32)
    qg.qgemv_attn(s.args())
    s.check()
    del big, kc, vc, s
    torch.cuda.empty_cache()


# --------------------------------------------------------------------------------------------------------- sampling

EPS = 1e-5


def check_sample(x, T, k, p, mp, u, token, prob):
    """Every row's token holds u within EPS in the 64-bit distribution of its kept tokens.  Tokens whose place at a filter's
    edge is closer than EPS may be kept or not: they widen the interval by their share."""
    for i in range(x.shape[0]):
        row, n = x[i], x.shape[1]
        if np.isnan(row).any() or (row == np.inf).any():
            assert token[i] == np.argmax(np.isnan(row) if np.isnan(row).any() else row == np.inf) and np.isnan(prob[i])
            continue
        if (row == -np.inf).all():
            assert token[i] == -1 and prob[i] == 0
            continue
        if T[i] <= 0 or k[i] == 1:
            assert token[i] == np.argmax(row) and prob[i] == 1
            continue
        e = np.exp((row - row.max()) / T[i])
        order = np.argsort(-row, kind="stable")
        if 0 < k[i] < n:
            order = order[:k[i]]
        keep = np.ones(order.size, bool)
        maybe = np.zeros(order.size, bool)
        if p[i] < 1:
            d = e[order] / e[order].sum()
            before = np.cumsum(d) - d
            keep &= before < p[i]
            maybe |= np.abs(before - p[i]) < EPS
        maybe |= np.abs(e[order] - mp[i]) < EPS * mp[i]
        keep &= e[order] >= mp[i]
        keep[0], maybe[0] = True, False
        sure, either = order[keep & ~maybe], order[maybe]
        kept = np.sort(np.concatenate([sure, either]))
        slack = EPS + e[either].sum() / e[sure].sum()
        assert token[i] in kept, i
        d = e[kept] / e[kept].sum()
        at = np.searchsorted(kept, token[i])
        c = np.cumsum(d)
        assert c[at] - d[at] - slack <= u[i] <= c[at] + slack, (i, c[at] - d[at], u[i], c[at])
        assert abs(prob[i] - d[at]) <= 10 * slack * d[at] + 1e-12


def run_sample(x, T=None, k=None, p=None, mp=None, u=None, flags=0, check=True):
    m = x.shape[0]
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, t)).cuda()  # noqa: E731
    token = torch.full((m,), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((m,), -9.0, device="cuda")
    qg.qgemv_sample(x, dev(T, np.float32), dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32), dev(u, np.float32), token,
                    prob, flags)
    token, prob = token.cpu().numpy(), prob.cpu().numpy().astype(np.float64)
    if check:
        full = lambda a, d, t: np.full(m, d) if a is None else np.asarray(a, t).astype(np.float64)  # noqa: E731
        kk = np.zeros(m, int) if k is None else np.asarray(k, int)
        check_sample(f64(x), full(T, 1.0, np.float32), kk, full(p, 1.0, np.float32), full(mp, 0.0, np.float32),
                     full(u, 0.0, np.float32), token, prob)
    return token, prob


@pytest.mark.parametrize("dtype", [torch.float32, B16, H16])
@pytest.mark.parametrize("m,n", [(1, 1), (5, 2), (7, 33), (64, 1000), (3, 32001), (9, 151936), (1, 1 << 20)])
def test_sampling(m, n, dtype):
    rng = np.random.default_rng(n)
    x = rnd(rng, (m, n), dtype, 3.0)
    u = rng.random(m, dtype=np.float32)
    run_sample(x, u=u)
    run_sample(x, T=rng.uniform(0.3, 2.0, m), u=u)
    run_sample(x, k=rng.integers(0, 60, m), u=u)
    run_sample(x, T=np.full(m, 0.7), p=rng.uniform(0.2, 0.999, m), u=u)
    run_sample(x, mp=rng.uniform(0.0, 0.3, m), u=u)
    run_sample(x, T=rng.uniform(0.3, 2.0, m), k=rng.integers(1, 2 * n, m), p=rng.uniform(0.5, 1.1, m), mp=rng.uniform(0.0, 0.01, m), u=u)


@pytest.mark.parametrize("dtype", [B16, torch.float32])
def test_sampling_many_rows(dtype):
    # more rows than fill the GPU with short slices
    rng = np.random.default_rng(12)
    m, n = 90, 151936
    x = rnd(rng, (m, n), dtype, 2.0)
    x[::7, rng.integers(0, n, 100000)] = -float("inf")
    u = rng.random(m, dtype=np.float32)
    a = run_sample(x, T=rng.uniform(0.5, 1.5, m), k=rng.choice([0, 1, 40, 512, 513, 3000], m), p=rng.choice([0.5, 0.95, 1.0], m), u=u)
    b = run_sample(x, T=rng.uniform(0.5, 1.5, m), p=np.full(m, 0.9), mp=rng.choice([0.0, 0.01], m), u=u)
    assert a[0].shape == b[0].shape == (m,)


@pytest.mark.parametrize("dtype", [torch.float32, B16, H16])
def test_sampling_special_rows(dtype):
    rng = np.random.default_rng(3)
    n = 5003
    x = rnd(rng, (12, n), dtype, 2.0)
    inf = float("inf")
    x[0] = -inf
    x[1, 4000] = float("nan")
    x[1, 17] = inf
    x[2, 300] = inf
    x[2, 4999] = inf
    x[3] = -inf
    x[3, 77] = -3.0
    x[4, ::2] = -inf
    x[5] = 0.25          # one tie of the whole row
    x[6] = -0.0
    x[6, ::3] = 0.0      # both zeros are one value
    x[7, 100:4000] = x[7].max()
    x[8, 4999] = 3e38 if dtype is not H16 else 6e4
    x[9] *= 1e-4
    x[10, 5] = float("nan")
    x[10, 4] = float("nan")
    x[11] = -6e4
    u = rng.random(12, dtype=np.float32)
    for kw in (dict(), dict(k=np.full(12, 7)), dict(p=np.full(12, 0.5)), dict(mp=np.full(12, 0.1)), dict(T=np.zeros(12)),
               dict(k=np.full(12, 1000), p=np.full(12, 0.9), mp=np.full(12, 0.05)), dict(k=np.ones(12)),
               dict(T=np.full(12, 1e-3)), dict(p=np.full(12, 0.999))):
        run_sample(x, u=u, **kw)
    for edge in (0.0, np.float32(1 - 2.0 ** -24)):
        run_sample(x, u=np.full(12, edge), k=np.full(12, 50))
    # settings that leave rank 0 alone
    for kw in (dict(p=np.zeros(12)), dict(p=np.full(12, -1.0)), dict(mp=np.full(12, 1.5)), dict(T=np.full(12, -1.0)),
               dict(p=np.full(12, np.nan)), dict(T=np.full(12, np.nan)), dict(T=np.full(12, 1e-40))):
        token, prob = run_sample(x, u=u, check=False, **kw)
        ok = [3, 4, 5, 6, 7, 8, 9, 11]
        assert np.array_equal(token[ok], f64(x).argmax(1)[ok]) and np.all(prob[ok] == 1)
    token, _ = run_sample(x, u=u, check=False, T=np.full(12, np.inf))  # flat over what is not masked
    assert all(np.isfinite(f64(x)[i, token[i]]) for i in (3, 4, 5, 6, 7, 8, 9, 11))


def test_sampling_follows_the_distribution():
    rng = np.random.default_rng(8)
    n, m = 200, 20000
    row = rng.standard_normal(n).astype(np.float32)
    x = torch.from_numpy(np.broadcast_to(row, (m, n)).copy()).cuda()
    u = (np.arange(m) + 0.5) / m
    token, _ = run_sample(x, k=np.full(m, 40), p=np.full(m, 0.9), u=u, check=False)
    e = np.exp(row.astype(np.float64) - row.max())
    order = np.argsort(-row, kind="stable")[:40]
    d = e[order] / e[order].sum()
    order = order[np.cumsum(d) - d < np.float32(0.9)]
    want = np.zeros(n)
    want[order] = e[order] / e[order].sum()
    # evenly spaced u: the share of each token is off by at most two grid steps
    assert np.all(np.abs(np.bincount(token, minlength=n) / m - want) <= 2.0 / m + 1e-6)


def test_sampling_strided_rows_and_missing_prob():
    rng = np.random.default_rng(9)
    wide = rnd(rng, (6, 1021), torch.float32, 2.0)  # rows that start at no 16-byte boundary
    x = wide[:, :1013]
    u = rng.random(6, dtype=np.float32)
    a = run_sample(x, k=np.full(6, 50), p=np.full(6, 0.8), u=u)
    b = run_sample(x.contiguous(), k=np.full(6, 50), p=np.full(6, 0.8), u=u)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    token = torch.empty(6, dtype=torch.int32, device="cuda")
    qg.qgemv_sample(x, None, torch.full((6,), 50, dtype=torch.int32, device="cuda"), torch.full((6,), 0.8, device="cuda"), None,
                    torch.from_numpy(u).cuda(), token)
    assert np.array_equal(token.cpu().numpy(), a[0])


# ------------------------------------------------------------------------------- streams, graphs, dependent launch

def test_step_in_a_graph_with_dependent_launch():
    """rope + append, attention over the cache just written, and sampling from the result's first values, captured on a side
    stream with programmatic dependent launch and replayed: the same bits as plain calls."""
    rng = np.random.default_rng(11)
    H, KH, D, page = 8, 2, 64, 16
    s = Step(31, [1, 1, 2], [50, 333, 20], H, KH, D, page, B16)
    T = 4
    qkv = rnd(rng, (T, (H + 2 * KH) * D), torch.float32)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([H * D, KH * D, KH * D], 1))
    pos = torch.tensor([49, 332, 18, 19], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 1, 2, 2], device="cuda")
    slots = s.table[seq, pos.long() // page].long() * page + pos.long() % page
    freqs = qg.qgemv_rope_freqs(D)[0].cuda()
    qo = torch.empty(T, H, D, dtype=B16, device="cuda")
    rope = qg.rope_args(q, k, v, pos, freqs, qo, cache=qg.kv_cache(s.kc, s.vc), slots=slots)
    args = s.args(q=qo)
    u = torch.rand(T, device="cuda")
    token = torch.empty(T, dtype=torch.int32, device="cuda")
    topk = torch.full((T,), 20, dtype=torch.int32, device="cuda")

    def step(flags, stream=None):
        qg.qgemv_rope(rope, flags, stream)
        qg.qgemv_attn(args, flags, stream)
        qg.qgemv_sample(s.out.view(T, -1), None, topk, None, None, u, token, None, flags, stream)

    step(0)
    torch.cuda.synchronize()
    want = (s.out.clone(), s.lse.clone(), token.clone(), s.kc.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(qg.QGEMV_FLAG_PDL)
    for t in (s.out, s.lse, token):
        t.fill_(0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    got = (s.out, s.lse, token, s.kc)
    assert all(torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(got, want))
