"""Attention over a packed cache on the GPU, against its formula in 64 bits (numpy) on the exact values d c + m.

Tolerances, from the arithmetic (p the probabilities, k = d c + m in blocks of 32):
 - a score is an fp32 sum of products that are exact in fp32 (codes are whole numbers, q is f16 times a power of two, or off by 2^-30 of its
   row's largest element), scaled by steps and with the bases' product (block sums of q in 22 bits): off by at most
   off = 2^-19 scale max_t sum |q| (d c + |m|);
 - p is rounded to f16 (2^-11 of it), and its product with a step once more; both lose bits below 2^-24 of what stands for 2^10 p, that is 2^-34
   of the largest p, times the largest code or |m|, a key, and more where a step is above 2, by that half step;
 - so with A = sum p (d c + |m|): out is off by u |ref| + (2^-10 + 4 off + 2^-18) A + 2^-34 sum_t (L + |m|) max(1, d/2), lse by
   off + 2^-20 max(1, |lse|).
The 128-row kernel reads an f16 copy: with f16 queries its results are those of the same call on such a copy made by qgemv_cache_read, bit for bit.
With bf16 ones the formula holds with keys and values rounded to f16 (2^-11 of each: off grows by 2^-11 scale sum |q||k|, the output by 2^-11 of sum
p |v|), p to f16 once (those below 2^-21 of the largest lose bits: 2^-32 |v| a key).
"""
import math

import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from . import packedref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_step_gpu import TINY, U, f64, rnd  # noqa: E402

B16, H16 = torch.bfloat16, torch.float16
BITS = {"Q4": 4, "Q8": 8}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.build()
    qg.lib()
    qg.qgemv_device_error(reset=True)
    yield
    assert qg.qgemv_device_error() == 0


@pytest.fixture
def rows_kernel():
    qg.qgemv_tune_attn(1)
    yield
    qg.qgemv_tune_attn(0)


class Packed:
    """A batch over a packed cache: sequences with `new[b]` new tokens over contexts of `ctx[b]` tokens in shuffled pages; whatever no
    context holds is 0xFF: steps and bases that are no numbers."""

    def __init__(self, seed, kind, new, ctx, H, KH, D, page, dtype, order="token-head", scale=None, kscale=1.0, vscale=1.0):
        rng = np.random.default_rng(seed)
        self.kind, self.bits, self.new, self.ctx, self.H, self.KH, self.D, self.page, self.dtype = kind, BITS[kind], new, ctx, H, KH, D, page, dtype
        need = [-(-c // page) for c in ctx]
        total = sum(need) + 2
        row = ref.row_bytes(self.bits, D)
        kc, vc = (np.full((total, page, KH, row), 0xFF, np.uint8) for _ in range(2))
        perm = rng.permutation(total).astype(np.int32)
        table = np.full((len(ctx), max([1] + need)), 2 ** 30, np.int32)  # entries that no context reaches
        at = 0
        self.k, self.v = [], []  # rows of bytes
        for b, c in enumerate(ctx):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            t = np.arange(c)
            for cache, held, s in ((kc, self.k, kscale), (vc, self.v, vscale)):
                x = rng.standard_normal((c, KH, D)).astype(np.float32)
                x += 4.0 * (rng.random((1, KH, D)) < 0.05)
                rows = ref.to_bytes(*ref.pack(x * np.float32(s), self.bits), self.bits)
                n = D * self.bits // 8 + D // 32 * 4
                rows[..., n:] = 0xFF
                held.append(rows)
                cache[table[b, t // page], t % page] = rows
        self.kc, self.vc = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
        if order != "token-head":
            self.kc, self.vc = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (self.kc, self.vc))
        self.table = torch.from_numpy(table).cuda()
        self.q = rnd(rng, (sum(new), H, D), dtype, 1.5)
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.scale = 1.0 / math.sqrt(D) if scale is None else scale

    def put(self, b, k=None, v=None):
        """Other rows of bytes [c, KH, row] for sequence b."""
        t = torch.arange(self.ctx[b], device="cuda")
        where = (self.table[b, t // self.page].long(), t % self.page)
        for rows, cache, held in ((k, self.kc, self.k), (v, self.vc, self.v)):
            if rows is not None:
                held[b] = rows
                cache[where] = torch.from_numpy(rows).cuda()

    def args(self, causal=True, window=0, lse=True, scratch=None, q=None, out=None, max_q=None, max_kv=None):
        max_q, max_kv = max(self.new) if max_q is None else max_q, max(self.ctx) if max_kv is None else max_kv
        q = self.q if q is None else q
        self.out = torch.full_like(q.contiguous(), 7.0) if out is None else out
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if lse else None
        cache = qg.packed_cache(self.kind, self.kc, self.vc, self.D)
        n = qg.qgemv_attn_scratch_bytes(len(self.new), q.shape[0], self.H, self.KH, self.D, max_q, max_kv, cache=cache)
        self.scratch = torch.zeros(n, dtype=torch.uint8, device="cuda") if scratch is None else scratch
        return qg.attn_args(q, cache, self.table, self.starts, self.lens, self.out, self.scratch, max_q, max_kv, self.scale, causal, window,
                            self.lse)

    def check(self, causal=True, window=0, copy=False):
        out, lse, first, u = f64(self.out), None if self.lse is None else f64(self.lse), 0, U[self.dtype]
        top_code = (1 << self.bits) - 1
        for b, (n, c) in enumerate(zip(self.new, self.ctx)):
            q = f64(self.q[first:first + n])
            k, v = ref.values(self.k[b], self.bits, self.D), ref.values(self.v[b], self.bits, self.D)
            sizes = []
            for rows in (self.k[b], self.v[b]):  # d c + |m|
                code, d, m = ref.parts(rows, self.bits, self.D)
                wide = lambda x: np.repeat(x.astype(np.float64), 32, -1)  # noqa: E731
                sizes.append((code * wide(d) + np.abs(wide(m)), d.astype(np.float64), np.abs(m.astype(np.float64))))
            (kmag, _, _), (vmag, vd, vm) = sizes
            pos = c - n + np.arange(n)
            t = np.arange(c)
            sees = np.ones((n, c), bool)
            if causal or window:
                sees &= t[None] <= pos[:, None]
            if window:
                sees &= t[None] > pos[:, None] - window
            group = self.H // self.KH
            for h in range(self.H):
                kv, qh = h // group, q[:, h]
                s = np.where(sees, self.scale * (qh @ k[:, kv].T), -np.inf)
                top = s.max(1, initial=-np.inf, keepdims=True)
                top = np.where(np.isinf(top), 0.0, top)
                p = np.exp(s - top)
                l = p.sum(1, keepdims=True)
                p = p / np.where(l == 0, 1, l)
                want, A = p @ v[:, kv], p @ vmag[:, kv]
                off = 2.0 ** -19 * self.scale * (np.abs(qh) @ kmag[:, kv].T).max(1, initial=0.0)[:, None]
                floor = 2.0 ** -34 * ((top_code + vm[:, kv].max(-1)) * np.maximum(1, vd[:, kv].max(-1) / 2)).sum() if c else 0.0
                if copy:
                    off = off + 2.0 ** -11 * self.scale * (np.abs(qh) @ np.abs(k[:, kv]).T).max(1, initial=0.0)[:, None]
                    A, floor = p @ np.abs(v[:, kv]), 2.0 ** -32 * np.abs(v[:, kv]).max(-1).sum()
                tol = u * np.abs(want) + (2.0 ** -10 + 4 * off + 2.0 ** -18) * A + floor + TINY[self.dtype]
                err = np.abs(out[first:first + n, h] - want)
                assert np.all(err <= tol), (b, h, float((err - tol).max()), np.unravel_index((err - tol).argmax(), err.shape))
                if lse is not None:
                    with np.errstate(divide="ignore"):
                        full = np.where(l[:, 0] > 0, top[:, 0] + np.log(l[:, 0]), -np.inf)
                    got = lse[first:first + n, h]
                    empty = np.isinf(full)
                    assert np.array_equal(np.isneginf(got), empty)
                    got, full, o = got[~empty], full[~empty], off[~empty, 0]
                    assert np.all(np.abs(got - full) <= o + 2.0 ** -20 * np.maximum(1, np.abs(full)))
            first += n


CASES = [
    # new tokens, contexts, heads, kv heads, dim, page, type
    ([1], [1], 1, 1, 32, 1, B16),
    ([1], [777], 32, 8, 128, 16, B16),
    ([1], [5000], 16, 8, 128, 64, H16),
    ([1, 1, 1, 1], [1, 16, 17, 2000], 4, 4, 64, 16, B16),
    ([1, 1, 1], [0, 33, 0], 8, 2, 128, 16, B16),               # idle slots: rows that see nothing
    ([3, 1, 5], [2, 0, 5], 6, 2, 64, 7, H16),                  # fewer cached than new: the first tokens see nothing
    ([5, 4, 0, 3], [4000, 130, 50, 3], 16, 8, 128, 32, H16),   # drafts; a sequence without new tokens
    ([2, 7], [300, 129], 5, 1, 96, 33, B16),                   # odd sizes: dim inside a padded tile, one kv head for five
    ([4], [1000], 12, 4, 160, 16, H16),
    ([3], [260], 8, 4, 192, 5, B16),
    ([6, 1], [515, 64], 8, 2, 256, 64, H16),
    ([2], [700], 4, 2, 224, 24, B16),                          # pages of 24: copies of 8 tokens
    ([16], [16], 8, 8, 128, 8, B16),
    ([17, 40], [17, 300], 8, 2, 128, 16, B16),
    ([1], [3001], 7, 1, 32, 3, H16),
    ([9], [600], 1, 1, 64, 128, B16),
]
MASKS = [dict(), dict(window=100), dict(window=1), dict(causal=False)]


@pytest.mark.parametrize("mask", MASKS, ids=str)
@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(case, kind, mask, rows_kernel):
    new, ctx, H, KH, D, page, dtype = CASES[case]
    s = Packed(case, kind, new, ctx, H, KH, D, page, dtype)
    qg.qgemv_route_reset()
    qg.qgemv_attn(s.args(**mask))
    assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_PACKED] == 1
    s.check(**mask)
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("case", ["few tiles", "more tiles than blocks", "idle", "long heads", "no context"])
def test_attention_many_sequences(case, kind, rows_kernel):
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
        new, ctx, H, KH, D = [150, 33, 2], [0, 20, 0], 4, 1, 64
    s = Packed(40, kind, new, ctx, H, KH, D, 16, B16)
    for mask in (dict(), dict(window=64)):
        qg.qgemv_attn(s.args(**mask))
        s.check(**mask)
        first = s.out.clone()
        qg.qgemv_attn(s.args(**mask))
        assert torch.equal(first, s.out)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


MANY = [([300], 64, {}), ([150, 20], 16, dict(window=70)), ([129, 0, 64], 5, {}), ([40], 48, dict(causal=False)), ([260], 128, {}), ([7, 3], 16, {})]


@pytest.fixture
def copying():
    qg.qgemv_tune_attn(2)
    yield
    qg.qgemv_tune_attn(0)


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("new,page,mask", MANY)
def test_many_rows_equal_the_same_call_on_a_copy(new, page, mask, kind, copying):
    ctx = [900, 260, 333][:len(new)]
    s = Packed(5, kind, new, ctx, 8, 2, 128, page, H16)
    a = s.args(**mask)
    qg.qgemv_route_reset()
    qg.qgemv_attn(a)
    assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_TILES] == 1
    packed = s.out.clone(), s.lse.clone()
    # the contexts one after another in a 16-bit cache of the same pages
    starts = np.concatenate([[0], np.cumsum(ctx)]).astype(np.int32)
    k, v = (torch.zeros(sum(ctx), 2, 128, dtype=H16, device="cuda") for _ in range(2))
    qg.qgemv_cache_read(qg.cache_read_args(qg.packed_cache(kind, s.kc, s.vc, 128), s.table, torch.from_numpy(starts).cuda(), k, v))
    kc, vc = (torch.zeros(*s.kc.shape[:3], 128, dtype=H16, device="cuda") for _ in range(2))
    for b, c in enumerate(ctx):
        t = torch.arange(c, device="cuda")
        where = s.table[b, t // page].long(), t % page
        kc[where], vc[where] = k[starts[b]:starts[b + 1]], v[starts[b]:starts[b + 1]]
    out, lse = torch.full_like(s.out, 7.0), torch.full_like(s.lse, 7.0)
    qg.qgemv_attn(qg.attn_args(s.q, qg.kv_cache(kc, vc), s.table, s.starts, s.lens, out, s.scratch, max(new), max(ctx), s.scale, lse=lse, **mask))
    assert torch.equal(out, packed[0]) and torch.equal(lse, packed[1])
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("new,page,mask", MANY)
def test_many_rows(new, page, mask, D, kind, copying):
    ctx = [900, 260, 333][:len(new)]
    for qscale in (1.0, 1e-6, 3e4):  # (bf16 queries of any size: rows scaled by powers of two)
        s = Packed(6, kind, new, ctx, 6, 2, D, page, B16, scale=D ** -0.5 / qscale)
        s.q.mul_(qscale)
        a = s.args(**mask)
        qg.qgemv_attn(a)
        s.check(copy=True, **mask)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
        first = s.out.clone()
        qg.qgemv_attn(a, qg.QGEMV_FLAG_PDL)
        assert torch.equal(first, s.out)


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("new", [1, 6])
def test_orders_strides_loose_bounds_and_repeats(kind, new):
    s = Packed(21, kind, [new, new], [3000, 41], 8, 2, 128, 16, B16, order="head-token")
    wide = torch.full((s.q.shape[0], 3, 8, 128 + 8), float("nan"), dtype=B16, device="cuda")
    wide[:, 1, :, :128] = s.q
    target = torch.full((8, s.q.shape[0], 128), float("nan"), dtype=B16, device="cuda").transpose(0, 1)
    qg.qgemv_attn(s.args(q=wide[:, 1, :, :128], out=target))
    s.check()
    s.args(max_kv=60000, max_q=new + 70)
    scratch = torch.full_like(s.scratch, 0x5A)  # only the head has to start as zeros
    scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD] = 0
    outs = []
    for kw in (dict(max_kv=40000), dict(max_q=new + 1), dict(max_kv=40000), dict()):
        qg.qgemv_attn(s.args(scratch=scratch, **kw))
        s.check()
        outs.append((s.out, s.lse))
        assert int(scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
    assert torch.equal(outs[0][0], outs[2][0]) and torch.equal(outs[0][1], outs[2][1])


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("new", [1, 3])
def test_large_scores_and_a_rising_maximum(kind, new, rows_kernel):
    s = Packed(23, kind, [new], [1500], 8, 2, 128, 16, B16, scale=2.0)
    qg.qgemv_attn(s.args())
    s.check()
    s = Packed(24, kind, [new], [1500], 4, 1, 128, 16, B16)
    ramp = np.linspace(0.01, 3.0, 1500)[:, None, None]
    x = (f64(s.q[-1, 0]) * ramp * 0.2).astype(np.float32)
    s.put(0, k=ref.to_bytes(*ref.pack(x, s.bits), s.bits))
    qg.qgemv_attn(s.args())
    s.check()


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("vscale", [1e-3, 30.0, 3000.0, 15000.0])
def test_values_of_any_size(kind, vscale, rows_kernel):
    # steps below fp16's normal range and above 2, the largest fp16 in reach; keys with a far offset, queries of any size
    for qscale in (1e-6, 1.0, 300.0):
        s = Packed(31, kind, [2, 1], [700, 90], 8, 2, 64, 16, B16, vscale=vscale, scale=0.125 / qscale)
        s.q.mul_(qscale)
        x = np.random.default_rng(3).standard_normal((700, 2, 64)).astype(np.float32) * 0.5 + 40.0
        s.put(0, k=ref.to_bytes(*ref.pack(x, s.bits), s.bits))
        # growing values: the steps rise along the context
        y = np.random.default_rng(4).standard_normal((700, 2, 64)).astype(np.float32) * np.geomspace(1e-3, 4, 700)[:, None, None] * vscale
        s.put(0, v=ref.to_bytes(*ref.pack(y.astype(np.float32), s.bits), s.bits))
        qg.qgemv_attn(s.args())
        s.check()


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_queries_that_are_no_numbers_and_zeros(kind, rows_kernel):
    s = Packed(32, kind, [2, 1], [300, 20], 8, 2, 128, 16, B16)
    s.q[1, 3, 77] = float("nan")
    s.q[2, 5] = 0
    a = s.args()
    qg.qgemv_attn(a)
    assert bool(s.out[1, 3].isnan().all()) and bool(s.lse[1, 3].isnan())
    assert int(s.out.isnan().any(-1).sum()) == 1 and int(s.lse.isnan().sum()) == 1
    s.q[1, 3], s.out[1, 3], s.lse[1, 3] = 0, 0, 0
    keep = s.out.clone(), s.lse.clone()
    qg.qgemv_attn(s.args())
    keep[0][1, 3], keep[1][1, 3] = s.out[1, 3], s.lse[1, 3]
    assert torch.equal(keep[0], s.out) and torch.equal(keep[1], s.lse)
    s.check()


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("new", [1, 150])
def test_bad_page_is_masked_and_reported(new, page, kind):
    for D in (128, 64):
        s = Packed(25, kind, [new], [400], 4, 2, D, page, B16)
        s.table[0, 3], s.table[0, 7] = -1, 2 ** 30
        qg.qgemv_attn(s.args(causal=False))
        assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
        gone = np.r_[3 * page:4 * page, 7 * page:8 * page]
        keep = np.setdiff1d(np.arange(400), gone)
        if new == 1:
            s.k[0], s.v[0], s.ctx = s.k[0][keep], s.v[0][keep], [keep.size]
            s.check(causal=False)
        else:  # by the copy: its rounding is the 16-bit cache's, so the tokens left are only compared with one another
            out = s.out.clone()
            qg.qgemv_attn(s.args(causal=False))
            assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
            assert torch.equal(out, s.out) and bool(out.isfinite().all())


def test_tokens_beyond_the_bounds_are_left_alone(rows_kernel):
    s = Packed(26, "Q4", [3, 2], [50, 60], 4, 2, 64, 16, B16)
    qg.qgemv_attn(s.args(max_q=2, causal=False))
    assert bool((s.out[2] == 7.0).all()) and bool((s.lse[2] == 7.0).all()) and not bool((s.out[[0, 1, 3, 4]] == 7.0).any())
    s = Packed(27, "Q4", [1], [50], 4, 2, 64, 16, B16)
    s.table = s.table[:, :2].contiguous()
    qg.qgemv_attn(s.args(causal=False, max_kv=50))
    s.k[0], s.v[0], s.ctx = s.k[0][:32], s.v[0][:32], [32]
    s.check(causal=False)


@pytest.mark.parametrize("page", [16, 7])
def test_offsets_past_32_bits(page):
    # pages 2^32 bytes apart in one allocation
    assert torch.cuda.mem_get_info()[0] > 60 << 30
    big = torch.empty((5 << 32) + (1 << 21), dtype=torch.uint8, device="cuda")
    KH, D, row = 2, 128, 80
    kc, vc = (big.as_strided((5, page, KH, row), (1 << 32, KH * row, row, 1), at) for at in (0, 1 << 20))
    s = Packed(28, "Q4", [1], [5 * page - 3], 4, KH, D, page, B16)
    at = torch.tensor([4, 0, 3, 1, 2], device="cuda")
    for b in range(5):
        c = slice(b * page, min(s.ctx[0], (b + 1) * page))
        kc[at[b], :c.stop - c.start] = torch.from_numpy(s.k[0][c]).cuda()
        vc[at[b], :c.stop - c.start] = torch.from_numpy(s.v[0][c]).cuda()
    s.kc, s.vc, s.table = kc, vc, at[None].to(torch.int32)
    qg.qgemv_attn(s.args())
    s.check()
    out = torch.empty(s.ctx[0], KH, D, device="cuda")
    qg.qgemv_cache_read(qg.cache_read_args(qg.packed_cache("Q4", kc, vc, D), s.table, torch.tensor([0, s.ctx[0]], dtype=torch.int32, device="cuda"),
                                           out))
    assert np.array_equal(out.cpu().numpy(), ref.values(s.k[0], 4, D).astype(np.float32))
    x = torch.randn(5, KH, D, device="cuda")
    qg.qgemv_cache_write(qg.cache_write_args(x, x, qg.packed_cache("Q4", kc, vc, D), torch.arange(5, device="cuda") * page))
    want = ref.to_bytes(*ref.pack(x.cpu().numpy(), 4), 4)
    assert np.array_equal(kc[:, 0].cpu().numpy(), want) and np.array_equal(vc[:, 0].cpu().numpy(), want)
    del big, kc, vc, s
    torch.cuda.empty_cache()
