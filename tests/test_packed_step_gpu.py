"""The packed cache's operators together, as a serving step calls them: in graphs, on other streams, with dependent launches, after one another on
one scratch, with padding; and the step of rotary positions, cache and attention against its 64-bit form.

Attention's tolerances are those of test_packed_attn_gpu.py."""
import math

import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from . import packedref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import B16, BITS, H16, Packed  # noqa: E402
from .test_step_gpu import f64  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qg.build()
    qg.lib()
    qg.qgemv_device_error(reset=True)
    yield
    assert qg.qgemv_device_error() == 0


def graph_of(f):
    f()  # every kernel has been launched once before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f()
    return g


class Decoder:
    """Sequences whose tokens go through rotary positions into a packed cache and attend over it; every address is fixed."""

    def __init__(self, kind, seqs, longest, H, KH, D, page, dtype, layout="token"):
        self.kind, self.seqs, self.H, self.KH, self.D, self.page = kind, seqs, H, KH, D, page
        pages = -(-longest // page)
        row = qg.qgemv_cache_row_bytes(kind, D)
        shape = (seqs * pages, page, KH, row) if layout == "token" else (seqs * pages, KH, page, row)
        self.kc, self.vc = (torch.full(shape, 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))  # (0xFF: scales that are no numbers)
        if layout != "token":
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.cache = qg.packed_cache(kind, self.kc, self.vc, D)
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        self.table = torch.randperm(seqs * pages, generator=g, device="cuda").to(torch.int32).view(seqs, pages)
        self.freqs = qg.qgemv_rope_freqs(D, 1e4)[0].cuda()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.x = torch.empty(seqs, (H + 2 * KH) * D, device="cuda")  # a merged GEMV's fp32 rows
        q, k, v = (t.unflatten(1, (-1, D)) for t in self.x.split([H * D, KH * D, KH * D], 1))
        self.pos = torch.empty(seqs, dtype=torch.int32, device="cuda")
        self.slots = torch.empty(seqs, dtype=torch.int64, device="cuda")
        self.q = torch.empty(seqs, H, D, dtype=dtype, device="cuda")
        self.out = torch.empty_like(self.q)
        self.rope = qg.rope_args(q, k, v, self.pos, self.freqs, self.q, cache=self.cache, slots=self.slots)
        n = qg.qgemv_attn_scratch_bytes(seqs, seqs, H, KH, D, 1, longest, cache=self.cache)
        self.scratch = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self.start = torch.arange(seqs + 1, dtype=torch.int32, device="cuda")
        self.attn = qg.attn_args(self.q, self.cache, self.table, self.start, self.lens, self.out, self.scratch, 1, longest, D ** -0.5)

    def step(self, flags=0):
        at = self.lens.long()
        self.pos.copy_(at)
        self.slots.copy_(self.table.gather(1, (at // self.page)[:, None])[:, 0].long() * self.page + at % self.page)
        self.lens += 1
        qg.qgemv_rope(self.rope, flags)
        qg.qgemv_attn(self.attn, flags)


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("kind,dtype", [("Q4", B16), ("Q8", H16)])
def test_tokens_through_rotary_positions_cache_and_attention(kind, dtype, layout):
    seqs, steps, H, KH, D = 3, 40, 8, 2, 64
    runs = []
    rng = np.random.default_rng(11)
    xs = torch.from_numpy(rng.standard_normal((steps, seqs, (H + 2 * KH) * D)).astype(np.float32)).cuda()
    for mode in ("calls", "dependent", "graph"):
        d = Decoder(kind, seqs, steps + 8, H, KH, D, 16, dtype, layout)
        flags = 0 if mode == "calls" else qg.QGEMV_FLAG_PDL
        outs, qs = [], []
        d.x.copy_(xs[0])
        if mode == "graph":
            g = graph_of(lambda: d.step(flags))
            d.lens.zero_()
        for i in range(steps):
            d.x.copy_(xs[i])
            g.replay() if mode == "graph" else d.step(flags)
            outs.append(d.out.clone()), qs.append(d.q.clone())
        runs.append((torch.stack(outs), torch.stack(qs), d))
    for out, q, d in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(q, runs[0][1])
    # attention over what the cache holds, in 64 bits
    outs, qs, d = runs[0]
    bits = BITS[kind]
    s = Packed.__new__(Packed)
    s.kind, s.bits, s.H, s.KH, s.D, s.page, s.dtype, s.scale, s.lse = kind, bits, H, KH, D, 16, dtype, D ** -0.5, None
    s.new = [1] * seqs
    t = torch.arange(steps, device="cuda")
    rows = [[c[d.table[b, t // 16].long(), t % 16].cpu().numpy() for b in range(seqs)] for c in (d.kc, d.vc)]
    for i in (0, 1, 15, 16, 39):
        s.ctx = [i + 1] * seqs
        s.k, s.v = ([r[:i + 1] for r in x] for x in rows)
        s.q, s.out = qs[i], outs[i]
        s.check()
    # and the values that were put there: the definition's bytes of the fp32 rows
    want = ref.to_bytes(*ref.pack(xs[:, 0, (H + KH) * D:].cpu().numpy().reshape(steps, KH, D), bits), bits)
    n = D * bits // 8 + D // 32 * 4
    assert np.array_equal(rows[1][0][..., :n], want[..., :n])


def test_write_read_and_attention_in_one_graph_on_another_stream():
    s = Packed(50, "Q4", [1, 3], [500, 90], 8, 2, 128, 16, B16)
    a = s.args()
    x = torch.randn(4, 2, 128, device="cuda")
    at = [499, 87, 88, 89]
    seq = [0, 1, 1, 1]
    slots = torch.tensor([int(s.table[b, p // 16]) * 16 + p % 16 for b, p in zip(seq, at)], device="cuda")
    cache = qg.packed_cache("Q4", s.kc, s.vc, 128)
    w = qg.cache_write_args(x, x, cache, slots)
    ko = torch.empty(590, 2, 128, dtype=H16, device="cuda")
    r = qg.cache_read_args(cache, s.table, torch.tensor([0, 500, 590], dtype=torch.int32, device="cuda"), ko)

    def step(flags=0, stream=None):
        qg.qgemv_cache_write(w, flags, stream), qg.qgemv_cache_read(r, flags, stream), qg.qgemv_attn(a, flags, stream)

    step()
    new = ref.to_bytes(*ref.pack(x.cpu().numpy(), 4), 4)
    s.k[0][499], s.v[0][499], s.k[1][87:], s.v[1][87:] = new[0], new[0], new[1:], new[1:]
    s.check()
    want = torch.from_numpy(np.concatenate([ref.values(k, 4, 128) for k in s.k]).astype(np.float32)).to(H16)
    assert torch.equal(ko.cpu(), want)
    out, lse = s.out.clone(), s.lse.clone()
    for flags in (0, qg.QGEMV_FLAG_PDL):
        g = graph_of(lambda: step(flags))
        for b, p in zip(seq, at):
            s.kc[int(s.table[b, p // 16]), p % 16] = 0xFF
        s.out.zero_(), s.lse.zero_(), ko.zero_()
        g.replay(), g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, out) and torch.equal(s.lse, lse) and torch.equal(ko.cpu(), want)
    side = torch.cuda.Stream()
    s.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(0, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s.out, out)


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_one_scratch_for_calls_of_all_kinds(kind):
    """Decode, a chunk by the copy, a 16-bit cache: after one another on the scratch of the largest."""
    few, many = Packed(51, kind, [1, 2], [2000, 30], 8, 2, 128, 16, B16), Packed(52, kind, [200], [700], 8, 2, 128, 16, B16)
    a = few.args()
    b = many.args()
    n = max(few.scratch.numel(), many.scratch.numel())
    scratch = torch.full((n,), 0x77, dtype=torch.uint8, device="cuda")
    scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD] = 0
    for _ in range(2):
        qg.qgemv_attn(few.args(scratch=scratch))
        few.check()
        qg.qgemv_tune_attn(2)
        qg.qgemv_attn(many.args(scratch=scratch))
        qg.qgemv_tune_attn(0)
        many.check(copy=True)
        assert int(scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
    del a, b


@pytest.mark.parametrize("heads,seqs,longest", [(1, 30, 900), (3, 30, 900), (2, 130, 1500), (4, 80, 2500), (12, 24, 2600)])
@pytest.mark.parametrize("kind,order,D,page", [("Q4", "token-head", 128, 16), ("Q4", "head-token", 128, 16), ("Q8", "head-token", 64, 16),
                                               ("Q8", "token-head", 128, 24)])
def test_heads_side_by_side(heads, seqs, longest, kind, order, D, page):
    """Batches large enough that a block takes one, two or four heads, where their number allows: every way of copying."""
    rng = np.random.default_rng(heads)
    ctx = rng.integers(longest // 2, longest, seqs).tolist()
    s = Packed(53, kind, [1] * seqs, ctx, heads, heads, D, page, H16, order=order)
    qg.qgemv_attn(s.args())
    s.check()
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


@pytest.mark.parametrize("heads,seqs,longest", [(2, 130, 1500), (4, 80, 2500)])
@pytest.mark.parametrize("kind,order,D,page", [("Q4", "token-head", 128, 24), ("Q4", "token-head", 96, 8), ("Q4", "token-head", 128, 1),
                                               ("Q4", "head-token", 128, 24), ("Q8", "head-token", 64, 8), ("Q8", "head-token", 128, 7)])
def test_heads_side_by_side_over_short_pages(heads, seqs, longest, kind, order, D, page):
    """Pages that are no multiple of 16 tokens: a token's rows at once, a page's runs, from any place of a page."""
    rng = np.random.default_rng(page)
    ctx = rng.integers(longest // 2, longest, seqs).tolist()
    s = Packed(55, kind, [1] * seqs, ctx, heads, heads, D, page, H16, order=order)
    qg.qgemv_attn(s.args())
    s.check()
    assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0


def test_more_sequences_than_are_kept():
    rng = np.random.default_rng(3)
    ctx = rng.integers(0, 90, 1100).tolist()
    s = Packed(54, "Q4", [1] * 1100, ctx, 2, 1, 64, 16, B16)
    qg.qgemv_attn(s.args())
    s.check()


def test_caches_inside_larger_allocations_and_unlike_strides():
    """Keys and values in one allocation, rows further apart than they are long: every row is copied for itself or by tensor map."""
    for page in (16, 3):
        s = Packed(55, "Q4", [2], [333], 8, 4, 128, page, B16)
        pages = s.kc.shape[0]
        wide = torch.full((pages, page, 4, 2, 96), 0xFF, dtype=torch.uint8, device="cuda")
        wide[..., 0, :80], wide[..., 1, :80] = s.kc, s.vc
        s.kc, s.vc = wide[..., 0, :80], wide[..., 1, :80].clone()  # values packed closely, keys not
        qg.qgemv_attn(s.args())
        s.check()
        s.vc = wide[..., 1, :80]
        qg.qgemv_attn(s.args())
        s.check()


def test_rows_of_the_output_that_no_sequence_has():
    s = Packed(56, "Q8", [2, 1], [40, 20], 4, 2, 64, 16, B16)
    s.starts = torch.tensor([1, 3, 4], dtype=torch.int32, device="cuda")
    q = torch.full((6, 4, 64), float("nan"), dtype=B16, device="cuda")
    q[1:4] = s.q
    out, s.q = torch.full_like(q, 7.0), q
    a = s.args(out=out, max_q=2)
    qg.qgemv_attn(a)
    assert bool((out[[0, 4, 5]] == 7.0).all()) and bool((s.lse[[0, 4, 5]] == 7.0).all())
    s.q, s.out, s.lse = q[1:4], out[1:4], s.lse[1:4]
    s.check()
