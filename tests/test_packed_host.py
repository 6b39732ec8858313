"""The packed key/value cache without a GPU: argument checks, sizes, and the reference of its rows against the definition."""
import ctypes
import glob
import os

import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from . import packedref as ref
from .test_step_host import BF16, F16, F32, FREQ, KC, KO, LEN, LSE, POS, Q, QO, SCR, SLOT, ST, TAB, VC, G, K, V

torch = pytest.importorskip("torch")

# fake addresses must never reach a GPU: none of this runs where there is one
pytestmark = pytest.mark.skipif(bool(glob.glob("/dev/nvidia[0-9]*")) or os.path.exists("/dev/nvidiactl"), reason="for hosts without a GPU")
Q4, Q8 = qg.QGEMV_CACHE_Q4, qg.QGEMV_CACHE_Q8


@pytest.fixture(scope="module")
def L():
    qg.build()
    return qg.lib()


def cache(**kw):
    c = dict(k=KC, v=VC, k_page=16 * 8 * 80, k_token=8 * 80, k_head=80, v_page=16 * 8 * 80, v_token=8 * 80, v_head=80, kind=Q4,
             num_pages=100, page_size=16, heads=8, dim=128)
    c.update(kw)
    return qg.QgemvCache(**c)


def put(record, c):
    if c is not None:
        record.cache = ctypes.pointer(c)
    return record


def write(**kw):
    c = kw.pop("cache", cache())
    a = dict(k=K, v=V, k_token=1024, k_head=128, v_token=1024, v_head=128, slots=SLOT, x_kind=F32, tokens=5)
    a.update(kw)
    return put(qg.QgemvCacheWriteArgs(**a), c)


def read(**kw):
    c = kw.pop("cache", cache())
    a = dict(pages=TAB, pages_stride=40, out_start=ST, first=LEN, k_out=KO, v_out=QO, k_token=1024, k_head=128, v_token=1024, v_head=128,
             out_kind=BF16, tokens=30, seqs=3, max_kv=600)
    a.update(kw)
    return put(qg.QgemvCacheReadArgs(**a), c)


def attn(**kw):
    c = kw.pop("cache", cache())
    a = dict(q=Q, out=QO, lse=None, q_token=4096, q_head=128, out_token=4096, out_head=128, pages=TAB, pages_stride=40, q_start=ST,
             kv_len=LEN, scratch=SCR, scratch_bytes=1 << 29, kind=BF16, tokens=6, heads=32, seqs=3, max_q=2, max_kv=600, scale=0.088,
             causal=1, window=0)
    a.update(kw)
    return put(qg.QgemvAttnArgs(**a), c)


def rope(**kw):
    c = kw.pop("cache", cache())
    a = dict(q=Q, k=K, v=V, q_out=QO, k_out=KO, q_token=4096, q_head=128, k_token=1024, k_head=128, v_token=1024, v_head=128,
             q_out_token=4096, q_out_head=128, k_out_token=1024, k_out_head=128, positions=POS, freqs=FREQ, slots=SLOT, x_kind=F32,
             out_kind=BF16, tokens=5, heads=32, kv_heads=8, dim=128, rot_dim=128, layout=0, mscale=1.0)
    a.update(kw)
    return put(qg.QgemvRopeArgs(**a), c)


CACHES = [  # refused by every operator that takes a packed cache
    (dict(k=None), 1), (dict(kind=5), 1), (dict(kind=F32), 1), (dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1),
    (dict(dim=120), 1), (dict(dim=16), 1), (dict(k_page=-80), 1), (dict(k_token=0), 1), (dict(v_head=0), 1), (dict(v_page=0), 1),
    (dict(dim=288), 2), (dict(k_token=1 << 31), 2), (dict(v_head=1 << 32), 2), (dict(v_page=(1 << 39) + 16), 2),
    (dict(k=KC + 8), 3), (dict(v=VC + 4), 3), (dict(k_head=88), 3), (dict(v_token=8 * 80 + 8), 3), (dict(k_page=16 * 8 * 80 + 4), 3),
]


@pytest.mark.parametrize("case,status", CACHES)
def test_packed_caches_that_are_refused(L, case, status):
    # (heads and dim of the other arguments go along, so that the cache itself is what is wrong)
    heads, dim = case.get("heads", 8), case.get("dim", 128)
    assert L.qgemv_cache_write(write(cache=cache(**case)), 0, None) == status
    assert L.qgemv_cache_read(read(cache=cache(**case)), 0, None) == status
    assert L.qgemv_attn(attn(cache=cache(**case)), 0, None) == status
    if heads == 8 and dim == 128:
        assert L.qgemv_rope(rope(cache=cache(**case)), 0, None) == status


def test_a_stride_over_one_element_is_not_looked_at(L):
    c = cache(num_pages=1, page_size=1, heads=1, k_page=0, k_token=0, k_head=0, v_page=0, v_token=1 << 40, v_head=0)
    assert L.qgemv_cache_write(write(cache=c, k_token=128, v_token=128), 0, None) in (4, 5)


WRITE = [
    (dict(cache=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(x_kind=0), 1), (dict(x_kind=Q4), 1),
    (dict(tokens=-1), 1), (dict(k_token=-1024), 1), (dict(cache=cache(kind=BF16)), 1),
    (dict(cache=cache(heads=70000, k_token=70000 * 80, v_token=70000 * 80, k_page=70000 * 1280, v_page=70000 * 1280)), 2),
    (dict(k=K + 8), 3), (dict(v_token=1028), 3), (dict(v_head=132), 3), (dict(slots=SLOT + 4), 3),
    (dict(k=KC), 6), (dict(v=VC + 512), 6), (dict(k=VC), 6), (dict(slots=KC + 64), 6),
]


@pytest.mark.parametrize("case,status", WRITE)
def test_write_refuses_on_host(L, case, status):
    assert L.qgemv_cache_write(write(**case), 0, None) == status


READ = [
    (dict(cache=None), 1), (dict(k_out=None, v_out=None), 1), (dict(pages=None), 1), (dict(out_start=None), 1), (dict(out_kind=0), 1),
    (dict(out_kind=Q8), 1), (dict(tokens=-1), 1), (dict(seqs=-1), 1), (dict(pages_stride=-1), 1), (dict(max_kv=-1), 1),
    (dict(cache=cache(kind=F16)), 1), (dict(pages_stride=1 << 41), 2),
    (dict(k_out=KO + 8), 3), (dict(v_token=1028), 3), (dict(pages=TAB + 2), 3), (dict(out_start=ST + 1), 3), (dict(first=LEN + 2), 3),
    (dict(k_out=KC), 6), (dict(v_out=VC + 64), 6), (dict(v_out=TAB), 6), (dict(k_out=ST - 64), 6), (dict(v_out=LEN), 6), (dict(v_out=KO), 6),
]


@pytest.mark.parametrize("case,status", READ)
def test_read_refuses_on_host(L, case, status):
    assert L.qgemv_cache_read(read(**case), 0, None) == status


ATTN = [
    (dict(kind=F32), 1), (dict(kind=Q4), 1), (dict(heads=31), 1), (dict(scratch=None), 1), (dict(scale=float("nan")), 1),
    (dict(scratch_bytes=qg.QGEMV_ATTN_SCRATCH_HEAD), 1), (dict(out=KC), 6), (dict(scratch=VC), 6), (dict(out=KC + 100 * 16 * 8 * 80 - 16), 6),
]


@pytest.mark.parametrize("case,status", ATTN)
def test_attn_refuses_on_host(L, case, status):
    assert L.qgemv_attn(attn(**case), 0, None) == status


def test_valid_calls_without_a_gpu(L):
    for f, record in ((L.qgemv_cache_write, write), (L.qgemv_cache_read, read), (L.qgemv_attn, attn), (L.qgemv_rope, rope)):
        for kind, row in ((Q4, 80), (Q8, 144)):
            c = cache(kind=kind, k_page=16 * 8 * row, k_token=8 * row, k_head=row, v_page=16 * 8 * row, v_token=8 * row, v_head=row)
            assert f(record(cache=c), 0, None) in (4, 5) and f(record(cache=c), qg.QGEMV_FLAG_PDL, None) in (4, 5)
            assert f(record(cache=c), 2, None) == 1 and f(None, 0, None) == 1
    assert L.qgemv_attn(attn(kind=F16, lse=LSE), 0, None) in (4, 5)  # queries of either type
    assert L.qgemv_cache_read(read(first=None, v_out=None), 0, None) in (4, 5)
    assert L.qgemv_rope(rope(k=K, k_out=K, x_kind=BF16), 0, None) in (4, 5)  # keys turned in place and packed
    assert L.qgemv_attn(attn(out=KC + 100 * 16 * 8 * 80), 0, None) in (4, 5)  # right behind the cache's last byte


def test_no_tokens_is_nothing_to_do(L):
    assert L.qgemv_cache_write(write(tokens=0, k=None, v=None, slots=None), 0, None) == 0
    assert L.qgemv_cache_read(read(tokens=0, k_out=None, v_out=None, out_start=None), 0, None) == 0
    assert L.qgemv_cache_read(read(seqs=0), 0, None) == 0
    assert L.qgemv_attn(attn(tokens=0), 0, None) == 0 and L.qgemv_rope(rope(tokens=0), 0, None) == 0


def test_failure_injection_reaches_the_operators(L):
    qg.qgemv_debug_fail_next(4, 2)
    assert L.qgemv_cache_write(write(), 0, None) == 4 and L.qgemv_cache_read(read(), 0, None) == 4
    qg.qgemv_debug_fail_next(0, 0)


def test_row_bytes(L):
    for bits, kind in ((4, "Q4"), (8, "Q8")):
        for dim in ref.DIMS:
            assert qg.qgemv_cache_row_bytes(kind, dim) == ref.row_bytes(bits, dim)
    assert qg.qgemv_cache_row_bytes("Q4", 128) == 80 and qg.qgemv_cache_row_bytes("Q8", 128) == 144
    for kind, dim in ((Q4, 0), (Q4, 48), (Q4, 288), (BF16, 128), (0, 128)):
        assert qg.qgemv_cache_row_bytes(kind, dim) == 0


def scratch(kind, *sizes):
    return int(qg.lib().qgemv_attn_scratch_bytes_ex(kind, *sizes))


def test_scratch_sizes(L):
    assert scratch(BF16, 1, 1, 32, 8, 128, 1, 100000) == qg.qgemv_attn_scratch_bytes(1, 1, 32, 8, 128, 1, 100000)
    assert scratch(0, 1, 1, 32, 8, 128, 1, 1) == 0 and scratch(Q4, 1, 1, 32, 8, 40, 1, 1) == 0 and scratch(Q4, 1, 1, 30, 8, 128, 1, 1) == 0
    # no copy for single tokens and drafts, whatever the batch; one of the contexts where many rows may read it
    for seqs, new, ctx in ((1, 1, 1 << 20), (64, 1, 32768), (4096, 1, 4096), (300, 7, 1 << 17)):
        assert 0 < scratch(Q4, seqs, seqs * new, 32, 8, 128, new, ctx) <= 64 << 20
    copy = 24000 * 8 * 128 * 4
    plain = qg.qgemv_attn_scratch_bytes(1, 2000, 32, 8, 128, 2000, 24000)  # (of parts)
    assert copy <= scratch(Q4, 1, 2000, 32, 8, 128, 2000, 24000) <= copy + plain + 2000 * 32 * 260 + (4 << 20)
    # it never falls as a size grows
    for kind in (Q4, Q8):
        for dim in (64, 128, 256):
            last = 0
            for seqs, new, ctx in ((1, 1, 10), (1, 2, 10), (1, 3, 10), (1, 8, 500), (1, 9, 500), (1, 40, 500), (1, 40, 5000), (2, 40, 5000),
                                   (2, 700, 5000), (3, 700, 70000)):
                n = scratch(kind, seqs, seqs * new, 32, 8, dim, new, ctx)
                assert n >= last
                last = n


@pytest.mark.parametrize("forced", [0, 1, 2])
@pytest.mark.parametrize("kind", [Q4, Q8])
def test_calls_of_given_sizes_are_content_with_their_scratch(L, kind, forced):
    """What the sizes' function says serves the call of those sizes and smaller ones, with any window."""
    row = qg.qgemv_cache_row_bytes(kind, 128)
    c = cache(kind=kind, k_page=16 * 8 * row, k_token=8 * row, k_head=row, v_page=16 * 8 * row, v_token=8 * row, v_head=row)
    qg.qgemv_tune_attn(forced)
    try:
        for seqs, new, ctx in ((1, 1, 777), (48, 1, 16384), (16, 5, 4000), (1, 2000, 24000), (2, 40, 300), (7, 130, 9000)):
            n = scratch(kind, seqs, seqs * new, 32, 8, 128, new, ctx)
            for q, kv, window in ((new, ctx, 0), (new, ctx, 100), (max(1, new // 2), ctx, 0), (new, ctx // 3, 1000), (1, 1, 0)):
                a = attn(cache=c, seqs=seqs, tokens=seqs * new, max_q=q, max_kv=kv, window=window, pages_stride=-(-ctx // 16), scratch_bytes=n, scratch=1 << 46)
                assert L.qgemv_attn(a, 0, None) in (4, 5)
    finally:
        qg.qgemv_tune_attn(0)


def test_binding_refuses_unlike_tensors():
    rows = torch.zeros(4, 16, 2, 80, dtype=torch.uint8)
    c = qg.packed_cache("Q4", rows, rows, 128)
    assert (c.kind, c.num_pages, c.page_size, c.heads, c.dim, c.k_page, c.k_token, c.k_head) == (Q4, 4, 16, 2, 128, 2560, 160, 80)
    x, slots = torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int64)
    table, start = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: qg.packed_cache("Q8", rows, rows, 128), lambda: qg.packed_cache("Q4", rows, rows, 120), lambda: qg.packed_cache("Q4", rows, rows[:2], 128),
        lambda: qg.packed_cache("Q4", rows.to(torch.int8), rows, 128), lambda: qg.packed_cache("Q4", rows.transpose(2, 3), rows, 128),
        lambda: qg.cache_write_args(x, x[:2], c, slots), lambda: qg.cache_write_args(x[:, :1], x[:, :1], c, slots),
        lambda: qg.cache_write_args(x, x, c, slots[:2]), lambda: qg.cache_write_args(x, x, c, slots.int()),
        lambda: qg.cache_write_args(x.double(), x.double(), c, slots),
        lambda: qg.cache_read_args(c, table, start), lambda: qg.cache_read_args(c, table, start, x, x.bfloat16()),
        lambda: qg.cache_read_args(c, table, start[:1], x), lambda: qg.cache_read_args(c, table.long(), start, x),
        lambda: qg.cache_read_args(c, table, start, x, first=start), lambda: qg.cache_read_args(c, table, start, x[..., :64]),
        lambda: qg.attn_args(x[..., :64].bfloat16(), c, table, start, start[:1], x[..., :64].bfloat16(), rows, 1, 1, 1.0),
    ]
    for f in bad:
        with pytest.raises(qg.QgemvError):
            f()
    assert qg.cache_read_args(c, table, start, x).max_kv == 64


@pytest.mark.parametrize("bits", [4, 8])
def test_the_reference_keeps_the_definition(bits):
    """The reference that GPU tests compare with, against the definition in exact fractions."""
    from fractions import Fraction
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((40, 32)).astype(np.float32) * np.float32(10.0) ** rng.integers(-6, 5, (40, 1)).astype(np.float32)
    x[0] = 3.25
    x[1, :5] = 1e6
    codes, d, m = ref.pack(x, bits)
    top = (1 << bits) - 1
    for i in range(40):
        v = [min(65504, max(-65504, Fraction(float(t)))) for t in x[i]]
        base, step = Fraction(float(m[i, 0])), Fraction(float(d[i, 0]))
        up = Fraction(float(np.nextafter(m[i, 0], np.float16(np.inf)))) if m[i, 0] < 65504 else Fraction(70000)
        assert base <= min(v) < up
        need = (max(v) - base) / top
        below = Fraction(float(np.nextafter(d[i, 0], np.float16(-np.inf)))) if d[i, 0] > 0 else Fraction(-1)
        slack = 1 + Fraction(1, 2 ** 22)  # the fp32 of the difference and of the quotient
        assert step * slack >= need and below <= need * slack
        for j in range(32):
            c = int(codes[i, j])
            assert 0 <= c <= top
            assert abs(v[j] - base - c * step) <= step / 2 * (1 + Fraction(1, 2 ** 12))
