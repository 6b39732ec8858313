"""The scratch of attention over a packed cache without a GPU: what its sizes serve, and what becomes of a call whose copy it has no room for."""
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from .test_packed_host import BF16, F16, L, Q4, Q8, attn, cache, pytestmark, scratch  # noqa: F401

SIZES = [(1, 1, 777), (48, 1, 16384), (48, 9, 131072), (16, 5, 4000), (1, 2000, 24000), (48, 2000, 16384), (2, 40, 300), (7, 130, 9000),
         (256, 512, 131072)]


def least(kind, *sizes):
    return int(qg.lib().qgemv_attn_scratch_least(kind, *sizes))


@pytest.fixture(params=[0, 1, 2], ids=["planned", "few rows", "many rows"])
def hook(request):
    qg.qgemv_tune_attn(request.param)
    yield request.param
    qg.qgemv_tune_attn(0)


def rows_of(kind, dim=128):
    row = qg.qgemv_cache_row_bytes(kind, dim)
    return cache(kind=kind, dim=dim, k_page=16 * 8 * row, k_token=8 * row, k_head=row, v_page=16 * 8 * row, v_token=8 * row, v_head=row)


def call(L, kind, dtype, seqs, new, ctx, n, window=0):  # noqa: F811
    return L.qgemv_attn(attn(cache=rows_of(kind), q=1 << 41, out=1 << 42, pages=1 << 43, q_start=1 << 44, kv_len=1 << 45, kind=dtype, seqs=seqs, tokens=seqs * new, max_q=new, max_kv=ctx, window=window,
                             pages_stride=-(-ctx // 16), scratch=1 << 50, scratch_bytes=n), 0, None)


@pytest.mark.parametrize("kind", [Q4, Q8])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_a_scratch_without_room_for_the_copy_is_taken(L, kind, size, hook):  # noqa: F811
    """Any number of rows is served without a copy, so that no call is refused for want of one."""
    seqs, new, ctx = size
    n = least(kind, seqs, seqs * new, 32, 8, 128, new, ctx)
    assert qg.QGEMV_ATTN_SCRATCH_HEAD < n <= scratch(kind, seqs, seqs * new, 32, 8, 128, new, ctx)
    if hook != 2:
        assert n <= 64 << 20
    for dtype in (BF16, F16):
        for q, kv, window in ((new, ctx, 0), (new, ctx, 100), (max(1, new // 2), ctx, 0), (new, max(1, ctx // 3), 1000), (1, 1, 0)):
            assert call(L, kind, dtype, seqs, q, kv, n, window) in (4, 5)
            assert call(L, kind, dtype, seqs, q, kv, qg.QGEMV_ATTN_SCRATCH_HEAD, window) == 1
    assert call(L, kind, BF16, 1, min(new, 2), min(ctx, 50), n) in (4, 5)


def test_the_least_of_a_16_bit_cache_is_all_of_it(L, hook):  # noqa: F811
    for seqs, new, ctx in SIZES:
        assert least(BF16, seqs, seqs * new, 32, 8, 128, new, ctx) == qg.qgemv_attn_scratch_bytes(seqs, seqs * new, 32, 8, 128, new, ctx)
    assert least(0, 1, 1, 32, 8, 128, 1, 1) == 0 and least(Q4, 1, 1, 32, 8, 40, 1, 1) == 0 and least(Q4, 1, 1, 30, 8, 128, 1, 1) == 0


def test_the_binding_asks_for_the_least(L):  # noqa: F811
    c = rows_of(Q8)
    assert qg.qgemv_attn_scratch_bytes(1, 2000, 32, 8, 128, 2000, 24000, cache=c, least=True) == least(Q8, 1, 2000, 32, 8, 128, 2000, 24000)
    assert qg.qgemv_attn_scratch_bytes(1, 2000, 32, 8, 128, 2000, 24000, cache=c) == scratch(Q8, 1, 2000, 32, 8, 128, 2000, 24000)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 1, 32), (32, 8, 128), (16, 8, 64)])
@pytest.mark.parametrize("kind", [Q4, Q8])
def test_the_scratch_never_falls_at_the_ends_of_the_copys_range(L, kind, heads, kv_heads, dim):  # noqa: F811
    """Around 65535 sequences and 2^31 tokens, beyond which a call makes no copy, and around the bytes that are counted for one."""
    for new in (9, 17, 40, 512):
        for fixed, sizes in (("context", [(s, c) for c in (0, 256, 4096) for s in (1, 300, 40000, 65534, 65535, 65536, 65537, 100000)]),
                             ("sequences", [(s, c) for s in (1, 63, 64, 4096) for c in (1, 1 << 16, (1 << 19) - 129, 1 << 19, (1 << 25) - 129, (1 << 25) - 128,
                                                                                         (1 << 25) - 127, 1 << 25, 1 << 27, 1 << 30)])):
            last, key = 0, None
            for s, c in sizes:
                n = scratch(kind, s, s * new, heads, kv_heads, dim, new, c)
                if n == 0:  # (more row tiles than the kernel's arithmetic takes: the sizes are refused)
                    assert s * kv_heads * -(-new * (heads // kv_heads) // 16) > 10 ** 8
                    continue
                here = c if fixed == "context" else s
                assert n >= (last if here == key else 0), (new, s, c)
                # beside the copy, parts: up to 16 waves of 152 row tiles of 256 rows, dim floats and two more a row
                assert n <= qg.QGEMV_ATTN_COPY_MAX + 16 * 152 * 256 * (4 * dim + 8) + (1 << 20)
                last, key = n, here


@pytest.mark.parametrize("kind", [Q4, Q8])
def test_the_scratch_of_the_largest_sizes_serves_calls_with_and_without_a_copy(L, kind):  # noqa: F811
    for most in ((65536, 9, 256), (65535, 9, 256), (64, 512, 1 << 26), (256, 512, 131072)):
        seqs, new, ctx = most
        n = scratch(kind, seqs, seqs * new, 32, 8, 128, new, ctx)
        for s, q, c in (most, (1, new, min(ctx, 24000)), (seqs - 1, new, ctx), (min(seqs, 100), new, ctx), (seqs, 1, ctx), (2, new // 2, ctx // 2)):
            for dtype in (BF16, F16):
                assert call(L, kind, dtype, s, q, c, n) in (4, 5)


def test_the_bindings_bound_is_the_headers():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qgemv.h")).read()
    assert int(re.search(r"#define QGEMV_ATTN_COPY_MAX (\d+)ull", text).group(1)) == qg.QGEMV_ATTN_COPY_MAX
