"""What qgemv_attn plans for a call's sizes, without a GPU."""
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

B16, H16, Q4, Q8 = qg.QGEMV_ACT_BF16, qg.QGEMV_ACT_F16, qg.QGEMV_CACHE_Q4, qg.QGEMV_CACHE_Q8
ROWS, TILES, PACKED = qg.ROUTE_ATTN_ROWS, qg.ROUTE_ATTN_TILES, qg.ROUTE_ATTN_PACKED


@pytest.fixture(scope="module", autouse=True)
def _lib():
    qg.build()


def plan(cache, kind, seqs, new, ctx, heads=32, kv_heads=8, dim=128, window=0):
    return qg.qgemv_attn_plan_info(cache, kind, seqs, seqs * new, heads, kv_heads, dim, new, ctx, window)


def test_the_kernels_of_a_16_bit_cache():
    one, chunk = plan(B16, B16, 1, 1, 777), plan(H16, H16, 1, 2000, 24000)
    assert (one["route"], one["heads_side"], one["tile_rows"]) == (ROWS, 1, 16)
    assert (chunk["route"], chunk["heads_side"], chunk["tile_rows"]) == (TILES, 1, 256)
    assert one["scratch_bytes"] <= qg.qgemv_attn_scratch_bytes(1, 1, 32, 8, 128, 1, 777)
    assert chunk["scratch_bytes"] <= qg.qgemv_attn_scratch_bytes(1, 2000, 32, 8, 128, 2000, 24000)


@pytest.mark.parametrize("cache", [Q4, Q8])
@pytest.mark.parametrize("kind", [B16, H16])
def test_the_kernels_of_a_packed_cache(cache, kind):
    assert plan(cache, kind, 1, 1, 777)["route"] == PACKED and plan(cache, kind, 1, 1, 777)["heads_side"] == 1
    assert plan(cache, kind, 48, 1, 16384)["heads_side"] == 4 and plan(cache, kind, 48, 1, 16384)["tile_rows"] == 8
    assert plan(cache, kind, 16, 5, 4000, 16, 8)["tile_rows"] == 16
    assert plan(cache, kind, 48, 1, 16384, 32, 1)["heads_side"] == 1
    assert plan(cache, kind, 1, 2000, 24000)["route"] == TILES and plan(cache, kind, 1, 2000, 24000, dim=256)["route"] == PACKED


def test_refusals():
    L, buf = qg.lib(), (qg.ctypes.c_longlong * 4)()
    good = [Q4, B16, 1, 1, 32, 8, 128, 1, 777, 0]
    assert L.qgemv_attn_plan_info(*good, buf) == 0 and L.qgemv_attn_plan_info(*good, None) == 1
    for i, v in ((0, 5), (0, H16), (1, 0), (1, Q4), (2, -1), (4, 30), (5, 0), (6, 40), (6, 0), (7, -1), (8, -1), (9, -1)):
        bad = list(good)
        bad[i] = v
        assert L.qgemv_attn_plan_info(*bad, buf) == 1, (i, v)
    assert L.qgemv_attn_plan_info(Q4, B16, 1, 1, 32, 8, 288, 1, 777, 0, buf) == 2


# packed cache's own kernel against the 128-row kernel over the copy, measured (us), where one is clearly faster.  8 key/value heads, 32 query heads:
# (cache, sequences, new tokens, bound of the contexts, dim, us of the packed kernel, of the copy); lengths equal to the bound, or as said
CHOICES = [
    (Q4, 1, 9, 100000, 64, 84.5, 140.2), (Q4, 1, 16, 100000, 64, 108.3, 140.0), (Q8, 1, 12, 100000, 64, 90.6, 140.4),
    (Q4, 1, 16, 24000, 64, 37.6, 51.1), (Q8, 1, 16, 24000, 64, 39.2, 52.7), (Q4, 1, 16, 100000, 128, 150.3, 201.9),
    (Q8, 1, 12, 100000, 128, 148.2, 203.1), (Q4, 8, 12, 16000, 128, 157.9, 268.2), (Q4, 32, 16, 4000, 128, 182.8, 279.7),
    (Q4, 48, 16, 16384, 128, 486.9, 797.8),  # 0.42 of the bound in the mean
    (Q4, 1, 32, 24000, 128, 85.3, 70.0), (Q4, 1, 64, 100000, 64, 398.3, 153.9), (Q8, 1, 32, 24000, 64, 66.7, 53.6),
    (Q4, 2, 32, 24000, 128, 152.1, 110.9), (Q4, 8, 32, 16000, 128, 375.7, 259.6), (Q4, 8, 32, 16000, 64, 260.4, 183.0),
    (Q8, 32, 32, 4000, 128, 397.3, 274.8), (Q4, 32, 32, 4000, 128, 330.3, 272.7),
    (Q4, 8, 24, 16000, 128, 117.7, 183.4),   # 0.36 of the bound
    (Q4, 32, 32, 4000, 128, 305.5, 192.8),   # 0.47 of the bound
    (Q4, 48, 32, 16384, 128, 1063.5, 776.1), # 0.42 of the bound
]


@pytest.mark.parametrize("case", CHOICES, ids=str)
def test_many_rows_go_to_the_faster_kernel(case):
    """Whatever the lengths' mean is of their bound: no batch is judged by that of another."""
    cache, seqs, new, ctx, dim, packed, copy = case
    for kind in (B16, H16):
        assert plan(cache, kind, seqs, new, ctx, dim=dim)["route"] == (PACKED if packed < copy else TILES)


@pytest.mark.parametrize("cache", [Q4, Q8])
def test_drafts_ask_for_no_copy(cache):
    """Up to 64 rows of a sequence the copy is never faster, so that none is counted in the scratch of such calls."""
    for seqs, new, ctx in ((48, 9, 131072), (64, 16, 32768), (300, 12, 1 << 17)):
        assert qg.lib().qgemv_attn_scratch_bytes_ex(cache, seqs, seqs * new, 32, 8, 128, new, ctx) <= 64 << 20


@pytest.mark.parametrize("cache", [Q4, Q8])
def test_a_mixed_step_is_judged_by_all_its_tokens(cache):
    """One chunk among 47 single tokens (us of the packed kernel / of the copy, 4 bits): not as if every sequence had a chunk."""
    for new, ctx, route in ((40, 4000, PACKED), (500, 4000, PACKED), (2000, 16384, TILES)):  # 68 / 238, 198 / 275, 2355 / 1288
        assert qg.qgemv_attn_plan_info(cache, B16, 48, new + 47, 32, 8, 128, new, ctx)["route"] == route
        assert qg.qgemv_attn_plan_info(cache, B16, 48, 48 * new, 32, 8, 128, new, ctx)["route"] == TILES
