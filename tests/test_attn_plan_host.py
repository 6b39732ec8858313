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
