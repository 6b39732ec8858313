"""Attention of many rows over a packed cache with and without room for the copy of its contexts, against the formula in 64 bits."""
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import B16, H16, Packed, _lib  # noqa: E402,F401


# The least scratch of 9 rows and more holds 38912 records of 520 bytes, 20.2 MB.  Two sequences' copy (2 x 2128 tokens of 1028 bytes, 4.4 MB, and the
# queries' 2.1 MB) has room in it, twelve sequences' (26 MB) has none.
@pytest.mark.parametrize("others,room_for_copy", [(1, True), (11, False)])
@pytest.mark.parametrize("dtype", [B16, H16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_a_chunk_with_the_least_scratch(kind, dtype, others, room_for_copy):
    s = Packed(51, kind, [1000] + [1] * others, [2000] + [300] * others, 8, 2, 128, 16, dtype)
    qg.qgemv_route_reset()
    qg.qgemv_attn(s.args())  # (the planner's own choice)
    assert qg.qgemv_route_counts()[qg.ROUTE_ATTN_TILES] == 1
    s.check(copy=True)
    n = qg.qgemv_attn_scratch_bytes(1 + others, 1000 + others, 8, 2, 128, 1000, 2000, cache=qg.packed_cache(kind, s.kc, s.vc, 128), least=True)
    room = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    room[:qg.QGEMV_ATTN_SCRATCH_HEAD] = 0
    for mask in (dict(), dict(window=300), dict(causal=False)):
        qg.qgemv_route_reset()
        qg.qgemv_attn(s.args(scratch=room[:n], **mask))
        counts = qg.qgemv_route_counts()
        assert counts[qg.ROUTE_ATTN_PACKED] + counts[qg.ROUTE_ATTN_TILES] == 1
        if not room_for_copy:
            assert counts[qg.ROUTE_ATTN_PACKED] == 1
        s.check(copy=counts[qg.ROUTE_ATTN_TILES] == 1, **mask)
        assert int(room[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0 and bool((room[n:] == 0x5A).all())
