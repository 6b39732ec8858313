"""The copy of a packed cache's contexts that many rows read, on the GPU: what it keeps of values that are no numbers and of pages outside the
cache.  Tolerances are those of test_packed_attn_gpu.py."""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import B16, H16, Packed, _lib, copying, rows_kernel  # noqa: E402,F401


@pytest.fixture(params=[1, 2], ids=["codes", "copy"])
def kernel(request):
    qg.qgemv_tune_attn(request.param)
    yield qg.ROUTE_ATTN_PACKED if request.param == 1 else qg.ROUTE_ATTN_TILES
    qg.qgemv_tune_attn(0)


@pytest.mark.parametrize("dtype", [B16, H16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_a_nan_in_the_cache_is_seen(kind, dtype, kernel):
    """A key that is no number takes the rows of its head, a value's block its 32 elements of them: by either kernel."""
    for D in (128, 64):
        s = Packed(61, kind, [40], [300], 8, 2, D, 16, dtype)
        cache = qg.packed_cache(kind, s.kc, s.vc, D)
        for side in ("k", "v"):
            held = s.kc.clone(), s.vc.clone()
            rows = torch.randn(2, 1, 2, D, device="cuda")
            rows[0 if side == "k" else 1, 0, 1, 37] = float("nan")
            slot = s.table[0, 5].long().reshape(1) * 16 + 9  # token 89, which every row sees
            qg.qgemv_cache_write(qg.cache_write_args(rows[0], rows[1], cache, slot))
            qg.qgemv_route_reset()
            qg.qgemv_attn(s.args())
            assert qg.qgemv_route_counts()[kernel] == 1
            want = torch.zeros(40, 8, D, dtype=torch.bool, device="cuda")
            want[:, 4:, slice(None) if side == "k" else slice(32, 64)] = True
            assert torch.equal(s.out.isnan(), want)
            assert bool(s.lse[:, :4].isfinite().all())
            assert bool(s.lse[:, 4:].isnan().all()) == (side == "k")
            s.kc.copy_(held[0]), s.vc.copy_(held[1])


@pytest.mark.parametrize("dtype", [B16, H16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("page,gone", [(16, (3, 7)), (5, (0, 1, 40, 79)), (64, (0, 6)), (128, (1,)), (48, (0, 8))])
@pytest.mark.parametrize("new", [9, 150])
def test_pages_outside_the_cache_are_masked_for_many_rows(new, page, gone, kind, dtype, kernel):
    """Every row sees the same keys, those of the pages that are there, and nothing of the others."""
    for D in (128, 64):
        s = Packed(62, kind, [new, 3], [400, 70], 6, 2, D, page, dtype)
        for i, p in enumerate(gone):
            s.table[0, p] = (-1, 2 ** 30, s.kc.shape[0])[i % 3]
        qg.qgemv_route_reset()
        qg.qgemv_attn(s.args(causal=False))
        assert qg.qgemv_route_counts()[kernel] == 1
        assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
        keep = np.setdiff1d(np.arange(400), np.concatenate([np.arange(p * page, (p + 1) * page) for p in gone]))
        s.k[0], s.v[0], s.ctx = s.k[0][keep], s.v[0][keep], [keep.size, 70]
        s.check(causal=False, copy=kernel == qg.ROUTE_ATTN_TILES)


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_only_pages_outside_the_cache(kind, kernel):
    s = Packed(63, kind, [70], [100], 4, 2, 128, 32, B16)
    s.table[0, :4] = -1
    qg.qgemv_attn(s.args())
    assert qg.qgemv_device_error(reset=True) == qg.QGEMV_DEVERR_BAD_INDEX
    assert not bool(s.out.any()) and bool(s.lse.isneginf().all())


@pytest.mark.parametrize("dtype", [B16, H16], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", ["Q4", "Q8"])
def test_a_chunk_by_the_planners_choice(kind, dtype):
    """Many rows reach the copy without the tuning hook, and are held to the formula, f16 ones too."""
    for mask in (dict(), dict(window=500), dict(causal=False)):
        s = Packed(64, kind, [700, 90, 1], [2500, 90, 800], 16, 2, 128, 16, dtype)
        qg.qgemv_route_reset()
        qg.qgemv_attn(s.args(**mask))
        counts = qg.qgemv_route_counts()
        if not mask.get("window"):
            assert counts[qg.ROUTE_ATTN_TILES] == 1
        s.check(copy=counts[qg.ROUTE_ATTN_TILES] == 1, **mask)
