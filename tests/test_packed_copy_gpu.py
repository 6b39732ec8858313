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
