"""qgemv_attn with a few rows of many sequences, at the numbers of them where the division over the blocks keeps them elsewhere (registers,
shared memory, nowhere), against the formula in 64 bits.  Tolerances are those of test_step_gpu.py and test_packed_attn_gpu.py."""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import Packed, _lib  # noqa: E402,F401
from .test_step_gpu import B16, H16, Step  # noqa: E402


@pytest.fixture(autouse=True)
def rows_kernel():
    qg.qgemv_tune_attn(1)
    yield
    qg.qgemv_tune_attn(0)


@pytest.mark.parametrize("cache", ["16 bits", "Q4", "Q8"])
@pytest.mark.parametrize("D,dtype", [(64, B16), (128, H16), (160, B16)])
@pytest.mark.parametrize("seqs", [32, 33, 299, 300, 301, 1024, 1025])
def test_numbers_of_sequences(seqs, D, dtype, cache):
    rng = np.random.default_rng(seqs)
    new = rng.integers(0, 4, seqs).tolist()
    ctx = [int(c) for c in rng.integers(0, 60, seqs)]
    new[5], ctx[5], new[seqs // 2], ctx[seqs // 2], new[-1], ctx[-1] = 3, 900, 1, 0, 2, 70
    s = Step(3, new, ctx, 4, 2, D, 16, dtype) if cache == "16 bits" else Packed(3, cache, new, ctx, 4, 2, D, 16, dtype)
    for mask in (dict(), dict(window=20)):
        a = s.args(**mask)
        qg.qgemv_attn(a)
        s.check(**mask)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
        first = s.out.clone(), s.lse.clone()
        qg.qgemv_attn(a, qg.QGEMV_FLAG_PDL)
        assert torch.equal(first[0], s.out) and torch.equal(first[1], s.lse)
