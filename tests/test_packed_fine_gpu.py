"""What attention over a packed cache keeps of its probabilities where results are f16.

A value is v = (m + Z d) + d (c - Z) with Z the middle code.  The kernel's p d, rounded to f16 once, stands in the sum of codes and in a sum of its own alike, so that
    out = sum p (m + Z d) + sum (p d) (c - Z),
whatever p d is rounded to.  Codes that are all Z leave nothing of the second part: with m = -Z d the values are 0, and so has the result to be, but for
the arithmetic of the sums.  p and p d rounded one after another, as for bf16 results, would leave up to 2^-11 of sum p d Z.

The sums' arithmetic: tensor cores add the 16 products of a step and the sum so far with every addend cut below 2^-23 of the largest exponent among them (Fasi,
Higham, Mikaitis, Pranesh, "Numerical behavior of NVIDIA tensor cores", 2021); a product's exponent is the sum of its factors', and a subnormal factor
has that of 2^-14.  A code c stands as c 2^-24 (or, the upper half of a byte of two, c 2^-20), that is 2^10 (2^6) codes below its nominal exponent: a step
loses at most 17 2^-23 2^10 = 17 2^-13 (17 2^-17) of its largest p d.  The other sums lose 17 2^-23 of p |m| = Z p d a step, three of them together less than
2^-18 of A = 2 Z sum p d, and so does fp32 in what follows.  Steps are 16 keys from a multiple of 16 on."""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

from . import packedref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import H16, Packed, _lib, rows_kernel  # noqa: E402,F401
from .test_step_gpu import TINY, f64  # noqa: E402


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("ctx,D,KH,new", [(3, 128, 2, 1), (40, 64, 4, 2), (1000, 128, 2, 4), (300, 256, 2, 1), (90, 96, 1, 5), (2000, 32, 2, 1)])
def test_middle_codes_cancel(kind, ctx, D, KH, new, rows_kernel):
    s = Packed(81, kind, [new], [ctx], 4 * KH, KH, D, 16, H16)
    rng, z = np.random.default_rng(4), 1 << (s.bits - 1)
    d = (2.0 ** rng.uniform(-6, 1, (ctx, KH, D // 32))).astype(np.float16)
    m = (-z * d.astype(np.float64)).astype(np.float16)  # (exact)
    s.put(0, v=ref.to_bytes(np.full((ctx, KH, D), z, np.uint8), d, m, s.bits))
    assert not ref.values(s.v[0], s.bits, D).any()
    qg.qgemv_attn(s.args())
    out, broken = f64(s.out[-1]), False
    lost = np.full(D, 17 * 2.0 ** -13)
    if s.bits == 4:
        lost[1::2] /= 16
    for h in range(s.H):
        score = s.scale * (ref.values(s.k[0], s.bits, D)[:, h // 4] @ f64(s.q[-1, h]))  # the last token sees all
        p = np.exp(score - score.max())
        lifted, p = p, p / p.sum()
        step = np.repeat(d[:, h // 4].astype(np.float64), 32, -1)
        pd = p[:, None] * step
        A = 2 * z * pd.sum(0)
        tops = np.concatenate([pd, np.zeros((-ctx % 16, D))]).reshape(-1, 16, D).max(1).sum(0)
        tol = (1 + 2.0 ** -6) * (lost * tops + 2.0 ** -18 * A) + TINY[H16]  # (p itself is known to 2^-7)
        assert np.all(np.abs(out[h]) <= tol), (h, float((np.abs(out[h]) / tol).max()))
        # p and then p d rounded, 2^10 times as large as here
        once = (lifted * 1024).astype(np.float16).astype(np.float64)[:, None] * step
        left = np.abs((once.astype(np.float16).astype(np.float64) - once).sum(0)) * z / (1024 * lifted.sum())
        broken |= bool((left > tol).any())
    assert broken
