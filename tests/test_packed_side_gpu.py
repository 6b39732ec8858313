"""Attention over a packed cache where a block takes several key/value heads side by side: every build and way of copying, with grouped queries,
several new tokens, windows and idle slots, against the formula in 64 bits.  Each case says how many heads the planner has to take, so that
none is emptied by another choice.  Tolerances are those of test_packed_attn_gpu.py."""
import numpy as np
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
from .test_packed_attn_gpu import B16, H16, Packed, _lib, rows_kernel  # noqa: E402,F401

CASES = [
    # sequences, new tokens of each up to, contexts up to, heads, kv heads, dim, page, order, type; heads side by side without and with the window
    (16, 5, 4000, 16, 8, 128, 32, "token-head", H16, 2, 1),      # drafts, rows of a tile up to 16
    (16, 5, 4000, 16, 8, 128, 32, "token-head", B16, 2, 1),
    (40, 4, 1500, 32, 8, 128, 16, "token-head", B16, 4, 2),      # 16 rows, four heads: whole lines of a token's heads
    (40, 4, 1500, 32, 8, 64, 16, "head-token", H16, 4, 2),       # lines of a head's tokens
    (40, 1, 2100, 64, 8, 128, 16, "head-token", B16, 4, 2),      # eight query heads to one of the cache
    (40, 9, 1500, 32, 8, 64, 24, "token-head", B16, 4, 4),       # more rows than a tile; pages that are no multiple of 16: a token's rows
    (40, 2, 2400, 8, 8, 96, 40, "head-token", H16, 4, 2),        # runs of a page's tokens; heads inside a padded tile
    (40, 3, 1500, 16, 8, 256, 16, "token-head", B16, 4, 2),      # long heads
    (40, 3, 1500, 16, 8, 256, 16, "head-token", H16, 4, 2),
    (70, 1, 1100, 12, 6, 160, 16, "token-head", H16, 2, 2),      # six heads: two side by side
    (1030, 1, 90, 8, 4, 64, 16, "token-head", B16, 2, 2),        # more sequences than are kept in shared memory
]
WINDOW = 1024


@pytest.mark.parametrize("kind", ["Q4", "Q8"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_heads_side_by_side(case, kind, rows_kernel):
    seqs, most, ctx, H, KH, D, page, order, dtype, side, window_side = CASES[case]
    rng = np.random.default_rng(case)
    new = rng.integers(max(1, most // 2), most + 1, seqs).tolist()
    lens = rng.integers(most, ctx + 1, seqs).tolist()
    new[0], lens[0], new[3], lens[3], new[-1], lens[-1], new[-2] = most, ctx, 1, 0, 1, 1, 0
    s = Packed(70 + case, kind, new, lens, H, KH, D, page, dtype, order)
    for mask, want in ((dict(), side), (dict(window=WINDOW), window_side)):
        a = s.args(**mask)
        plan = qg.qgemv_attn_plan_info(a.cache.contents.kind, a.kind, seqs, a.tokens, H, KH, D, a.max_q, a.max_kv, a.window)
        assert (plan["route"], plan["heads_side"]) == (qg.ROUTE_ATTN_PACKED, want)
        qg.qgemv_attn(a)
        s.check(**mask)
        assert int(s.scratch[:qg.QGEMV_ATTN_SCRATCH_HEAD].sum()) == 0
        first = s.out.clone(), s.lse.clone()
        qg.qgemv_attn(a, qg.QGEMV_FLAG_PDL)
        assert torch.equal(first[0], s.out) and torch.equal(first[1], s.lse)
