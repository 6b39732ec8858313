"""Edges of the operators between the GEMVs without a GPU: sizes at the ends of the arithmetic, the scratch over all sizes, what
the binding takes."""
import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")

from tests.test_step_host import HAS_GPU_NODE, KC, Q, QO, L, attn, cache, rope, sample  # noqa: E402,F401

HUGE, MANY = 1 << 40, 2 ** 31 - 1


# strides and sizes that are each allowed, but whose product leaves 64 bits: the memory a tensor spans cannot be told then, and
# an overlap went unseen
@pytest.mark.parametrize("case", [
    dict(q_token=HUGE, tokens=MANY), dict(q_out_token=HUGE, tokens=MANY), dict(k_token=HUGE, tokens=1 << 24),
    dict(v_token=HUGE, tokens=1 << 24), dict(cache=cache(k_page=HUGE, num_pages=1 << 24)), dict(cache=cache(v_page=HUGE, num_pages=MANY)),
    dict(cache=cache(k_token=HUGE, page_size=1 << 24)), dict(cache=cache(v_token=HUGE, page_size=MANY)),
])
def test_rope_refuses_spans_past_64_bits(L, case):  # noqa: F811
    assert L.qgemv_rope(rope(**case), 0, None) == 2


@pytest.mark.parametrize("case", [
    dict(q_token=HUGE, tokens=MANY), dict(out_token=HUGE, tokens=1 << 24), dict(seqs=MANY, pages_stride=HUGE),
    dict(pages_stride=HUGE + 1), dict(cache=cache(k_page=HUGE, num_pages=MANY)), dict(cache=cache(k_token=HUGE, page_size=MANY)),
    dict(cache=cache(v_token=HUGE, page_size=1 << 24)),
])
def test_attn_refuses_spans_past_64_bits(L, case):  # noqa: F811
    assert L.qgemv_attn(attn(**case), 0, None) == 2


def test_sample_refuses_spans_past_64_bits(L):  # noqa: F811
    assert sample(L, m=MANY, stride=HUGE) == 2
    assert sample(L, m=1 << 24, stride=HUGE) == 2


@pytest.mark.skipif(HAS_GPU_NODE, reason="checks the no-GPU path only (fake addresses must never reach a GPU)")
def test_large_strides_of_small_tensors_are_taken(L):  # noqa: F811
    assert L.qgemv_attn(attn(cache=cache(k=1 << 50, v=3 << 50, k_page=1 << 38, v_page=1 << 38)), 0, None) in (4, 5)
    # only what a row of the page table has to hold counts as read, not its whole stride
    assert L.qgemv_attn(attn(pages=KC + (1 << 29), pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) in (4, 5)
    assert L.qgemv_attn(attn(pages=QO - 256, pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) in (4, 5)
    assert L.qgemv_attn(attn(pages=QO - 148, pages_stride=1 << 26, seqs=1, max_kv=600), 0, None) == 6
