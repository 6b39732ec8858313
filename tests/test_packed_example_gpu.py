"""The example over a packed cache: a graph replayed step by step samples what the same calls one by one do."""
import os
import sys

import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("kind,seqs,prompt,steps", [("Q4", 1, 1, 5), ("Q8", 3, 41, 20), ("Q4", 16, 70, 4)])
def test_decode_step_over_a_packed_cache(kind, seqs, prompt, steps):
    import decode_step
    qg.build()
    qg.qgemv_device_error(reset=True)
    a = decode_step.generate(seqs, prompt, steps, graph=False, kind=kind)
    b = decode_step.generate(seqs, prompt, steps, graph=True, kind=kind)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(((a[0] >= 0) & (a[0] < decode_step.VOCAB)).all()) and bool(((a[1] > 0) & (a[1] <= 1)).all())
    assert qg.qgemv_device_error() == 0
