"""The example that runs the operators together: a graph replayed step by step samples what the same calls one by one do."""
import os
import sys

import pytest

import quantized_weight_gemv_quantize_gb300 as qg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("seqs,prompt,steps", [(1, 1, 5), (3, 41, 20), (16, 70, 4)])
def test_decode_step_example(seqs, prompt, steps):
    import decode_step
    qg.build()
    qg.qgemv_device_error(reset=True)
    a = decode_step.generate(seqs, prompt, steps, graph=False)
    b = decode_step.generate(seqs, prompt, steps, graph=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(((a[0] >= 0) & (a[0] < decode_step.VOCAB)).all()) and bool(((a[1] > 0) & (a[1] <= 1)).all())
    assert qg.qgemv_device_error() == 0
