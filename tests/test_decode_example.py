"""The decoding example: the low-bit operators together, as one layer's steps
recorded in a CUDA graph, against the same step in float32."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("batch,steps", [(1, 3), (8, 40)])
def test_decode_step(libgemm, batch, steps):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # bfloat16 results of bfloat16 queries: roundings of 2^-9 on average at the
    # projection, the attention's result and the output
    assert example.main(batch, steps) < 3 * 2.0 ** -8
