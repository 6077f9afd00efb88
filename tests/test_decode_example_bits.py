"""The decoding example over a cache of 4 bits."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
@pytest.mark.parametrize("batch,steps", [(1, 3), (8, 40)])
def test_decode_step_over_4_bits(libgemm, batch, steps):
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # the same roundings as over 8 bits: the comparison reads the cache's values back
    assert example.main(batch, steps, bits=4) < 3 * 2.0 ** -8
