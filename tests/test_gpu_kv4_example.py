"""The decode example over the 4-bit cache runs and agrees with float64."""

import runpy
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [1, 64])
def test_kv4_decode_example(cuda_device, steps):
    run = runpy.run_path(str(Path(__file__).parent.parent / "examples" / "kv4_decode_step.py"))["run"]
    # BF16 output (2^-9) and probabilities with 8 bits: below 2^-7 of the largest
    assert run(steps=steps) < 2.0 ** -7
