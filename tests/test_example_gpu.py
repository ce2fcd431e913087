"""The block-step example on the GPU: every output and gradient close to float32."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_step_example():
    spec = importlib.util.spec_from_file_location("block_step",
                                                  os.path.join(ROOT, "examples", "block_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    apart = example.main(["--tokens", "257", "--width", "520", "--outs", "136", "--ranks", "3"])
    assert set(apart) == {"stream", "y", "dx", "dpart", "post", "pre", "gate", "proj"}
    # Outputs are rounded to bfloat16 (half a step 2^-8 each) and activations
    # kept with 7 bits: a block's step is at most 1/64 of its largest value,
    # some 2.5 times the typical one, so that a kept value is off by a uniform
    # error of at most 1/128 of that, 2.5 / 128 / sqrt(3) = 1.1e-2 of the
    # typical value.  At most three such roundings meet in one gradient.
    for name, distance in apart.items():
        assert distance < (2.0 ** -7 if name in ("stream",) else 3 * 1.2e-2), (name, distance)
