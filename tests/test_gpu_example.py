"""The example's blocks: a prompt and single tokens give what the whole sequence gives at once."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "hybrid_blocks.py")
    spec = importlib.util.spec_from_file_location("hybrid_blocks", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("prompt,new", [(90, 7), (3, 30), (1, 1)])
def test_steps_equal_the_whole(prompt, new):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    steps, whole = load().run(prompt, new)
    assert bool(torch.isfinite(whole).all())
    # Both ways differ by fp32 roundings, which now and then move a value over a border of the 8-bit quantization (half a
    # step of 1/127 of its block's largest value).  Four products, were every value of each moved by a whole step:
    assert float((steps - whole).norm() / whole.norm()) < 4 / 127
