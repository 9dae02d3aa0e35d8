"""The channel-mixing example end to end: it learns, and serves single pixels
with the weights it learned."""
import importlib.util
import os

import pytest

from helpers import torch_cuda

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mixer_block_learns_and_serves():
    torch_cuda()
    spec = importlib.util.spec_from_file_location("mixer_block", os.path.join(ROOT, "examples", "mixer_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.main(steps=20, h=40, w=30)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.6 * losses[0], losses
    # both passes round u, h and y to fp16 (half a step, 2^-11, of values below 8 here, weights of norm about 1)
    assert off <= 8 * 2.0 ** -11 * 4
