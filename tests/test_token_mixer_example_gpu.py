"""examples/token_mixer.py on the GPU: prompts continued token by token agree with one pass over
everything, and gradient descent through the backward calls lowers the loss."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "token_mixer.py")
    spec = importlib.util.spec_from_file_location("token_mixer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_single_tokens_continue_the_prompts():
    # four blocks in bf16: each adds a few roundings (2^-8) of its own in either path, and the chunked
    # delta rule keeps its operands in bf16; independent errors of eight roundings per block
    assert _example().serve() < 2.0 ** -8 * math.sqrt(4 * 8)


def test_training_lowers_the_loss():
    losses = _example().train(steps=20)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.9 * losses[0]
