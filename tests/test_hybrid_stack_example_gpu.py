"""examples/hybrid_stack.py on the GPU: recurrent and attention blocks run together, prompts continued token by token or
several tokens at a time agree with one pass over everything; gradients through the norms of queries and keys
agree with 64-bit ones."""

from __future__ import annotations

import importlib.util
import math
import os

import pytest
import torch

import attention_reference as aref

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_stack.py")
    spec = importlib.util.spec_from_file_location("hybrid_stack", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


# Four blocks in bf16: each adds about eight roundings (2^-8) of its own in either path. With an 8-bit cache an input that
# differs by a rounding of bf16 may be stored a step apart (2^-3 of the value at most, one value in about 2^4 of
# them, since bf16 has 2^4 numbers in a step): 2^-3 2^-2 over the values, weighted sums over keys make it smaller.
@pytest.mark.parametrize("kind,tol", [(torch.bfloat16, 2.0 ** -8 * math.sqrt(4 * 8)), (torch.float8_e4m3fn, 2.0 ** -5 + 2.0 ** -8 * math.sqrt(4 * 8))])
@pytest.mark.parametrize("extra,at_once", [(5, 1), (8, 4), (7, 3)])
def test_tokens_continue_the_prompts(kind, tol, extra, at_once):
    assert _example().serve(kind=kind, extra=extra, at_once=at_once) < tol


def test_gradients():
    ex = _example()
    args, target, got = ex.gradients()
    leaves = [t.double().requires_grad_() for t in args]
    pos = torch.arange(target.shape[1]).repeat(target.shape[0])

    def norm(q, k, a, b):
        turn = lambda x, w: aref.norm_rope(x.flatten(0, 1), w, pos, aref.inv_freq(ex.ROTATED), 1e-6, False).reshape(x.shape)  # noqa: E731
        return turn(q, a), turn(k, b)

    want = torch.autograd.grad(ex.loss(*leaves, target.double(), norm), leaves)
    for x, y in zip(got, want):
        # 32-bit attention and softmax around the norms: about sqrt(64) 2^-24 a product, five in a row
        assert float((x.double().cpu() - y).norm() / y.norm()) < 2.0 ** -17
