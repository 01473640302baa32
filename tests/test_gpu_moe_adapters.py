"""GPU: the example's mixture-of-experts block, which runs dispatch, combine and the
adapters with their gradients beside the W4A16 products.

Bounds on the relative (Frobenius) errors, from the roundings to bf16 (at most 2^-8
each): h has two; gate and up one more, and silu(gate) * up carries both sides'
errors; the product, z and down one each; y one; the router's probabilities carry
about one.  With the product counted twice: 2 * 3 + 1 + 1 + 1 + 1 = 10.  The
gradients pass the same stages once more on the way back: 20.  The router's gradient
is a difference of products <dy, ys> that nearly cancel, for which no such count
holds: an error below 0.5 says that its direction is right to 30 degrees."""
from __future__ import annotations

import os
import sys

import pytest
import torch

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    import moe_adapters
    return moe_adapters


@pytest.mark.parametrize("tokens", [1, 5, 64, 700])
@torch.no_grad()
def test_block_against_64_bits(example, tokens):
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    y, a, b, router = example.step_errors(tokens, example.Block(seed=tokens), gen)
    assert y <= 10 * 2.0**-8
    if tokens > 1:
        assert max(a, b) <= 20 * 2.0**-8
        assert router < 0.5


@torch.no_grad()
def test_training_lowers_the_loss(example):
    losses = example.train(example.Block(), gen=torch.Generator(device="cuda").manual_seed(1))
    assert losses[-1] < losses[0], losses
