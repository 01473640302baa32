"""GPU: sizes past 32 bits are refused by the binding of dispatch, combine and the
adapters (the wide tensor is never touched)."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_sizes_past_32_bits_are_refused():
    x = torch.zeros(4, 8, device="cuda").bfloat16()
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        w4.dispatch(x, ids, 2**32 + 2)
    wide = torch.empty(1, 2**32 + 8, device="cuda", dtype=torch.bfloat16)
    one = torch.zeros(1, 1, device="cuda", dtype=torch.int32)
    weight = torch.ones(1, 1, device="cuda")
    for call in (lambda: w4.dispatch(wide, one, 2), lambda: w4.combine(wide, one, weight),
                 lambda: w4.dispatch_backward(wide, one), lambda: w4.combine_backward(wide, wide, one, weight)):
        with pytest.raises(ValueError):
            call()
