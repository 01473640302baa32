"""GPU: the columns past a row's width are zeros, whatever stands in the row's last block."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# widths that end 1 to 8 elements into a lane's 8, with rows that start on 16 bytes and not;
# few rows and enough for eight blocks a CTA
@pytest.mark.parametrize("width", [1, 2, 3, 4, 5, 6, 7, 8, 9, 100, 127, 129, 133, 200, 1000])
@pytest.mark.parametrize("rows", [3, 33000])
@pytest.mark.parametrize("odd", [float("nan"), float("inf"), -float("inf")])
def test_padding_is_zeros(rows, width, odd):
    x = torch.randn(rows, width, device="cuda", generator=torch.Generator(device="cuda").manual_seed(width)).bfloat16()
    clean, clean_scales = w4.quantize_fp8(x)
    x[rows // 2, -1] = odd
    codes, scales = w4.quantize_fp8(x)
    bits = codes.view(torch.uint8)
    assert not bits[:, width:].any()
    # the block with it as it is documented, the others as if alone
    last = (width - 1) // 128
    value = codes[rows // 2].float()[128 * last:width]
    if odd != odd:
        assert torch.isnan(scales[last, rows // 2]) and torch.isnan(value).all()
    else:
        assert torch.isinf(scales[last, rows // 2]) and torch.isnan(value[-1]) and not value[:-1].any()
    bits[rows // 2, 128 * last:] = clean.view(torch.uint8)[rows // 2, 128 * last:]
    scales[last, rows // 2] = clean_scales[last, rows // 2]
    assert torch.equal(bits, clean.view(torch.uint8)) and torch.equal(scales, clean_scales)


def test_product_over_padded_columns():
    """The row with the NaN is NaN, every other as without it."""
    g = torch.Generator(device="cuda").manual_seed(1)
    w = w4.quantize_fp8(torch.randn(200, 256, device="cuda", generator=g).bfloat16(), blocks=True)
    dy = torch.randn(40, 200, device="cuda", generator=g).bfloat16()
    clean = w4.gemm_fp8(*w4.quantize_fp8(dy), *w, transposed=True)
    dy[7, 199] = float("nan")
    got = w4.gemm_fp8(*w4.quantize_fp8(dy), *w, transposed=True)
    assert torch.isnan(got[7]).all()
    got[7] = clean[7]
    assert torch.equal(got, clean)
