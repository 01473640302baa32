"""GPU: rows and weights in e4m3 against the definition in 64 bits, bit for bit.

A code is the nearest e4m3 to 448 x / max |x|, ties to even: the model divides in 64
bits, whose quotient of an 11-bit and an 8-bit number is a border between two codes
only if the exact one is (it is 2^-13 away otherwise), and rounds to the step of its
binade.  The scale is max |x| / 448 rounded to 32 bits."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def model(x, most):
    """The values of x's codes, in 64 bits."""
    x, most = x.double(), most.double()
    q = torch.where(most > 0, 448.0 * x / most, 0.0)
    step = torch.exp2((torch.frexp(q).exponent - 1).clamp(min=-6).double() - 3)
    return torch.round(q / step) * step


def model_rows(x):
    rows, width = x.shape
    x = torch.nn.functional.pad(x, (0, -width % 128)).view(rows, -1, 128)
    most = x.abs().amax(2)
    return model(x, most[..., None]).view(rows, -1), (most.double() / 448.0).float().t()


def model_blocks(w):
    rows, width = w.shape
    p = torch.nn.functional.pad(w, (0, 0, 0, -rows % 128)).view(-1, 128, width // 128, 128)
    most = p.abs().amax((1, 3))
    return model(p, most[:, None, :, None]).reshape(-1, width)[:rows], (most.double() / 448.0).float()


def spread(g, *shape):
    """Values over many binades, with zeros and repeated maxima."""
    x = torch.randn(*shape, device="cuda", generator=g) * torch.exp2(
        torch.randint(-12, 4, shape, device="cuda", generator=g).float())
    x = torch.where(torch.rand(*shape, device="cuda", generator=g) < 0.05, torch.zeros_like(x), x)
    return x.bfloat16()


def check_rows(x):
    codes, scales = w4.quantize_fp8(x)
    want, want_scales = model_rows(x)
    assert codes.shape == want.shape and codes.dtype == torch.float8_e4m3fn
    assert scales.shape == want_scales.shape and scales.is_contiguous()
    assert torch.equal(scales, want_scales)
    assert torch.equal(codes.float().double(), want)


# one row, rows beside a CTA's 16, one block a CTA and four, a last group of blocks that is
# short, widths that end inside a block or give rows no alignment
ROWS = [(1, 128), (1, 1), (16, 8192), (15, 256), (17, 640), (100, 129), (33, 1000), (1322, 2560), (4099, 4224),
        (70000, 128), (7, 9727), (2051, 4097)]


@pytest.mark.parametrize("rows,width", ROWS)
def test_rows(rows, width):
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    check_rows(spread(g, rows, width))


def test_every_quotient_of_a_binade():
    """All 128 x 128 pairs of significands, in several binades below the maximum: among them
    every tie that bf16 values can make."""
    sig = torch.arange(128, 256, device="cuda").float()
    for e in (0, -1, -5, -14, -18):
        # row m holds the maximum sig[m], then all significands
        x = sig[None, :127].expand(128, 127) * 2.0 ** e
        both = [x, sig[None, 1:].expand(128, 127) * 2.0 ** e]
        for part in both:
            part = torch.where(part.abs() > sig[:, None], part * 0.5, part)
            check_rows(torch.cat([sig[:, None], part], 1).bfloat16())
            check_rows(-torch.cat([part, sig[:, None]], 1).bfloat16())


@pytest.mark.parametrize("power", [-133, -126, -110, -64, -60, 0, 100, 120])
def test_far_magnitudes(power):
    """From the smallest subnormal to the largest finite values."""
    g = torch.Generator(device="cuda").manual_seed(power + 200)
    x = (torch.randn(64, 256, device="cuda", generator=g).clamp(-4, 4).double() * 2.0 ** power).bfloat16()
    codes, scales = w4.quantize_fp8(x)
    want, want_scales = model_rows(x)
    assert torch.equal(codes.float().double(), want)
    assert torch.equal(scales, want_scales)


def test_blocks_without_a_finite_maximum():
    x = torch.randn(6, 256, device="cuda").bfloat16()
    x[0, :128] = 0
    x[1, 5] = float("inf")
    x[2, 5] = -float("inf")
    x[3, 5] = float("nan")
    x[4] = -0.0
    codes, scales = w4.quantize_fp8(x)
    value = codes.float()
    assert scales[0, 0] == 0 and not value[0, :128].any()
    assert scales[0, 4] == 0 and scales[1, 4] == 0 and not value[4].any()
    for row in (1, 2):
        assert torch.isinf(scales[0, row]) and torch.isnan(value[row, 5])
        others = torch.arange(128, device="cuda") != 5
        assert not value[row, :128][others].any()
    assert torch.isnan(scales[0, 3]) and torch.isnan(value[3, :128]).all()
    # their neighbours are as if alone
    rest = w4.quantize_fp8(x[:, 128:].contiguous())
    assert torch.equal(rest[0].float(), value[:, 128:]) and torch.equal(rest[1], scales[1:])


def test_rows_that_start_anywhere():
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = spread(g, 1, 300 * 264 + 8)[0]
    for start in range(0, 8):
        check_rows(flat[start:start + 300 * 264].view(300, 264))


@pytest.mark.parametrize("lead,rows,width", [((), 128, 128), ((), 1, 128), ((), 300, 1280), ((), 129, 2560),
                                             ((3,), 200, 384), ((1,), 1000, 640), ((64,), 5, 128)])
def test_weights(lead, rows, width):
    g = torch.Generator(device="cuda").manual_seed(rows + width)
    w = spread(g, *lead, rows, width)
    codes, scales = w4.quantize_fp8(w, blocks=True)
    assert codes.shape == w.shape and scales.shape == (*lead, -(-rows // 128), width // 128)
    for c, s, one in zip(codes.view(-1, rows, width), scales.view(-1, *scales.shape[-2:]), w.view(-1, rows, width)):
        want, want_scales = model_blocks(one)
        assert torch.equal(c.float().double(), want) and torch.equal(s, want_scales)


def test_weights_with_odd_blocks():
    w = torch.randn(256, 384, device="cuda").bfloat16()
    w[:128, :128] = 0
    w[130, 130] = float("nan")
    w[3, 300] = float("inf")
    codes, scales = w4.quantize_fp8(w, blocks=True)
    v = codes.float()
    assert scales[0, 0] == 0 and not v[:128, :128].any()
    assert torch.isnan(scales[1, 1]) and torch.isnan(v[128:, 128:256]).all()
    assert torch.isinf(scales[0, 2]) and torch.isnan(v[3, 300]) and int(torch.isnan(v[:128, 256:]).sum()) == 1
    assert not torch.isnan(v[128:, :128]).any()


def test_no_rows():
    codes, scales = w4.quantize_fp8(torch.empty(0, 300, dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 384) and scales.shape == (3, 0)


def test_captured_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(9)
    x, w = spread(g, 33, 640), spread(g, 200, 640)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        w4.quantize_fp8(x)
        w4.quantize_fp8(w, blocks=True)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        rows, blocks = w4.quantize_fp8(x), w4.quantize_fp8(w, blocks=True)
    for seed in (1, 2):
        x.copy_(spread(torch.Generator(device="cuda").manual_seed(seed), 33, 640))
        graph.replay()
        torch.cuda.synchronize()
        want = model_rows(x)
        assert torch.equal(rows[0].float().double(), want[0]) and torch.equal(rows[1], want[1])
        want = model_blocks(w)
        assert torch.equal(blocks[0].float().double(), want[0]) and torch.equal(blocks[1], want[1])
