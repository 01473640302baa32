"""GPU: scales at both ends of what the 8-bit products allow: a row's times a weight block's
is a normal fp32 number, or 0 because one of them is.

A block's sum is 0 or between 2^-18 and 2^25 in magnitude.  Bounds: those of fp8_model;
below 2^-126 every one of B additions rounds by at most 2^-150 more and the result by
2^-134."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from fp8_model import check, codes, product, scales
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum(k * 31 ** i for i, k in enumerate(key)) % 2**31)


# few rows: tiles of 16, 32, 64 and 128, alone and shared by a cluster; many: pairs, clusters, alone
SHAPES = [(5, 260, 512), (30, 261, 1024), (60, 1000, 2560), (700, 1000, 2560), (512, 2560, 9728), (100, 264, 640),
          (330, 9001, 1280), (800, 600, 20480), (1, 4096, 8192), (16, 3, 128)]


def times_power(xs, power):
    """xs 2^power, formed in 64 bits."""
    return (xs.double() * torch.exp2(power.double())).float()


def operands(g, M, N, K, transposed, lead):
    C = -(-N // 128) * 128 if transposed else K
    return C, codes(g, M, C), codes(g, *lead, N, K), scales(g, C // 128, M), scales(g, *lead, -(-N // 128), K // 128)


def small(g, M, N, K, transposed, lead=()):
    """Products of scales from 2^-126 to 2^-118, ordinary ones and 0."""
    C, x, w, xs, ws = operands(g, M, N, K, transposed, lead)
    power = torch.tensor([-55, 55, -55], device="cuda").repeat(-(-M // 3))[:M]
    xs = times_power(xs, power)
    xs[:, 2::3] = 0.0
    return x, xs, w, ws * 2.0 ** -55


def large(g, M, N, K, transposed, lead=()):
    """Products of scales from 2^120 to 2^128 under sums that bring the results back, and under
    sums of zeros."""
    C, x, w, xs, ws = operands(g, M, N, K, transposed, lead)
    # one element of 2^-9 a block, weights up to 7 x 2^-9: sums up to 2^-15.1, 160 of them 2^-7.8
    x = torch.zeros(M, C // 128, 128, dtype=torch.uint8, device="cuda")
    at = torch.randint(0, 128, (M, C // 128, 1), device="cuda", generator=g)
    x.scatter_(2, at, torch.randint(0, 2, at.shape, device="cuda", generator=g).to(torch.uint8) * 0x80 + 1)
    x = x.view(M, C)
    x[2::3] = 0
    w = (w.view(torch.uint8) & 0x87).view(torch.float8_e4m3fn)
    power = torch.tensor([68, -60, 68], device="cuda").repeat(-(-M // 3))[:M]
    return x.view(torch.float8_e4m3fn), times_power(xs, power), w, times_power(ws, torch.tensor(68, device="cuda"))


def compare(got, args, transposed):
    xs, ws = args[1].double(), args[3].double()
    assert float(xs[xs > 0].min() * ws.min()) >= 2.0 ** -126 and float(xs.max() * ws.max()) < 2.0 ** 128
    want, bound = product(*args, transposed)
    blocks = xs.shape[0]
    check(got, want, bound + blocks * 2.0 ** -149 + 2.0 ** -134)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("make", [small, large])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_ends_of_the_range(M, N, K, make, transposed):
    args = make(gen(M, N, K, transposed), M, N, K, transposed)
    got = w4.gemm_fp8(*args, transposed=transposed)
    compare(got, args, transposed)
    assert not got[2::3].any()                           # zero scales, sums of zeros


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("make", [small, large])
@pytest.mark.parametrize("sizes,N,K", [([3, 0, 9, 4], 264, 2560), ([100, 0, 0, 40], 520, 9728), ([700, 300, 5], 1000, 640)])
def test_ends_of_the_range_by_group(sizes, N, K, make, transposed):
    M, E = sum(sizes), len(sizes)
    x, xs, w, ws = make(gen(M, N, K, transposed), M, N, K, transposed, (E,))
    m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    y, _ = w4.gemm_fp8_grouped(x, xs, w, ws, m, transposed=transposed)
    row = 0
    for e, n in enumerate(sizes):
        if n:
            at = slice(row, row + n)
            compare(y[at], (x[at], xs[:, at], w[e], ws[e]), transposed)
        row += n


def test_magnitudes_that_the_quantiser_keeps_in_the_range():
    """Both sides' largest magnitudes at 2^-54, and just below 2^72."""
    g = gen(1)
    for power in (-54, 71):
        x = torch.randint(-128, 129, (40, 512), device="cuda", generator=g).double() / 128
        w = torch.randint(-128, 129, (264, 512), device="cuda", generator=g).double() / 128
        most = 1.0 if power < 0 else 255 / 128
        x[:, ::128], w[:, ::128] = most, -most           # the largest, in every block
        x, w = ((v * 2.0 ** power).bfloat16() for v in (x, w))
        xq, wq = w4.quantize_fp8(x), w4.quantize_fp8(w, blocks=True)
        products = xq[1].double().amin() * wq[1].double().amin(), xq[1].double().amax() * wq[1].double().amax()
        assert 2.0 ** -126 <= float(products[0]) and float(products[1]) < 2.0 ** 128
        got = w4.gemm_fp8(*xq, *wq)
        want, bound = product(*xq, *wq, False)
        if power < 0:
            check(got, want, bound + 4 * 2.0 ** -149 + 2.0 ** -134)
        else:
            # results past bf16's largest are infinite
            fits = want.abs() < 2.0 ** 127
            assert bool(((got.double() - want).abs() <= bound)[fits].all())


def test_scales_that_are_not_finite_or_zero():
    """An infinite or NaN scale makes its row so, a zero one makes zeros."""
    for M, N, K in ((20, 260, 512), (300, 260, 512)):
        g = gen(M)
        x, xs, w, ws = codes(g, M, K), scales(g, K // 128, M), codes(g, N, K), scales(g, 3, K // 128)
        clean = w4.gemm_fp8(x, xs, w, ws)
        xs[0, 3], xs[1, 7], xs[:, 9] = float("inf"), float("nan"), 0.0
        got = w4.gemm_fp8(x, xs, w, ws)
        assert not torch.isfinite(got[3]).any() and torch.isnan(got[7]).all() and not got[9].any()
        rest = torch.ones(M, dtype=torch.bool, device="cuda")
        rest[[3, 7, 9]] = False
        assert torch.equal(got[rest], clean[rest])
