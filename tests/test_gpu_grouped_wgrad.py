"""GPU: gradients of the weights of a product by group against 64 bits.

A product of two bf16 values is exact in fp32; a sum of n of them, rounded or cut at
every step, is off by at most n * 2^-23 of the sum of their magnitudes; a bf16 result is
rounded once more, 2^-8 of it."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rows(g, M, N, K):
    return (torch.randn(M, N, device="cuda", generator=g).bfloat16(),
            torch.randn(M, K, device="cuda", generator=g).bfloat16())


def check(dy, x, sizes, dtype, status=0):
    M, N = dy.shape
    out = torch.full((len(sizes), N, x.shape[1]), float("nan"), dtype=dtype, device="cuda")
    got, word = w4.gemm_grouped_wgrad(dy, x, torch.tensor(sizes, dtype=torch.int32, device="cuda"), dtype=dtype,
                                      out=out)
    assert got is out and int(word[0]) == status
    row = 0
    for e, n in enumerate(sizes):
        n = max(0, min(n, M - row))
        a, b = dy[row:row + n].double(), x[row:row + n].double()
        want = a.t() @ b
        bound = n * 2.0 ** -23 * (a.abs().t() @ b.abs())
        if dtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * want.abs()
        err = (got[e].double() - want).abs()
        assert bool((err <= bound).all()), (e, n, float((err - bound).max()))
        row += n
    return got


# groups that end inside a step of 16, of 64, on both; empty ones; N and K inside a box, past
# it, inside a tile and past it; more tiles than SMs
SHAPES = [([1], 8, 8), ([64], 128, 256), ([15], 64, 64), ([16, 17, 63, 65], 136, 264), ([0, 5, 0], 40, 72),
          ([128, 0, 1, 300], 200, 512), ([1000], 520, 1000), ([77, 200], 1024, 2560), ([33] * 40, 128, 128),
          ([4096], 256, 384), ([0, 0], 64, 128)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_wgrad(sizes, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(sizes) + N + K)
    check(*rows(g, max(1, sum(sizes)), N, K), sizes, dtype)


def test_many_groups():
    g = torch.Generator(device="cuda").manual_seed(1)
    sizes = torch.randint(0, 9, (1024,), generator=torch.Generator().manual_seed(1)).tolist()
    check(*rows(g, sum(sizes), 72, 136), sizes, torch.float32)


@pytest.mark.parametrize("sizes,status", [([10, -5, 20], 1), ([30, 30, 30], 2), ([70, 0, -1], 3)])
def test_sizes_that_do_not_fit(sizes, status):
    g = torch.Generator(device="cuda").manual_seed(2)
    check(*rows(g, 50, 64, 72), sizes, torch.float32, status)


def test_rows_of_others_do_not_enter():
    """NaN and infinity in the rows of other groups and behind the last: none of them is
    multiplied, not even by zero."""
    g = torch.Generator(device="cuda").manual_seed(3)
    for first in (1, 15, 17, 63, 64, 70, 127):
        dy, x = rows(g, first + 90, 136, 264)
        dy[first:first + 40] = float("nan")
        x[first:first + 40] = float("inf")
        dy[first + 60:] = float("inf")
        x[first + 60:] = float("nan")
        sizes = torch.tensor([first, 40, 20], dtype=torch.int32, device="cuda")
        dw, _ = w4.gemm_grouped_wgrad(dy, x, sizes)
        for e, at in ((0, slice(0, first)), (2, slice(first + 40, first + 60))):
            want = dy[at].double().t() @ x[at].double()
            bound = 100 * 2.0 ** -23 * (dy[at].double().abs().t() @ x[at].double().abs())
            assert bool(((dw[e].double() - want).abs() <= bound).all())
        assert torch.isnan(dw[1]).all()


def test_against_differences():
    """<dw, d> is the change of <dy, x (w + d)^T>, which is linear in d."""
    g = torch.Generator(device="cuda").manual_seed(4)
    dy, x = rows(g, 90, 72, 128)
    sizes = torch.tensor([50, 40], dtype=torch.int32, device="cuda")
    dw = w4.gemm_grouped_wgrad(dy, x, sizes)[0].double()
    for _ in range(3):
        d = torch.randn(2, 72, 128, device="cuda", generator=g).double()
        y = torch.cat([x[:50].double() @ d[0].t(), x[50:].double() @ d[1].t()])
        change = (dy.double() * y).sum()
        slack = 90 * 2.0 ** -23 * (dy.double().abs() * torch.cat(
            [x[:50].double().abs() @ d[0].abs().t(), x[50:].double().abs() @ d[1].abs().t()])).sum()
        assert abs((dw * d).sum() - change) <= slack


def test_no_rows():
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    sizes = torch.zeros(2, dtype=torch.int32, device="cuda")
    dw, status = w4.gemm_grouped_wgrad(empty, empty, sizes, out=torch.ones(2, 64, 64, device="cuda"))
    assert not dw.any() and int(status[0]) == 0


def test_captured_with_new_sizes_and_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(5)
    dy, x = rows(g, 300, 136, 264)
    sizes = torch.tensor([300, 0, 0], dtype=torch.int32, device="cuda")
    want = {}
    news = ([300, 0, 0], [100, 100, 100], [1, 0, 299])
    for new in news:
        want[tuple(new)] = check(dy, x, new, torch.float32).clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        dw, _ = w4.gemm_grouped_wgrad(dy, x, sizes)
    for new in news:
        sizes.copy_(torch.tensor(new, dtype=torch.int32))
        dw.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want[tuple(new)])


def test_results_do_not_depend_on_timing():
    g = torch.Generator(device="cuda").manual_seed(6)
    dy, x = rows(g, 2000, 512, 1024)
    sizes = torch.tensor([700, 1300], dtype=torch.int32, device="cuda")
    first = w4.gemm_grouped_wgrad(dy, x, sizes)[0]
    for _ in range(20):
        assert torch.equal(w4.gemm_grouped_wgrad(dy, x, sizes)[0], first)
