"""GPU: the 8-bit operators at the largest rows, columns and groups' rows that they take, and
captured without rows."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from fp8_model import check, codes, product, scales
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

MOST = 1 << 24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


ENDS = (slice(0, 40), slice(MOST // 2 - 20, MOST // 2 + 20), slice(MOST - 40, MOST))


def test_most_rows():
    g = gen(1)
    x, xs = codes(g, MOST, 128), scales(g, 1, MOST)
    w, ws = codes(g, 72, 128), scales(g, 1, 1)
    y = w4.gemm_fp8(x, xs, w, ws, out=torch.full((MOST, 72), float("nan"), dtype=torch.bfloat16, device="cuda"))
    for at in ENDS:
        check(y[at], *product(x[at], xs[:, at], w, ws, False))
    assert not torch.isnan(y).any()
    # the same rows by group, the last group's at the end of all
    sizes = torch.tensor([5, MOST - 12, 0, 7], dtype=torch.int32, device="cuda")
    z, status = w4.gemm_fp8_grouped(x, xs, w.repeat(4, 1, 1), ws.repeat(4, 1, 1), sizes)
    assert int(status[0]) == 0
    for at in ENDS:
        check(z[at], *product(x[at], xs[:, at], w, ws, False))


def test_most_rows_quantised():
    x = torch.randn(1 << 20, 128, device="cuda", generator=gen(2)).bfloat16()
    want = w4.quantize_fp8(x)
    c, s = w4.quantize_fp8(x.repeat(16, 1))
    for i in range(16):
        at = slice(i << 20, (i + 1) << 20)
        assert torch.equal(c[at].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s[:, at], want[1])
    # as rows of weights
    c, s = w4.quantize_fp8(x.repeat(16, 1), blocks=True)
    want = w4.quantize_fp8(x, blocks=True)
    for i in range(16):
        at = slice(i << 20, (i + 1) << 20)
        assert torch.equal(c[at].view(torch.uint8), want[0].view(torch.uint8))
        assert torch.equal(s[i << 13:(i + 1) << 13], want[1])


@pytest.mark.parametrize("M", [1, 70])
def test_most_columns(M):
    g = gen(3)
    x, xs = codes(g, M, 128), scales(g, 1, M)
    w, ws = codes(g, MOST, 128), scales(g, MOST // 128, 1)
    y = w4.gemm_fp8(x, xs, w, ws, out=torch.full((M, MOST), float("nan"), dtype=torch.bfloat16, device="cuda"))
    assert not torch.isnan(y).any()
    for at in (slice(0, 256), slice(MOST // 2 - 128, MOST // 2 + 128), slice(MOST - 256, MOST)):
        check(y[:, at], *product(x, xs, w[at], ws[at.start // 128:at.stop // 128], False))


@pytest.mark.parametrize("sizes", [[MOST], [3, MOST - 10, 7], [MOST // 2 + 1, MOST // 2 - 1]])
def test_most_rows_summed(sizes):
    """Sums of 0, 1 and -1, whole numbers up to 2^24: exact in every order."""
    g = gen(4)
    dy = torch.randint(0, 2, (MOST, 8), device="cuda", generator=g).bfloat16()
    x = torch.randint(-1, 2, (MOST, 16), device="cuda", generator=g).bfloat16()
    dy[:, 0], x[:, 0], x[:, 1] = 1.0, 1.0, -1.0
    dw, status = w4.gemm_grouped_wgrad(dy, x, torch.tensor(sizes, dtype=torch.int32, device="cuda"))
    assert int(status[0]) == 0
    row = 0
    for e, n in enumerate(sizes):
        want = dy[row:row + n].double().t() @ x[row:row + n].double()
        assert torch.equal(dw[e].double(), want)
        row += n


def test_captured_without_rows():
    """Nothing to multiply, in a graph: the status and the zeros are written at every replay."""
    f8 = torch.float8_e4m3fn
    m = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, xs = torch.empty(0, 128, device="cuda").to(f8), torch.empty(1, 0, device="cuda")
    w, ws = torch.zeros(3, 64, 128, device="cuda").to(f8), torch.ones(3, 1, 1, device="cuda")
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dw = torch.ones(3, 64, 64, device="cuda")
    status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    word = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w4.quantize_fp8(empty)
        w4.gemm_fp8(x, xs, w[0], ws[0])
        w4.gemm_fp8_grouped(x, xs, w, ws, m, status=status)
        w4.gemm_grouped_wgrad(empty, empty, m, out=dw, status=word)
    for sizes, want in (([0, 0, 0], 0), ([0, 2, 0], 2), ([-1, 0, 0], 1)):
        m.copy_(torch.tensor(sizes, dtype=torch.int32))
        dw.fill_(1.0), status.fill_(9), word.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status[0]) == want and int(word[0]) == want and not dw.any()
