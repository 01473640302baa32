"""GPU: calls of the 8-bit products and the weights' gradients at the ends of their ranges:
the most groups in every form, the longest sums, offsets past 32 bits, a weight stream that
starts before its rows are written, calls on streams at once (bounds: fp8_model)."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from fp8_model import check, codes, problem, product, scales
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# 1024 groups of about 10, 25, 50, 100 and 200 rows: every tile size, with rings of two stages
# and more; N inside a tile and past it
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,K", [(10000, 72, 384), (25000, 200, 256), (50000, 64, 640), (100000, 136, 256),
                                   (200000, 264, 384)])
def test_most_groups(M, N, K, transposed):
    E = 1024
    x, xs, w, ws = problem(gen(M), M, N, K, transposed, E)
    ids = torch.randint(0, E, (M,), generator=torch.Generator().manual_seed(M))
    ids = torch.where(ids == 5, 6, ids)                  # a group without rows
    sizes = torch.bincount(ids, minlength=E)
    starts = torch.cumsum(sizes, 0) - sizes
    out = torch.full((M, K if transposed else N), float("nan"), dtype=torch.bfloat16, device="cuda")
    y, status = w4.gemm_fp8_grouped(x, xs, w, ws, sizes.to(torch.int32).cuda(), transposed=transposed, out=out)
    assert int(status[0]) == 0 and not torch.isnan(y).any()
    for e in (0, 1, 4, 6, 31, 32, 127, 128, 500, 1000, 1023):
        rows = slice(int(starts[e]), int(starts[e] + sizes[e]))
        check(y[rows], *product(x[rows], xs[:, rows], w[e], ws[e], transposed), f"group {e}")
    # the others against the plain product of their rows, in another form perhaps
    for e in range(0, E, 101):
        rows = slice(int(starts[e]), int(starts[e] + sizes[e]))
        want, bound = product(x[rows], xs[:, rows], w[e], ws[e], transposed)
        check(w4.gemm_fp8(x[rows], xs[:, rows].contiguous(), w[e], ws[e], transposed=transposed), want, bound)


# without rows any row a size names is past the last
@pytest.mark.parametrize("sizes,want", [([0, 0], 0), ([3, 0], 2), ([0, -1], 1), ([-4, 1], 3), ([0] * 1023 + [1], 2)])
def test_status_without_rows(sizes, want):
    E = len(sizes)
    m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    x, xs, w, ws = problem(gen(0), 0, 128, 128, False, E)
    for transposed in (False, True):
        status = torch.full((4,), 9, dtype=torch.int32, device="cuda")
        assert w4.gemm_fp8_grouped(x, xs, w, ws, m, transposed=transposed, status=status)[0].shape == (0, 128)
        assert int(status[0]) == want
    empty = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dw, status = w4.gemm_grouped_wgrad(empty, empty, m, out=torch.ones(E, 64, 64, device="cuda"))
    assert not dw.any() and int(status[0]) == want


@pytest.mark.parametrize("M", [1, 30, 150])
def test_longest_sums(M):
    """2^20 summed columns, and 2^20 summed rows of the weights."""
    args = problem(gen(M), M, 8, 1 << 20, False)
    check(w4.gemm_fp8(*args), *product(*args, False))
    args = problem(gen(M), M, 1 << 20, 128, True)
    check(w4.gemm_fp8(*args, transposed=True), *product(*args, True))
    x = torch.randn(M, 1 << 20, device="cuda", generator=gen(M)).bfloat16()
    c, s = w4.quantize_fp8(x)
    back = c.float() * s.t().repeat_interleave(128, 1)
    # half a step of a code's binade, or of the smallest codes': 2^-10 of a block's scale; the
    # scale's and the products' roundings are 4 x 2^-24 of |x| < 8 at most: below 2^-19
    far = (back - x.float()).abs() - (2.0 ** -4 * x.float().abs() + 2.0 ** -10 * s.t().repeat_interleave(128, 1))
    assert float(far.max()) <= 2.0 ** -19


def test_weights_past_32_bits_of_rows():
    """Codes of rows past 2^32, in a product and in their quantisation."""
    M, K, N = 300000, 16384, 128
    g = gen(1)
    x = torch.randn(1024, K, device="cuda", generator=g).bfloat16().repeat(-(-M // 1024), 1)[:M]
    c, s = w4.quantize_fp8(x)
    first = w4.quantize_fp8(x[:1024])
    for at in (0, 261 * 1024, 262 * 1024, 292 * 1024):
        n = min(1024, M - at)
        assert torch.equal(c[at:at + n].view(torch.uint8), first[0][:n].view(torch.uint8))
        assert torch.equal(s[:, at:at + n], first[1][:, :n])
    del x
    w, ws = codes(g, N, K), scales(g, 1, K // 128)
    y = w4.gemm_fp8(c, s, w, ws)
    for rows in (slice(0, 40), slice(262100, 262200), slice(M - 40, M)):
        check(y[rows], *product(c[rows], s[:, rows], w, ws, False))


def test_gradients_past_32_bits():
    G, N, K = 70, 8192, 8192
    g = gen(2)
    dy = torch.randn(90, N, device="cuda", generator=g).bfloat16()
    x = torch.randn(90, K, device="cuda", generator=g).bfloat16()
    sizes = torch.zeros(G, dtype=torch.int32)
    sizes[[0, 63, 64, 69]] = torch.tensor([20, 30, 17, 23], dtype=torch.int32)
    out = torch.full((G, N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dw, _ = w4.gemm_grouped_wgrad(dy, x, sizes.cuda(), dtype=torch.bfloat16, out=out)
    row = 0
    for e in range(G):
        n = int(sizes[e])
        if n:
            a, b = dy[row:row + n].double(), x[row:row + n].double()
            want = a.t() @ b
            assert bool(((dw[e].double() - want).abs() <= 2.0 ** -8 * want.abs() + n * 2.0 ** -23 * (a.abs().t() @ b.abs())).all())
        else:
            assert not dw[e].any()
        row += n


# every number of rows below and past a step, each before rows that are not its own
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("down", [False, True])
def test_every_end_of_a_group(dtype, down):
    sizes, N, K = list(range(132)), 72, 264
    if down:
        sizes.reverse()
    M = sum(sizes)
    g = gen(6)
    dy = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    dw, _ = w4.gemm_grouped_wgrad(dy, x, torch.tensor(sizes, dtype=torch.int32, device="cuda"), dtype=dtype)
    row = 0
    for e, n in enumerate(sizes):
        a, b = dy[row:row + n].double(), x[row:row + n].double()
        want = a.t() @ b
        bound = n * 2.0 ** -23 * (a.abs().t() @ b.abs()) + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0)
        assert bool(((dw[e].double() - want).abs() <= bound).all()), n
        row += n


def test_long_sums_do_not_drift():
    """The tensor core cuts off at 2^-23 of a sum, 2^-24 of it on average and all one way.  Over 512
    rows (32 steps) whose sums are 512^1/2 in the end and 15 on average that is 32 x 15 x 2^-24, one
    way in a part and any in the next: 64 parts come to 64^1/2 of it, 2.3e-4, 1.3e-6 of the
    result's 32768^1/2.  Adding the parts rounds 64 times by 2^-25 of up to that: 2.4e-7."""
    M = 32768
    g = gen(8)
    dy = torch.randn(M, 256, device="cuda", generator=g).bfloat16()
    x = torch.randn(M, 256, device="cuda", generator=g).bfloat16()
    dw, _ = w4.gemm_grouped_wgrad(dy, x, torch.tensor([M], dtype=torch.int32, device="cuda"))
    want = dy.double().t() @ x.double()
    assert float((dw[0].double() - want).norm() / want.norm()) <= 1.6e-6


# pairs that share a tile's rows: groups without rows, with fewer steps than pairs, rows behind
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,M,N,K", [([5000, 0], 5000, 256, 512), ([3, 2100], 2103, 512, 264),
                                         ([2500, 100], 4000, 136, 72), ([0], 3000, 256, 256), ([65], 9000, 264, 520),
                                         ([8191], 8191, 8, 8)])
def test_shared_rows(sizes, M, N, K, dtype):
    g = gen(M + N)
    dy = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    used = sum(sizes)
    dy[used:], x[used:] = float("nan"), float("inf")     # rows no group covers
    out = torch.full((len(sizes), N, K), float("nan"), dtype=dtype, device="cuda")
    dw, status = w4.gemm_grouped_wgrad(dy, x, torch.tensor(sizes, dtype=torch.int32, device="cuda"), dtype=dtype, out=out)
    assert int(status[0]) == 0
    row = 0
    for e, n in enumerate(sizes):
        a, b = dy[row:row + n].double(), x[row:row + n].double()
        want = a.t() @ b
        bound = n * 2.0 ** -23 * (a.abs().t() @ b.abs()) + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0)
        assert bool(((dw[e].double() - want).abs() <= bound).all()), e
        row += n


@pytest.mark.parametrize("M", [1, 40, 100, 700])
def test_rows_written_right_before(M):
    """quantise -> product, with the weights' stream started early, again and again on new
    rows in the same buffers."""
    g = gen(M)
    w = (torch.randn(1000, 2560, device="cuda", generator=g) * 0.02).bfloat16()
    wq = w4.quantize_fp8(w, blocks=True)
    xs = [torch.randn(M, 2560, device="cuda", generator=g).bfloat16() for _ in range(8)]
    want = [w4.gemm_fp8(*w4.quantize_fp8(x), *wq) for x in xs]
    torch.cuda.synchronize()
    x = xs[0].clone()
    got = []
    for i in range(24):
        x.copy_(xs[i % 8])
        got.append(w4.gemm_fp8(*w4.quantize_fp8(x), *wq, resident_weights=True))
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 8]), i
    # weights written right before, without the promise
    for i in range(8):
        w.mul_(-1.0)
        y = w4.gemm_fp8(*w4.quantize_fp8(xs[0]), *w4.quantize_fp8(w, blocks=True))
        assert torch.equal(y, -want[0] if i % 2 == 0 else want[0]), i


def test_nan_stays_in_its_rows_of_a_small_product():
    for M, N, K in ((5, 260, 512), (40, 130, 2560), (100, 260, 512)):
        x, xs, w, ws = problem(gen(M), M, N, K, False)
        clean = w4.gemm_fp8(x, xs, w, ws)
        x.view(torch.uint8)[1, 3] = 0x7f
        xs[1, M - 1] = float("inf")
        y = w4.gemm_fp8(x, xs, w, ws)
        hit = torch.zeros(M, dtype=torch.bool, device="cuda")
        hit[[1, M - 1]] = True
        assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()


def test_three_streams_at_once():
    """Few rows, many rows by group and weights' gradients at the same time, each as if alone."""
    g = gen(3)
    a = problem(g, 16, 4096, 4096, False)
    b = problem(g, 3000, 1000, 1280, False, 5)
    sizes = torch.tensor([700, 0, 1100, 200, 1000], dtype=torch.int32, device="cuda")
    dy = torch.randn(3000, 520, device="cuda", generator=g).bfloat16()
    x = torch.randn(3000, 1024, device="cuda", generator=g).bfloat16()
    calls = [lambda: w4.gemm_fp8(*a), lambda: w4.gemm_fp8_grouped(*b, sizes)[0],
             lambda: w4.gemm_grouped_wgrad(dy, x, sizes)[0]]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for _ in range(15):
        for s, c, out in zip(streams, calls, got):
            with torch.cuda.stream(s):
                out.append(c())
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        for y in outs:
            assert torch.equal(y, w)


def test_a_training_step_in_a_graph():
    """Rows to experts, quantised, multiplied, back, and every gradient, captured and replayed
    on new rows and sizes."""
    g = gen(4)
    T, k, E, N, K = 200, 2, 4, 264, 384
    w = (torch.randn(E, N, K, device="cuda", generator=g) * K ** -0.5).bfloat16()
    x, dy = torch.empty(T, K, dtype=torch.bfloat16, device="cuda"), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    probs = torch.rand(T, k, device="cuda", generator=g)

    def step():
        wq, ws = w4.quantize_fp8(w, blocks=True)
        rows, sizes, slots = w4.dispatch(x, ids, E)
        ys, _ = w4.gemm_fp8_grouped(*w4.quantize_fp8(rows), wq, ws, sizes, out=torch.zeros(T * k, N, dtype=torch.bfloat16, device="cuda"))
        y = w4.combine(ys, slots, probs)
        dys, dprobs = w4.combine_backward(dy, ys, slots, probs)
        dxs, _ = w4.gemm_fp8_grouped(*w4.quantize_fp8(dys), wq, ws, sizes, transposed=True,
                                     out=torch.zeros(T * k, K, dtype=torch.bfloat16, device="cuda"))
        dw, _ = w4.gemm_grouped_wgrad(dys, rows, sizes)
        return y, dprobs, w4.dispatch_backward(dxs, slots), dw

    def fill(seed):
        s = gen(seed)
        x.copy_(torch.randn(T, K, device="cuda", generator=s))
        dy.copy_(torch.randn(T, N, device="cuda", generator=s))
        ids.copy_(torch.randint(-1, E, (T, k), device="cuda", generator=s))

    want = []
    for seed in (10, 11, 12):
        fill(seed)
        want.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for i, seed in enumerate((10, 11, 12)):
            fill(seed)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, want[i]):
                assert torch.equal(a, b)
