"""GPU: products of 8-bit rows and weights, plain and by group, and the gradients of
their rows, against 64 bits (fp8_model has the bounds)."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from fp8_model import check, codes, dense_weights, problem, product, scales
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum(k * 31 ** i for i, k in enumerate(key)) % 2**31)


def poisoned(M, cols):
    return torch.full((M, cols), float("nan"), dtype=torch.bfloat16, device="cuda")


# rows: one, the borders of every tile size, ragged ones; N: one column, inside a tile, past
# it, odd; K: one block, few, many (split over a cluster)
SHAPES = [(1, 1, 128), (1, 8192, 8192), (1, 130, 4096), (2, 7, 256), (15, 128, 640), (16, 256, 1280), (17, 264, 384),
          (32, 1000, 2560), (33, 511, 1024), (61, 2560, 5120), (64, 128, 9728), (65, 640, 512), (100, 333, 2048),
          (128, 1024, 1024), (129, 128, 128), (130, 2568, 640), (250, 777, 384), (256, 512, 2560), (257, 1152, 256),
          (513, 392, 1152), (700, 2560, 2560), (1322, 1000, 896), (2858, 2049, 512)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, transposed):
    args = problem(gen(M, N, K, transposed), M, N, K, transposed)
    out = poisoned(M, K if transposed else N)
    got = w4.gemm_fp8(*args, transposed=transposed, out=out)
    assert got is out
    check(got, *product(*args, transposed), f"{M}x{N}x{K}")
    assert torch.equal(w4.gemm_fp8(*args, transposed=transposed, resident_weights=True), got)


@pytest.mark.parametrize("M", [1, 40, 128, 300])
def test_quantised_inputs(M):
    """What a caller does: quantise both sides, multiply, and back."""
    g = gen(M)
    x = torch.randn(M, 1280, device="cuda", generator=g).bfloat16()
    w = (torch.randn(1000, 1280, device="cuda", generator=g) * 0.03).bfloat16()
    dy = torch.randn(M, 1000, device="cuda", generator=g).bfloat16()
    wq = w4.quantize_fp8(w, blocks=True)
    xq, dq = w4.quantize_fp8(x), w4.quantize_fp8(dy)
    check(w4.gemm_fp8(*xq, *wq), *product(*xq, *wq, False))
    check(w4.gemm_fp8(*dq, *wq, transposed=True), *product(*dq, *wq, True))
    # against the unquantised product: both sides off by at most 2^-4 of an element (or half
    # the smallest step, 2^-10 of 448, of the block's largest)
    want = x.double() @ w.double().t()
    far = (w4.gemm_fp8(*xq, *wq).double() - want).norm() / want.norm()
    assert far < 2 * 2.0 ** -4


def test_row_gradient_against_differences():
    """The transposed product is the gradient of the product: <dy, Y(x + d) - Y(x)> for
    representable steps d, whose results differ by the roundings of both calls alone."""
    g = gen(5)
    M, N, K = 20, 300, 384
    x, xs, w, ws = problem(g, M, N, K, False)
    dy, ds = codes(g, M, 384), scales(g, 3, M)
    dx = w4.gemm_fp8(dy, ds, w, ws, transposed=True).double()
    d = dy.double() * ds.double().t().repeat_interleave(128, 1)
    y0, b0 = product(x, xs, w, ws, False)
    for seed in range(3):
        other = codes(gen(seed, 77), M, K)
        y1, b1 = product(other, xs, w, ws, False)
        step = (other.double() - x.double()) * xs.double().t().repeat_interleave(128, 1)
        got0, got1 = (w4.gemm_fp8(v, xs, w, ws).double() for v in (x, other))
        lhs = (d[:, :N] * (got1 - got0)).sum()
        _, bx = product(dy, ds, w, ws, True)
        slack = (d[:, :N].abs() * (b0 + b1)).sum() + (step.abs() * bx).sum()
        assert abs(lhs - (dx * step).sum()) <= slack


def test_padding_columns_do_not_enter():
    """Transposed, the columns of x past N meet rows that are not the weights'."""
    M, N, K = 50, 200, 256
    for groups in (None, 3):
        args = problem(gen(1), M, N, K, True, groups)
        sizes = torch.tensor([20, 0, 30], dtype=torch.int32, device="cuda")
        call = (lambda a: w4.gemm_fp8(*a, transposed=True)) if groups is None else \
            (lambda a: w4.gemm_fp8_grouped(*a, sizes, transposed=True)[0])
        first = call(args)
        other = args[0].clone()
        other.view(torch.uint8)[:, N:] = 0x7e                        # 448
        assert torch.equal(call((other,) + args[1:]), first)


def test_nan_and_infinity_stay_in_their_rows():
    M, N, K = 300, 260, 512
    x, xs, w, ws = problem(gen(2), M, N, K, False)
    clean = w4.gemm_fp8(x, xs, w, ws)
    x.view(torch.uint8)[17, 3] = 0x7f
    xs[1, 200] = float("inf")
    xs[2, 299] = float("nan")
    y = w4.gemm_fp8(x, xs, w, ws)
    hit = torch.zeros(M, dtype=torch.bool, device="cuda")
    hit[[17, 200, 299]] = True
    assert torch.equal(y[~hit], clean[~hit])
    assert not torch.isfinite(y[hit]).any()
    # a NaN of the weights: its column alone
    x, xs, w, ws = problem(gen(2), M, N, K, False)
    w.view(torch.uint8)[131, 5] = 0x7f
    y = w4.gemm_fp8(x, xs, w, ws)
    assert torch.isnan(y[:, 131]).all()
    y[:, 131] = clean[:, 131]
    assert torch.equal(y, clean)


def test_zero_scales():
    x, xs, w, ws = problem(gen(3), 5, 140, 256, False)
    assert not w4.gemm_fp8(x, torch.zeros_like(xs), w, ws).any()
    assert not w4.gemm_fp8(x, xs, w, torch.zeros_like(ws)).any()


def test_far_scales():
    """Scales whose product leaves fp32 only together with the result."""
    x, xs, w, ws = problem(gen(4), 33, 300, 1280, False)
    args = (x, xs * 2.0 ** -60, w, ws * 2.0 ** 50)
    check(w4.gemm_fp8(*args), *product(*args, False))


def test_unaligned_results():
    """Rows of Y that start on 2 bytes."""
    M, N, K = 40, 264, 256
    args = problem(gen(6), M, N, K, False)
    want = w4.gemm_fp8(*args)
    flat = torch.zeros(M * N + 16, dtype=torch.bfloat16, device="cuda")
    for start in (1, 2, 8):
        flat.zero_()
        assert torch.equal(w4.gemm_fp8(*args, out=flat[start:start + M * N].view(M, N)), want)
        assert not flat[:start].any() and not flat[start + M * N:].any()


def test_no_rows():
    x, xs, w, ws = problem(gen(7), 0, 100, 256, False)
    assert w4.gemm_fp8(x, xs, w, ws).shape == (0, 100)
    w3, ws3 = w[None], ws[None]
    y, status = w4.gemm_fp8_grouped(x, xs, w3, ws3, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 100) and int(status[0]) == 0


# ------------------------------------------------------------------ by group
def group_sizes(g, kind, groups, M):
    if kind == "even":
        s = [M // groups] * groups
        s[0] += M - sum(s)
    elif kind == "one":
        s = [0] * groups
        s[groups // 2] = M
    elif kind == "none":
        s = [0] * groups
    else:
        ids = torch.randint(0, groups, (M,), generator=g)
        if kind == "skew":
            ids = torch.where(torch.rand(M, generator=g) < 0.7, ids // 4, ids)
        s = torch.bincount(ids, minlength=groups).tolist()
        if kind == "short":                              # rows behind the last group
            s[-1] = 0
    return s


def check_grouped(args, sizes, transposed, M, cols, status=0):
    x, xs, w, ws = args
    out = poisoned(M, cols)
    got, word = w4.gemm_fp8_grouped(*args, torch.tensor(sizes, dtype=torch.int32, device="cuda"),
                                    transposed=transposed, out=out)
    assert int(word[0]) == status
    row = 0
    for e, n in enumerate(sizes):
        n = max(0, min(n, M - row))
        if n:
            check(got[row:row + n], *product(x[row:row + n], xs[:, row:row + n], w[e], ws[e], transposed), f"group {e}")
        row += n
    assert torch.isnan(got[row:]).all()                  # left as they were
    return got


GROUPED = [(1, 1, 128, 128), (8, 128, 256, 512), (128, 128, 200, 256), (40, 3, 1000, 640), (300, 8, 264, 384),
           (1000, 5, 130, 256), (3000, 4, 392, 512), (5000, 33, 128, 1152), (64, 1024, 64, 128), (4096, 8, 520, 640)]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kind", ["even", "one", "none", "random", "skew", "short"])
@pytest.mark.parametrize("M,groups,N,K", GROUPED)
def test_grouped(M, groups, N, K, kind, transposed):
    g = gen(M, groups, N, K)
    sizes = group_sizes(torch.Generator().manual_seed(M + groups), kind, groups, M)
    check_grouped(problem(g, M, N, K, transposed, groups), sizes, transposed, M, K if transposed else N)


@pytest.mark.parametrize("sizes,status", [([10, -5, 20], 1), ([30, 30, 30], 2), ([70, 0, -1], 3), ([50, 1, 1], 2),
                                          ([2**31 - 1, 2**31 - 1, 5], 2)])
def test_sizes_that_do_not_fit(sizes, status):
    check_grouped(problem(gen(8), 50, 130, 256, False, 3), sizes, False, 50, 130, status)


def test_a_group_is_the_plain_product():
    M, N, K = 300, 264, 640
    x, xs, w, ws = problem(gen(9), M, N, K, False, 2)
    sizes = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    a = w4.gemm_fp8_grouped(x, xs, w, ws, sizes)[0]
    check(a, *product(x, xs, w[1], ws[1], False))


def test_dispatched_rows_through_experts_and_back():
    """dispatch -> quantise -> product -> combine, and the gradient on the way back."""
    g = gen(10)
    T, k, E, N, K = 70, 3, 5, 200, 256
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    w = (torch.randn(E, N, K, device="cuda", generator=g) * K ** -0.5).bfloat16()
    ids = torch.randint(-1, E, (T, k), device="cuda", dtype=torch.int32, generator=g)
    probs = torch.rand(T, k, device="cuda", generator=g)
    wq, ws = w4.quantize_fp8(w, blocks=True)
    rows, sizes, slots = w4.dispatch(x, ids, E)
    ys, status = w4.gemm_fp8_grouped(*w4.quantize_fp8(rows), wq, ws, sizes)
    y = w4.combine(ys, slots, probs)
    assert int(status[0]) == 0
    dense = [dense_weights(wq[e], ws[e]) for e in range(E)]
    want = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        mine = torch.where(ids == e, probs.double(), 0.0).sum(1, keepdim=True)
        want += mine * (x.double() @ dense[e].t())
    # rows off by at most 2^-4 of an element, two roundings to bf16
    assert (y.double() - want).norm() < (2.0 ** -4 + 2 * 2.0 ** -8) * want.norm()
    dy = torch.randn(T, N, device="cuda", generator=g).bfloat16()
    dys, _ = w4.combine_backward(dy, ys, slots, probs)
    dxs, _ = w4.gemm_fp8_grouped(*w4.quantize_fp8(dys), wq, ws, sizes, transposed=True)
    kept = int(sizes.sum())
    dxs[kept:] = 0
    dx = w4.dispatch_backward(dxs, slots)
    dw, _ = w4.gemm_grouped_wgrad(dys, rows, sizes)
    want_dx = torch.zeros(T, K, dtype=torch.float64, device="cuda")
    want_dw = torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        mine = torch.where(ids == e, probs.double(), 0.0).sum(1, keepdim=True) * dy.double()
        want_dx += mine @ dense[e]
        want_dw[e] = mine.t() @ x.double()
    assert (dx.double() - want_dx).norm() < (2.0 ** -4 + 4 * 2.0 ** -8) * want_dx.norm()
    assert (dw.double() - want_dw).norm() < 2 * 2.0 ** -8 * want_dw.norm()


# -------------------------------------------------------- streams and graphs
def test_captured_with_new_sizes():
    g = gen(11)
    M, N, K, E = 200, 264, 512, 4
    args = problem(g, M, N, K, False, E)
    plain = problem(g, 30, N, K, False)
    sizes = torch.tensor([200, 0, 0, 0], dtype=torch.int32, device="cuda")
    w4.gemm_fp8_grouped(*args, sizes)
    w4.gemm_fp8(*plain)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, status = w4.gemm_fp8_grouped(*args, sizes)
        z = w4.gemm_fp8(*plain, resident_weights=True)
    for new in ([200, 0, 0, 0], [50, 50, 50, 50], [0, 1, 0, 199], [7, 100, 3, 0]):
        sizes.copy_(torch.tensor(new, dtype=torch.int32))
        plain[0].copy_(codes(gen(*new), 30, K))
        y.fill_(float("nan")), z.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert int(status[0]) == 0
        row = 0
        for e, n in enumerate(new):
            if n:
                check(y[row:row + n], *product(args[0][row:row + n], args[1][:, row:row + n], args[2][e], args[3][e], False))
            row += n
        assert torch.isnan(y[row:]).all()
        check(z, *product(*plain, False))


def test_two_streams_at_once():
    g = gen(12)
    a, b = problem(g, 61, 2560, 2560, False), problem(g, 700, 1000, 1280, False)
    want_a, want_b = w4.gemm_fp8(*a), w4.gemm_fp8(*b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(10):
        for s, args in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(w4.gemm_fp8(*args))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want_b if i % 2 else want_a)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (61, 2560, 5120), (1322, 1024, 1024)])
def test_results_do_not_depend_on_timing(M, N, K):
    args = problem(gen(M, 3), M, N, K, False)
    first = w4.gemm_fp8(*args)
    for _ in range(20):
        assert torch.equal(w4.gemm_fp8(*args), first)


def test_offsets_past_32_bits():
    """More than 2^32 elements of weights, and of results."""
    N, K, E = 8192, 8192, 66
    g = gen(13)
    w = codes(g, N, K).repeat(E, 1, 1)
    ws = scales(g, E, N // 128, K // 128)
    x, xs = codes(g, 40, K), scales(g, K // 128, 40)
    sizes = torch.zeros(E, dtype=torch.int32)
    sizes[[0, 63, 64, 65]] = 10
    y, _ = w4.gemm_fp8_grouped(x, xs, w, ws, sizes.cuda())
    for i, e in enumerate((0, 63, 64, 65)):
        rows = slice(10 * i, 10 * i + 10)
        check(y[rows], *product(x[rows], xs[:, rows], w[e], ws[e], False), f"group {e}")
    del w
    M, N, K = 300000, 16384, 128
    x, xs, w, ws = problem(g, M, N, K, False)
    y = w4.gemm_fp8(x, xs, w, ws)
    for rows in (slice(0, 50), slice(262100, 262200), slice(M - 50, M)):
        check(y[rows], *product(x[rows], xs[:, rows], w, ws, False))
