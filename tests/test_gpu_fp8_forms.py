"""GPU: every form of the 8-bit products and of the weights' gradients against 64 bits, at sizes
that take it (fp8_forms; tests of the rules on the host hold them to it)."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from fp8_forms import GROUPED, PLAIN, WGRAD
from fp8_model import check, problem, product
from gpu_util import require_gpu
from test_gpu_fp8_failure import PRODUCTS, run, stalling  # noqa: F401
from test_gpu_fp8_gemm import check_grouped, gen, group_sizes, poisoned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("form", PLAIN, ids=str)
def test_plain(form, transposed):
    M, N, K = PLAIN[form][transposed]
    args = problem(gen(M, N, K), M, N, K, transposed)
    got = w4.gemm_fp8(*args, transposed=transposed, out=poisoned(M, K if transposed else N))
    check(got, *product(*args, transposed), f"{form}: {M}x{N}x{K}")
    assert torch.equal(w4.gemm_fp8(*args, transposed=transposed, resident_weights=True), got)


# sizes that leave clusters without a tile ("none", "short", "one") and groups without rows
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("kind", ["even", "one", "none", "random", "skew", "short"])
@pytest.mark.parametrize("form", GROUPED, ids=str)
def test_grouped(form, kind, transposed):
    M, E, N, K = GROUPED[form][transposed]
    sizes = group_sizes(torch.Generator().manual_seed(M + E), kind, E, M)
    check_grouped(problem(gen(M, E, N, K), M, N, K, transposed, E), sizes, transposed, M, K if transposed else N)


@pytest.mark.parametrize("form", [(16, False, 4), (64, False, 8), (128, False, 2), (0, False, 2)], ids=str)
def test_group_sizes_that_do_not_fit_in_clusters(form):
    M, E, N, K = GROUPED[form][0]
    for sizes, status in (([M - 1] + [5] * (E - 1), 2), ([-3] + [M // E] * (E - 1), 1)):
        check_grouped(problem(gen(M, 7), M, N, K, False, E), sizes, False, M, N, status)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("split", WGRAD)
def test_weight_gradients(split, dtype):
    """Groups of one part of 512 rows, of several, odd and even, and of none in turn, with rows behind
    the last that no group covers."""
    for sizes, N, K in WGRAD[split]:
        used, g = sum(sizes), gen(split, N, K)
        M = used + (77 if split == 1 else 0)
        dy = torch.randn(M, N, device="cuda", generator=g).bfloat16()
        x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
        dy[used:], x[used:] = float("nan"), float("inf")
        out = torch.full((len(sizes), N, K), float("nan"), dtype=dtype, device="cuda")
        m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
        dw, status = w4.gemm_grouped_wgrad(dy, x, m, dtype=dtype, out=out)
        assert dw is out and int(status[0]) == 0
        row = 0
        for e, n in enumerate(sizes):
            a, b = dy[row:row + n].double(), x[row:row + n].double()
            want = a.t() @ b
            # n products, exact in fp32, added in any order, rounded or cut: 2^-23 of the magnitudes each
            bound = n * 2.0 ** -23 * (a.abs().t() @ b.abs()) + (2.0 ** -8 * want.abs() if dtype == torch.bfloat16 else 0.0)
            err = (dw[e].double() - want).abs()
            assert bool((err <= bound).all()), (sizes, e, float((err - bound).max()))
            row += n


# a wait that runs out in a cluster whose CTAs share a group's tile: NaN or right, nothing else
@pytest.mark.parametrize("at", [0, 1, 3])
@pytest.mark.parametrize("form", [(16, False, 4), (64, False, 8), (128, False, 2), (0, False, 2)], ids=str)
def test_waits_that_run_out_in_a_cluster(stalling, monkeypatch, form, at):  # noqa: F811
    for transposed, (M, E, N, K) in enumerate(GROUPED[form]):
        args = problem(gen(M, E), M, N, K, bool(transposed), E)
        sizes = torch.tensor(group_sizes(torch.Generator().manual_seed(M), "random", E, M), dtype=torch.int32, device="cuda")
        run(stalling, monkeypatch, PRODUCTS, at,
            lambda out: w4.gemm_fp8_grouped(*args, sizes, transposed=bool(transposed), out=out)[0],
            (M, K if transposed else N), torch.bfloat16)
