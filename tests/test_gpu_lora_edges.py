"""GPU: adapters where a kernel can go wrong without a random problem showing it --
sums that cancel, infinities, each form of lora_add by itself.

lora_add has two forms, by rank and tokens; FEW and MANY are on their sides of the
border for one adapter at every rank that is used here (up to rank 32 the few-token
form ends at 384 tokens, past it at 128; the gradient has one form)."""
from __future__ import annotations

import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

FEW, MANY = 5, 450
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def zeros(*shape):
    return torch.zeros(*shape, device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("r", [8, 16, 24, 48, 64, 128])
def test_h_and_g_keep_all_bits_of_32(T, r):
    """h (and g) of 1 + 2^-10 + 2^-20 beside 1 + 2^-10: 21 bits, all but the last of
    which cancel in the second product and in the weight gradients.  Every product and
    sum is exact in 24 bits, so the outputs have to be 2^-20 and nothing else."""
    N = K = 256
    ids, one = torch.zeros(T, device="cuda", dtype=torch.int32), torch.ones(1, device="cuda")
    long, short = torch.tensor([1, 2.0**-10, 2.0**-20], device="cuda"), torch.tensor([1, 2.0**-10, 0], device="cuda")
    p, q = r - 1, r - 2                                  # the two ranks
    # forward, and dB over two tokens: x = long and short (negated) under A = ones
    x, a, b = zeros(T, K), zeros(1, r, K), zeros(1, N, r)
    x[:, 130:133] = long.bfloat16()
    a[0, p, 130:133], a[0, q, 130:132] = 1, 1
    b[0, :, p], b[0, :, q] = 1, -1
    y, hidden = w4.lora_add(x, a, b, ids, one, return_hidden=True)
    assert hidden[:, p].tolist() == [1 + 2.0**-10 + 2.0**-20] * T and hidden[:, q].tolist() == [1 + 2.0**-10] * T
    assert bool((y == 2.0**-20).all())
    # dx: g from dy, the weights' parts exchanged
    dy, a, b = zeros(T, N), zeros(1, r, K), zeros(1, N, r)
    dy[:, 130:133] = long.bfloat16()
    b[0, 130:133, p], b[0, 130:132, q] = 1, 1
    a[0, p], a[0, q] = 1, -1
    dx = w4.lora_add_backward(dy, zeros(T, K), torch.zeros(T, r, device="cuda"), a, b, ids, one)[0]
    assert bool((dx == 2.0**-20).all())
    # dA: two tokens' g cancel; dB: two tokens' h
    dy[1:] = 0
    dy[T - 1, 130:133] = -short.bfloat16()
    x, hidden, b = zeros(T, K), torch.zeros(T, r, device="cuda"), zeros(1, N, r)
    x[0], x[T - 1] = 1, 1
    b[0, 130:133, p] = 1
    da = w4.lora_add_backward(dy, x, hidden, a, b, ids, one)[1]
    assert bool((da[0, p] == 2.0**-20).all()) and not bool(da[0, :p].any())
    dy.zero_()
    dy[0], dy[T - 1] = 1, 1
    hidden[0, p], hidden[T - 1, p] = 1 + 2.0**-10 + 2.0**-20, -(1 + 2.0**-10)
    db = w4.lora_add_backward(dy, x, hidden, a, b, ids, one)[2]
    assert bool((db[0, :, p] == 2.0**-20).all()) and not bool(db[0, :, :p].any())


def positive(g, *shape):
    return (torch.rand(*shape, device="cuda", generator=g) + 0.25).bfloat16()


@pytest.mark.parametrize("T", [FEW, MANY])
@pytest.mark.parametrize("r", [8, 16, 24, 40, 64, 72])
def test_an_infinite_scale_gives_infinities(T, r):
    """Every operand positive: s h, g and all that follows are +inf, also at ranks that
    the kernels pad and in tiles whose last rows hold no token; the other adapter's
    tokens and gradients stay finite."""
    g = torch.Generator(device="cuda").manual_seed(r)
    N, K = 136, 128
    x, dy, base = positive(g, T, K), positive(g, T, N), positive(g, T, N)
    a, b = positive(g, 2, r, K), positive(g, 2, N, r)
    ids = (torch.arange(T, device="cuda") % 2).to(torch.int32)
    scale = torch.tensor([INF, 1.0], device="cuda")
    y, hidden = w4.lora_add(x, a, b, ids, scale, base, return_hidden=True)
    dx, da, db = w4.lora_add_backward(dy, x, hidden, a, b, ids, scale)
    assert bool(torch.isfinite(hidden).all())
    for name, v in (("y", y), ("dx", dx)):
        assert bool((v[ids == 0] == INF).all()) and bool(torch.isfinite(v[ids == 1]).all()), name
    for name, v in (("dA", da), ("dB", db)):
        assert bool((v[0] == INF).all()) and bool(torch.isfinite(v[1]).all()), name


@pytest.mark.parametrize("r", [8, 24, 64, 128])
def test_an_infinity_of_a_row_reaches_its_column_of_the_weight_gradients(r):
    """x[t, c] = inf makes dA[:, c] = g[t] * inf, dy[t, n] = inf makes dB[n] = s h[t] *
    inf: infinities of g's and h's signs, whether these fill 24 bits or one."""
    T, N, K = 200, 136, 256
    g = torch.Generator(device="cuda").manual_seed(r)
    x, dy = positive(g, T, K), positive(g, T, N)
    a, b = positive(g, 1, r, K), positive(g, 1, N, r)
    sign = torch.where(torch.arange(r, device="cuda") % 2 == 0, 1.0, -1.0)
    b *= sign.bfloat16()
    ids, one = torch.zeros(T, device="cuda", dtype=torch.int32), torch.ones(1, device="cuda")
    hidden = (torch.rand(T, r, device="cuda", generator=g) + 0.25) * sign
    hidden[3] = 0.5 * sign                               # one bit: nothing in the lower planes
    finite_x, finite_dy = x.clone(), dy.clone()
    x[2, 5], x[3, 130], x[150, 255] = INF, -INF, INF
    da = w4.lora_add_backward(finite_dy, x, hidden, a, b, ids, one)[1][0]
    for c, s in ((5, 1), (130, -1), (255, 1)):
        assert da[:, c].tolist() == (INF * s * sign).tolist(), c
    rest = torch.ones(K, dtype=torch.bool, device="cuda")
    rest[[5, 130, 255]] = False
    assert bool(torch.isfinite(da[:, rest]).all())
    dy[2, 7], dy[3, 8], dy[150, 135] = INF, -INF, INF
    db = w4.lora_add_backward(dy, finite_x, hidden, a, b, ids, one)[2][0]
    for n, s in ((7, 1), (8, -1), (135, 1)):
        assert db[n].tolist() == (INF * s * sign).tolist(), n
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[[7, 8, 135]] = False
    assert bool(torch.isfinite(db[rest]).all())
