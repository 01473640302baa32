"""GPU: rows in expert order (dispatch), back (combine), and both gradients,
against a NumPy model in 64 bits.

Places and sizes are whole numbers and copies are bit for bit.  A combined
element is an fp32 sum of at most k products rounded once to bf16: its error
is at most 2^-8 of the result (bf16's unit roundoff) plus k * 2^-23 of the sum
of the terms' magnitudes.  An fp32 weight gradient is a sum of N products: at
most (N + 8) * 2^-24 of the sum of magnitudes for a sequential order, plus its
own rounding.  A bf16 one is that sum rounded once: the bits of the fp32
gradient's rounding."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import bf16_to_f64, bf16_to_u16, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def model_slots(ids: np.ndarray, groups: int):
    """Stable sort by group, dropped ids last: (slots, sizes)."""
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    row = np.empty_like(order)
    row[order] = np.arange(order.size)
    slots = np.where(key < groups, row, ~row).reshape(ids.shape)
    return slots, np.bincount(key, minlength=groups + 1)[:groups]


def make_ids(rng, tokens, top_k, groups, kind):
    if kind == "one":                       # every id the same
        return np.full((tokens, top_k), groups - 1)
    if kind == "none":                      # every slot dropped
        return np.full((tokens, top_k), -1)
    ids = rng.integers(0, groups, (tokens, top_k))
    if kind == "wild":                      # ids of all kinds outside the range
        wild = rng.choice([-1, -7, groups, groups + 5, 2**31 - 1, -2**31], (tokens, top_k))
        ids = np.where(rng.random((tokens, top_k)) < 0.3, wild, ids)
    if kind == "skew":
        ids = np.where(rng.random((tokens, top_k)) < 0.7, ids // 8, ids)
    return ids


# tokens, top_k, groups, width: one slot; a few; the counting launch's limit of
# 4096 ids and one more; chunk borders of the sort; the most groups; top_k past a
# register block; odd widths (no 16-byte rows).
SHAPES = [(1, 1, 1, 8), (1, 8, 128, 4096), (3, 2, 5, 130), (7, 9, 16, 264), (5, 40, 64, 72),
          (512, 8, 64, 256), (513, 8, 64, 256), (2048, 2, 8, 136), (2049, 2, 1024, 64),
          (1366, 3, 7, 33), (4097, 5, 1023, 40), (30000, 4, 256, 16), (64, 64, 1024, 2056)]


@pytest.mark.parametrize("i64", [False, True])
@pytest.mark.parametrize("kind", ["plain", "wild", "skew", "one", "none"])
@pytest.mark.parametrize("tokens,top_k,groups,width", SHAPES)
def test_dispatch(tokens, top_k, groups, width, kind, i64):
    rng = np.random.default_rng(tokens + top_k)
    ids = make_ids(rng, tokens, top_k, groups, kind)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    dev_ids = torch.from_numpy(ids.astype(np.int64 if i64 else np.int32)).cuda()
    xs, sizes, slots = w4.dispatch(x, dev_ids, groups)
    want_slots, want_sizes = model_slots(ids, groups)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(sizes.cpu().numpy(), want_sizes)
    want = np.zeros((tokens * top_k, width), np.uint16)
    bits = bf16_to_u16(x)
    for j in range(top_k):
        t = np.nonzero(want_slots[:, j] >= 0)[0]
        want[want_slots[t, j]] = bits[t]
    assert np.array_equal(bf16_to_u16(xs), want)


def test_dispatch_int64_ids_past_32_bits():
    ids = torch.tensor([[0, 2**32], [2**32 + 1, 1], [-2**40, 1]], device="cuda")
    x = torch.ones(3, 8, device="cuda").bfloat16()
    _, sizes, slots = w4.dispatch(x, ids, 2)
    assert sizes.tolist() == [1, 2]
    assert slots.tolist() == [[0, ~3], [~4, 1], [~5, 2]]


def test_dispatch_of_nothing_writes_the_sizes():
    xs, sizes, slots = w4.dispatch(torch.empty(0, 64, device="cuda").bfloat16(),
                                   torch.empty(0, 4, device="cuda", dtype=torch.int32), 6)
    assert tuple(xs.shape) == (0, 64) and tuple(slots.shape) == (0, 4)
    assert sizes.tolist() == [0] * 6
    empty = torch.empty(0, 64, device="cuda").bfloat16()
    assert tuple(w4.dispatch_backward(empty, slots).shape) == (0, 64)


def problem(tokens, top_k, groups, width, kind, dtype, seed=0):
    rng = np.random.default_rng(seed + tokens)
    ids = make_ids(rng, tokens, top_k, groups, kind)
    slots, _ = model_slots(ids, groups)
    ys = torch.randn(tokens * top_k, width, device="cuda").bfloat16()
    w = torch.rand(tokens, top_k, device="cuda").to(dtype)
    # what dropped slots own must never be read into a sum
    dropped = torch.from_numpy(~slots[slots < 0]).cuda()
    ys[dropped] = float("nan")
    if len(dropped):
        w[torch.from_numpy(slots < 0).cuda()] = float("inf")
    return slots, ys, w, torch.from_numpy(slots.astype(np.int32)).cuda()


COMBINE = [(1, 1, 1, 1), (1, 8, 128, 4096), (16, 8, 128, 4096), (5, 3, 7, 33), (9, 17, 40, 264),
           (1000, 4, 64, 136), (300, 2, 8, 2561)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("kind", ["plain", "wild", "one", "none"])
@pytest.mark.parametrize("tokens,top_k,groups,width", COMBINE)
def test_combine(tokens, top_k, groups, width, kind, dtype):
    slots, ys, w, dev = problem(tokens, top_k, groups, width, kind, dtype or torch.float32)
    got = w4.combine(ys, dev, w) if dtype else w4.dispatch_backward(ys, dev)
    y64, w64 = bf16_to_f64(ys), w.double().cpu().numpy()
    want = np.zeros((tokens, width))
    terms = np.zeros((tokens, width))
    for j in range(top_k):
        t = np.nonzero(slots[:, j] >= 0)[0]
        part = y64[slots[t, j]] * (w64[t, j, None] if dtype else 1.0)
        want[t] += part
        terms[t] += np.abs(part)
    assert np.all(np.abs(bf16_to_f64(got) - want) <= 2.0**-8 * np.abs(want) + top_k * 2.0**-23 * terms)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["plain", "wild", "none"])
@pytest.mark.parametrize("tokens,top_k,groups,width", COMBINE)
def test_combine_backward(tokens, top_k, groups, width, kind, dtype):
    slots, ys, w, dev = problem(tokens, top_k, groups, width, kind, dtype, seed=1)
    dy = torch.randn(tokens, width, device="cuda").bfloat16()
    dys, dw = w4.combine_backward(dy, ys, dev, w)
    g64, y64, w64 = bf16_to_f64(dy), bf16_to_f64(ys), w.double().cpu().numpy()
    want = np.zeros((tokens * top_k, width))
    want_dw, terms = np.zeros((tokens, top_k)), np.zeros((tokens, top_k))
    for j in range(top_k):
        t = np.nonzero(slots[:, j] >= 0)[0]
        want[slots[t, j]] = g64[t] * w64[t, j, None]
        part = g64[t] * y64[slots[t, j]]
        want_dw[t, j] = part.sum(1)
        terms[t, j] = np.abs(part).sum(1)
    # one product in fp32 and its rounding
    assert np.all(np.abs(bf16_to_f64(dys) - want) <= 2.0**-8 * np.abs(want))
    dw32 = w4.combine_backward(dy, ys, dev, w.float())[1]
    assert torch.equal(dw, dw32.to(dtype))
    err = np.abs(dw32.double().cpu().numpy() - want_dw)
    assert np.all(err <= 2.0**-24 * 1.01 * np.abs(want_dw) + (width + 8) * 2.0**-24 * terms)


def test_combine_gradient_against_differences():
    """<dY, combine(ys, w)> moved along the weights and along ys."""
    rng = np.random.default_rng(3)
    T, k, N, E = 6, 3, 40, 5
    slots, _ = model_slots(make_ids(rng, T, k, E, "wild"), E)
    dev = torch.from_numpy(slots.astype(np.int32)).cuda()
    # small whole numbers and halves: every product and sum is exact in bf16
    ys = torch.from_numpy(rng.integers(-2, 3, (T * k, N)).astype(np.float32)).cuda().bfloat16()
    dy = torch.from_numpy(rng.integers(-1, 2, (T, N)).astype(np.float32)).cuda().bfloat16()
    w = torch.from_numpy(rng.integers(1, 4, (T, k)).astype(np.float32)).cuda() / 2
    dys, dw = w4.combine_backward(dy, ys, dev, w)

    def loss(ys, w):
        return float((w4.combine(ys, dev, w).double() * dy.double()).sum())

    for t in range(T):
        for j in range(k):
            up, down = w.clone(), w.clone()
            up[t, j] += 0.5
            down[t, j] -= 0.5
            assert loss(ys, up) - loss(ys, down) == float(dw[t, j])
    for row, col in ((0, 0), (3, 7), (T * k - 1, N - 1), (8, 21)):
        up, down = ys.clone(), ys.clone()
        up[row, col] += 1
        down[row, col] -= 1
        assert (loss(up, w) - loss(down, w)) / 2 == float(dys[row, col])


def test_slots_out_of_range_are_skipped():
    ys = torch.ones(4, 16, device="cuda").bfloat16()
    slots = torch.tensor([[0, 4], [2**31 - 1, -2**31]], dtype=torch.int32, device="cuda")
    w = torch.ones(2, 2, device="cuda")
    y = w4.combine(ys, slots, w)
    assert y[0].tolist() == [1.0] * 16 and y[1].tolist() == [0.0] * 16
    dys, dw = w4.combine_backward(torch.ones(2, 16, device="cuda").bfloat16(), ys, slots, w)
    assert dw.tolist() == [[16.0, 0.0], [0.0, 0.0]] and dys[0].tolist() == [1.0] * 16


def test_unaligned_rows_take_the_narrow_path():
    # views whose start is 2 mod 16 bytes, and a width that is a multiple of 8
    flat = torch.randn(6 * 64 + 1, device="cuda").bfloat16()
    ys = flat[1:].view(6, 64)
    slots = torch.tensor([[1, 0], [~4, 3], [5, 2]], dtype=torch.int32, device="cuda")
    w = torch.rand(3, 2, device="cuda")
    assert torch.equal(w4.combine(ys, slots, w), w4.combine(ys.clone(), slots, w))
    dy = torch.randn(3, 64, device="cuda").bfloat16()
    got, want = w4.combine_backward(dy, ys, slots, w), w4.combine_backward(dy, ys.clone(), slots, w)
    assert torch.equal(got[0], want[0])
    # the dot products' order differs between the two paths
    assert torch.allclose(got[1], want[1], rtol=0, atol=72 * 2.0**-24 * 64 * 9)


@pytest.mark.parametrize("tokens,top_k,width", [(9, 2, 41), (9, 2, 42), (9, 2, 44), (9, 2, 64), (4200, 4, 42)])
def test_dispatch_of_a_view(tokens, top_k, width):
    # rows that start on 2, 4 or 8 bytes: both forms take the widest access that fits
    flat = torch.randn(tokens * width + 1, device="cuda").bfloat16()
    ids = torch.randint(-1, 5, (tokens, top_k), device="cuda")
    for x in (flat[1:].view(tokens, width), flat[:-1].view(tokens, width)):
        xs, _, slots = w4.dispatch(x, ids, 5)
        rows = torch.where(slots >= 0, slots, ~slots).long()
        want = torch.where((slots >= 0)[:, :, None], x[:, None, :], torch.zeros_like(x[:, None, :]))
        assert torch.equal(xs[rows], want)


def test_rows_feed_the_grouped_product_and_replay_in_a_graph():
    rng = np.random.default_rng(7)
    T, k, E, K, N = 24, 2, 4, 256, 384
    x = torch.randn(T, K, device="cuda").bfloat16()
    ids = torch.from_numpy(make_ids(rng, T, k, E, "wild").astype(np.int32)).cuda()
    w = torch.rand(T, k, device="cuda")
    packed = torch.stack([w4.pack(torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8))
                          for _ in range(E)])
    scales = (torch.rand(E, N, K // 128, device="cuda") * 0.02).bfloat16()

    def layer():
        xs, sizes, slots = w4.dispatch(x, ids, E)
        ys, status = w4.gemm_grouped(xs, packed, scales, sizes)
        return w4.combine(ys, slots, w), status

    y, status = layer()
    assert int(status[0]) == 0
    dense = torch.stack([w4.dequant_fp32(packed[e], scales[e]) for e in range(E)]).double()
    want = torch.zeros(T, N, device="cuda", dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < E:
                want[t] += w[t, j].double() * (dense[e] @ x[t].double())
    err = (y.double() - want).abs().max() / want.abs().max()
    assert err < 2e-2      # two bf16 roundings and the product's tolerance
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again, _ = layer()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, y)


def test_refusals():
    x = torch.zeros(4, 16, device="cuda").bfloat16()
    ids = torch.zeros(4, 2, device="cuda", dtype=torch.int32)
    for bad in (lambda: w4.dispatch(x.float(), ids, 4), lambda: w4.dispatch(x, ids.float(), 4),
                lambda: w4.dispatch(x, ids[:3], 4), lambda: w4.dispatch(x.cpu(), ids, 4),
                lambda: w4.dispatch(x.t(), ids, 4),
                lambda: w4.combine(x, ids, torch.zeros(4, 2, device="cuda")),
                lambda: w4.combine(x, ids[:2], torch.zeros(2, 2, device="cuda").half()),
                lambda: w4.combine(x, ids[:2], None),
                lambda: w4.combine_backward(x, x, ids[:2], torch.zeros(2, 2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for groups in (0, -1, 1025):
        with pytest.raises((w4.W4A16Error, RuntimeError)):
            w4.dispatch(x, ids, groups)
