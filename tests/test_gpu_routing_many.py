"""GPU: dispatch where its form changes: 16384 ids are the most of the one-launch form,
131072 the most that the sort's counting kernel takes in chunks of 2048 (beyond, chunks
are longer and no multiple of the 256 ids of a ranking CTA), and the most slots a token
can have.  Places and sizes against NumPy's stable sort, rows bit for bit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu
from test_gpu_routing import make_ids, model_slots

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(tokens, top_k, groups, width, kind, i64):
    rng = np.random.default_rng(tokens + top_k)
    ids = make_ids(rng, tokens, top_k, groups, kind)
    x = torch.randn(tokens, width, device="cuda").bfloat16()
    xs, sizes, slots = w4.dispatch(x, torch.from_numpy(ids.astype(np.int64 if i64 else np.int32)).cuda(), groups)
    want_slots, want_sizes = model_slots(ids, groups)
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert np.array_equal(sizes.cpu().numpy(), want_sizes)
    rows = torch.where(slots >= 0, slots, ~slots).long()
    want = torch.where((slots >= 0)[:, :, None], x[:, None, :], torch.zeros_like(x[:, None, :]))
    assert torch.equal(xs[rows].view(torch.int16), want.view(torch.int16))
    return x, slots


@pytest.mark.parametrize("i64", [False, True])
@pytest.mark.parametrize("kind", ["plain", "wild", "one"])
@pytest.mark.parametrize("tokens,top_k,groups,width", [
    (16384, 1, 64, 8), (16385, 1, 64, 8), (2048, 8, 1024, 16), (2049, 8, 1024, 16),
    (131072, 1, 128, 8), (131073, 1, 128, 8), (65536, 2, 3, 9), (66667, 3, 1000, 8), (200001, 1, 7, 8),
    (25000, 10, 256, 8), (3, 255, 300, 16), (3, 256, 300, 16), (64, 256, 128, 8), (65, 256, 128, 8)])
def test_dispatch(tokens, top_k, groups, width, kind, i64):
    check(tokens, top_k, groups, width, kind, i64)


def test_a_million_ids():
    check(1 << 20, 1, 513, 8, "wild", False)


@pytest.mark.parametrize("top_k", [255, 256])
def test_the_most_slots_come_back(top_k):
    x, slots = check(70, top_k, 40, 72, "wild", False)
    weights = torch.rand(70, top_k, device="cuda")
    kept = (slots >= 0).double()
    xs = w4.dispatch(x, torch.where(slots >= 0, 0, -1), 1)
    ys, place = xs[0], xs[2]
    # top_k fp32 terms of one sign pattern, rounded once
    want = (kept * weights).sum(1, keepdim=True) * x.double()
    got = w4.combine(ys, place, weights)
    assert bool(((got.double() - want).abs() <= 2.0**-8 * want.abs() + top_k * 2.0**-23 * want.abs()).all())
    dys, dw = w4.combine_backward(x, ys, place, weights)
    assert bool((dw[slots < 0] == 0).all())
    square = x.double().square().sum(1, keepdim=True) * kept
    assert bool(((dw.double() - square).abs() <= (72 + 8) * 2.0**-24 * square + 2.0**-23 * square).all())


def test_many_ids_on_a_side_stream_and_in_a_graph():
    """The copies read x before the sort has ended: inputs that change between replays."""
    T, k, E = 8195, 4, 64
    rng = np.random.default_rng(0)
    x = torch.randn(T, 128, device="cuda").bfloat16()
    ids = torch.from_numpy(make_ids(rng, T, k, E, "wild").astype(np.int32)).cuda()
    w = torch.rand(T, k, device="cuda")
    x0, ids0 = x.clone(), ids.clone()

    def step():
        h = x * 2
        xs, sizes, slots = w4.dispatch(h, ids, E)
        y = w4.combine(xs, slots, w)
        return (xs, sizes, slots, y, w4.dispatch_backward(xs, slots)) + tuple(w4.combine_backward(y, xs, slots, w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    for shift in (0, 5, 100):
        x.copy_(x0.roll(shift, 0))
        ids.copy_(ids0.roll(2 * shift, 0))
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in again]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), shift
