"""GPU: lora_add's two forms, each by itself, where a test of one size would reach one
of them: in place, without a base, rows off 16 bytes, infinities and NaN, on a side
stream and in a graph behind the projection, and the gradient in a graph.  The bounds
are test_gpu_lora's."""
from __future__ import annotations

import ctypes

import pytest
import torch

import bf16_activation_quantized_gb300 as w4
from bf16_activation_quantized_gb300 import _lib

from gpu_util import require_gpu
from test_gpu_lora import NAN, Problem, assert_within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def form(T, L, r):
    """The few-token form takes no workspace."""
    need = ctypes.c_size_t(1)
    assert _lib.lib().w4a16_lora_workspace_bytes(T, L, r, 0, ctypes.byref(need)) == 0
    return "many" if need.value else "few"


def problem(which, L, r, N, K, kind, **kw):
    T = 61 if which == "few" else 450
    assert form(T, L, r) == which
    return Problem(T, L, r, N, K, kind, **kw)


@pytest.mark.parametrize("which", ["few", "many"])
@pytest.mark.parametrize("r,N", [(8, 264), (16, 265), (64, 264), (128, 72)])
def test_in_place_and_without_a_base(which, r, N):
    p = problem(which, 3, r, N, 256, "wild")
    want, bound, _, _ = p.forward()
    y = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base)
    assert_within(y, want, bound, "y")
    buf = p.base.clone()
    assert w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, buf, out=buf) is buf
    assert torch.equal(buf, y)
    want, bound, _, _ = p.forward(base=False)
    assert_within(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale), want, bound, "delta")


@pytest.mark.parametrize("which", ["few", "many"])
@pytest.mark.parametrize("r", [8, 16, 24, 72])
def test_infinities_and_nans_stay_in_their_rows(which, r):
    p = problem(which, 2, r, 72, 128, "one")
    T = p.shape[0]
    p.a[-1], p.b[-1] = p.a[-1].abs() + 0.01, p.b[-1].abs() + 0.01
    p.x[1, 5], p.x[2, 5] = float("inf"), NAN
    p.x[T - 1, 127] = -float("inf")
    y = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base)
    assert bool((y[1] == float("inf")).all()) and bool((y[T - 1] == -float("inf")).all())
    assert bool(torch.isnan(y[2]).all())
    assert bool(torch.isfinite(y[[i for i in range(T) if i not in (1, 2, T - 1)]]).all())


@pytest.mark.parametrize("which", ["few", "many"])
@pytest.mark.parametrize("r", [16, 64])
def test_rows_off_16_bytes(which, r):
    p = problem(which, 2, r, 64, 128, "wild")
    T = p.shape[0]
    p.dy[~p.has] = 0

    def moved(v):
        flat = torch.empty(v.numel() + 1, device="cuda", dtype=torch.bfloat16)
        flat[1:].copy_(v.reshape(-1))
        return flat[1:].view(v.shape)

    want, hidden = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base, return_hidden=True)
    base = moved(p.base)
    assert torch.equal(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, base), want)
    assert torch.equal(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, base, out=base), want)
    out = moved(torch.zeros(T, 64))
    assert torch.equal(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base, out=out), want)
    got = w4.lora_add_backward(moved(p.dy), p.x, hidden, p.a, p.b, p.ids, p.scale, dx_base=moved(p.dx_base))
    want = w4.lora_add_backward(p.dy, p.x, hidden, p.a, p.b, p.ids, p.scale, dx_base=p.dx_base)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("which", ["few", "many"])
@pytest.mark.parametrize("L,r", [(4, 16), (12, 64)])
def test_a_training_step_on_a_side_stream_and_in_a_graph(which, L, r):
    """Projection, adapters in place and their gradients; the graph's inputs change
    between its replays, so that a kernel that read ahead of the one before it shows."""
    p = problem(which, L, r, 384, 256, "wild")
    p.x[~p.has], p.dy[~p.has] = 1.0, 1.0
    packed = w4.pack(torch.randint(0, 256, (384, 128), device="cuda", dtype=torch.uint8))
    scales = (torch.rand(384, 2, device="cuda") * 0.02).bfloat16()
    x, dy, ids = p.x.clone(), p.dy.clone(), p.ids.clone()

    def step():
        y = w4.gemm(x, packed, scales)
        y, hidden = w4.lora_add(x, p.a, p.b, ids, p.scale, y, out=y, return_hidden=True)
        return (y, hidden) + w4.lora_add_backward(dy, x, hidden, p.a, p.b, ids, p.scale)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = step()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(first, want))
    for shift in (0, 7, 0, 31):
        x.copy_(p.x.roll(shift, 0))
        dy.copy_(p.dy.roll(shift, 0))
        ids.copy_(p.ids.roll(shift // 2))
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in again]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), shift
    p.base = w4.gemm(p.x, packed, scales)
    full, bound, _, _ = p.forward()
    assert_within(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base), full, bound, "projection and adapters")
