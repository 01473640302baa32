"""GPU: low-rank adapters (lora_add) and their gradients against the formulas in
64 bits.

Bounds, element by element, from the roundings the kernels make.  With S(.) a sum
of magnitudes:
  h is an fp32 sum of K exact products:            e_h = K 2^-23 S(A x)
  it enters the second product to 2^-16 of it, and r terms are summed in fp32:
                                e = s |B| (e_h + (2^-16 + r 2^-22) |h|)
  base is added in fp32, the result rounded to bf16 (unit roundoff 2^-8):
                                |y - y64| <= 2^-8 |y64| + e + 2^-22 |base|
and the same for dx with (B, A, N) in place of (A, B, K); dA and dB sum the
adapter's T tokens, with (2^-16 + T 2^-22)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import bf16_activation_quantized_gb300 as w4

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def make_ids(rng, T, L, kind):
    if kind == "one":
        return np.full(T, L - 1)
    if kind == "none":
        return np.full(T, -1)
    ids = rng.integers(0, L, T)
    if kind == "segments":
        ids = np.sort(ids)
    if kind == "wild":
        ids = np.where(rng.random(T) < 0.3, rng.choice([-1, -9, L, L + 3, 2**31 - 1, -2**31], T), ids)
    return ids


class Problem:
    def __init__(self, T, L, r, N, K, kind, seed=0, i64=False):
        rng = np.random.default_rng(seed + T + r)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + T + N)

        def normal(*shape, std=1.0):
            return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()

        self.shape = (T, L, r, N, K)
        ids = make_ids(rng, T, L, kind)
        self.ids = torch.from_numpy(ids.astype(np.int64 if i64 else np.int32)).cuda()
        self.has = torch.from_numpy((ids >= 0) & (ids < L)).cuda()
        self.x, self.dy = normal(T, K), normal(T, N)
        self.base, self.dx_base = normal(T, N), normal(T, K)
        self.a, self.b = normal(L, r, K, std=K ** -0.5), normal(L, N, r, std=0.5 * r ** -0.5)
        self.scale = torch.rand(L, device="cuda", generator=g) + 0.5
        # rows of tokens without an adapter are never read
        self.x[~self.has] = NAN
        self.dy[~self.has] = NAN

    def forward(self, base=True):
        """(y, its bound, h, e_h) in 64 bits."""
        T, L, r, N, K = self.shape
        y = self.base.double().clone() if base else torch.zeros(T, N, device="cuda", dtype=torch.float64)
        e = y.abs() * 2.0**-22
        h = torch.zeros(T, r, device="cuda", dtype=torch.float64)
        eh = torch.zeros_like(h)
        for l in range(L):
            t = torch.nonzero(self.has & (self.ids == l))[:, 0]
            x, a, b, s = self.x[t].double(), self.a[l].double(), self.b[l].double(), self.scale[l].double()
            h[t] = x @ a.T
            eh[t] = K * 2.0**-23 * (x.abs() @ a.abs().T)
            y[t] += s * h[t] @ b.T
            e[t] += s * (eh[t] + (2.0**-16 + r * 2.0**-22) * h[t].abs()) @ b.abs().T
        return y, e + 2.0**-8 * y.abs(), h, eh

    def backward(self, h, eh, base=True):
        """((dx, dA, dB), their bounds) in 64 bits."""
        T, L, r, N, K = self.shape
        dx = self.dx_base.double().clone() if base else torch.zeros(T, K, device="cuda", dtype=torch.float64)
        ex = dx.abs() * 2.0**-22
        da, db = torch.zeros(L, r, K).cuda().double(), torch.zeros(L, N, r).cuda().double()
        ea, eb = torch.zeros_like(da), torch.zeros_like(db)
        for l in range(L):
            t = torch.nonzero(self.has & (self.ids == l))[:, 0]
            x, a, b, s = self.x[t].double(), self.a[l].double(), self.b[l].double(), self.scale[l].double()
            dy = self.dy[t].double()
            g = s * dy @ b
            eg = N * 2.0**-23 * s * dy.abs() @ b.abs() + 2.0**-24 * g.abs()
            many = 2.0**-16 + len(t) * 2.0**-22
            dx[t] += g @ a
            ex[t] += (eg + (2.0**-16 + r * 2.0**-22) * g.abs()) @ a.abs()
            da[l] = g.T @ x
            ea[l] = (eg + many * g.abs()).T @ x.abs()
            db[l] = s * dy.T @ h[t]
            eb[l] = s * dy.abs().T @ (eh[t] + many * h[t].abs())
        want = (dx, da, db)
        return want, tuple(e + 2.0**-8 * w.abs() for e, w in zip((ex, ea, eb), want))


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - bound).nan_to_num(1e9).max())}"


# T, L, r, N, K: one token; a tile and one more; both forms at every rank block; odd
# output widths; more adapters than tokens; past the ids one CTA counts.
SHAPES = [(1, 1, 8, 8, 128), (1, 8, 16, 8192, 1024), (2, 3, 24, 1, 128), (16, 1, 16, 264, 256), (17, 1, 32, 72, 384),
          (61, 64, 48, 1000, 640), (128, 4, 64, 136, 256), (128, 2, 128, 200, 256), (129, 2, 128, 200, 256),
          (129, 40, 16, 7, 128), (64, 1, 40, 2561, 1152), (193, 3, 64, 2561, 1152), (500, 16, 8, 33, 2560),
          (192, 1, 16, 72, 128), (193, 12, 16, 72, 128), (400, 25, 64, 136, 256), (401, 25, 64, 136, 256),
          (512, 32, 32, 40, 128), (513, 40, 32, 40, 128), (1000, 5, 32, 640, 256), (777, 300, 16, 96, 128), (2051, 2, 56, 300, 128), (17000, 9, 16, 24, 128),
          # the most tokens of the few-token form and one more, to rank 32 and past it
          (384, 1, 16, 72, 128), (385, 1, 16, 72, 128), (768, 24, 32, 40, 128), (769, 24, 32, 40, 128),
          (512, 32, 40, 40, 128), (513, 32, 40, 40, 128), (512, 31, 64, 40, 128)]


@pytest.mark.parametrize("kind", ["plain", "wild", "segments", "one", "none"])
@pytest.mark.parametrize("T,L,r,N,K", SHAPES)
def test_lora_add(T, L, r, N, K, kind):
    p = Problem(T, L, r, N, K, kind, i64=kind == "segments")
    want, bound, h, eh = p.forward()
    out = torch.full((T, N), NAN, device="cuda").bfloat16()
    y, hidden = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base, out=out, return_hidden=True)
    assert y is out
    assert_within(y, want, bound, "y")
    assert_within(hidden, h, eh + 2.0**-24 * h.abs(), "hidden")
    assert torch.equal(y[~p.has], p.base[~p.has])       # bit for bit
    again = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base)
    assert torch.equal(again, y)                         # a fixed order


@pytest.mark.parametrize("kind", ["plain", "wild", "one", "none"])
@pytest.mark.parametrize("T,L,r,N,K", SHAPES)
def test_lora_add_backward(T, L, r, N, K, kind):
    p = Problem(T, L, r, N, K, kind, seed=1)
    _, _, h, eh = p.forward()
    hidden = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base, return_hidden=True)[1]
    for base in (True, False):
        got = w4.lora_add_backward(p.dy, p.x, hidden, p.a, p.b, p.ids, p.scale,
                                   dx_base=p.dx_base if base else None)
        want, bound = p.backward(h, eh, base)
        for name, g, w, e in zip(("dx", "dA", "dB"), got, want, bound):
            assert_within(g, w, e, name)
    again = w4.lora_add_backward(p.dy, p.x, hidden, p.a, p.b, p.ids, p.scale)
    assert all(torch.equal(a, b) for a, b in zip(again, got))


@pytest.mark.parametrize("T", [5, 300])
def test_in_place_and_without_a_base(T):
    p = Problem(T, 3, 16, 264, 256, "wild")
    y = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base)
    buf = p.base.clone()
    assert w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, buf, out=buf) is buf
    assert torch.equal(buf, y)
    want, bound, _, _ = p.forward(base=False)
    assert_within(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale), want, bound, "delta")


@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("N", [40, 41])
def test_gradients_against_differences(T, N):
    """<dY, lora_add> moved along x, A and B; whole numbers small enough that every
    sum is exact in bf16 leave nothing but the derivative."""
    rng = np.random.default_rng(T)
    L, r, K = 2, 8, 128

    def sparse(*shape, share):
        v = rng.integers(-1, 2, shape) * (rng.random(shape) < share)
        return torch.from_numpy(v.astype(np.float32)).cuda().bfloat16()

    x, a, b = sparse(T, K, share=0.1), sparse(L, r, K, share=0.1), sparse(L, N, r, share=0.3)
    dy = sparse(T, N, share=4.0 / T)
    ids = torch.from_numpy(rng.integers(-1, L, T).astype(np.int32)).cuda()
    scale = torch.tensor([1.0, 2.0], device="cuda")
    _, hidden = w4.lora_add(x, a, b, ids, scale, return_hidden=True)
    grads = w4.lora_add_backward(dy, x, hidden, a, b, ids, scale)

    def loss(x, a, b):
        return float((w4.lora_add(x, a, b, ids, scale).double() * dy.double()).sum())

    where = [torch.nonzero(grads[0])[::97], torch.nonzero(grads[1])[::53], torch.nonzero(grads[2])[::29],
             torch.tensor([[T - 1, K - 1]]), torch.tensor([[L - 1, r - 1, K - 1]]), torch.tensor([[0, N - 1, 0]])]
    for k, places in enumerate(where):
        for at in places.tolist():
            at = tuple(at)
            up, down = [v.clone() for v in (x, a, b)], [v.clone() for v in (x, a, b)]
            up[k % 3][at] += 1
            down[k % 3][at] -= 1
            assert (loss(*up) - loss(*down)) / 2 == float(grads[k % 3][at])


@pytest.mark.parametrize("T", [4, 140])
def test_infinities_and_nans_stay_in_their_rows(T):
    p = Problem(T, 2, 8, 72, 128, "one")
    p.a[-1], p.b[-1] = p.a[-1].abs() + 0.01, p.b[-1].abs() + 0.01
    p.x[1, 5], p.x[2, 5] = float("inf"), NAN
    y = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base)
    # all of A and B positive: h is +inf in every rank, and so is y (a rank of 8 is
    # padded inside the kernel, where 0 * inf must not get in)
    assert bool((y[1] == float("inf")).all())
    assert bool(torch.isnan(y[2]).all())
    rest = [i for i in range(T) if i not in (1, 2)]
    assert bool(torch.isfinite(y[rest]).all())


def test_unaligned_rows_take_the_narrow_path():
    for T in (9, 200):
        p = Problem(T, 2, 16, 64, 128, "wild")
        p.dy[~p.has] = 0
        flat = torch.empty(T * 64 + 1, device="cuda", dtype=torch.bfloat16)
        base = flat[1:].view(T, 64)
        base.copy_(p.base)
        assert torch.equal(w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, base),
                           w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base))
        hidden = w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, p.base, return_hidden=True)[1]
        dy = torch.empty(T * 64 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(T, 64)
        dy.copy_(p.dy)
        got = w4.lora_add_backward(dy, p.x, hidden, p.a, p.b, p.ids, p.scale)
        want = w4.lora_add_backward(p.dy, p.x, hidden, p.a, p.b, p.ids, p.scale)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens():
    p = Problem(3, 2, 16, 64, 128, "plain")
    x, ids = p.x[:0], p.ids[:0]
    y, hidden = w4.lora_add(x, p.a, p.b, ids, p.scale, return_hidden=True)
    assert tuple(y.shape) == (0, 64) and tuple(hidden.shape) == (0, 16)
    dx, da, db = w4.lora_add_backward(p.dy[:0], x, hidden, p.a, p.b, ids, p.scale)
    assert tuple(dx.shape) == (0, 128) and not bool(da.any()) and not bool(db.any())


@pytest.mark.parametrize("T", [8, 300])
def test_beside_the_projection_on_a_side_stream_and_in_a_graph(T):
    p = Problem(T, 4, 16, 384, 256, "wild")
    p.x[~p.has] = 1.0
    packed = w4.pack(torch.randint(0, 256, (384, 128), device="cuda", dtype=torch.uint8))
    scales = (torch.rand(384, 2, device="cuda") * 0.02).bfloat16()

    def layer():
        y = w4.gemm(p.x, packed, scales)
        return w4.lora_add(p.x, p.a, p.b, p.ids, p.scale, y, out=y)

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            again = layer()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)
    p.base = w4.gemm(p.x, packed, scales)
    full, bound, _, _ = p.forward()
    assert_within(want, full, bound, "projection and adapters")


def test_refusals():
    p = Problem(4, 2, 16, 64, 128, "plain")
    ok = dict(x=p.x, a=p.a, b=p.b, ids=p.ids, s=p.scale, base=p.base)

    def call(**kw):
        v = {**ok, **kw}
        return w4.lora_add(v["x"], v["a"], v["b"], v["ids"], v["s"], v["base"])

    for bad in (dict(x=p.x.float()), dict(x=p.x.cpu()), dict(x=p.x[:, :64]), dict(a=p.a[:1]), dict(b=p.b[:, :, :8]),
                dict(a=p.a[:, :, :64].contiguous()), dict(ids=p.ids.float()), dict(ids=p.ids[:3]),
                dict(s=p.scale.double()), dict(s=p.scale[:1]), dict(base=p.base[:3]), dict(base=p.base.float())):
        with pytest.raises(ValueError):
            call(**bad)
    for r in (4, 12, 136):
        with pytest.raises(w4.W4A16Error) as e:
            call(a=torch.zeros(2, r, 128, device="cuda").bfloat16(), b=torch.zeros(2, 64, r, device="cuda").bfloat16())
        assert e.value.status == 2
    hidden = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: w4.lora_add_backward(p.dy[:3], p.x, hidden, p.a, p.b, p.ids, p.scale),
                lambda: w4.lora_add_backward(p.dy, p.x, hidden.bfloat16(), p.a, p.b, p.ids, p.scale),
                lambda: w4.lora_add_backward(p.dy, p.x, hidden[:, :8], p.a, p.b, p.ids, p.scale),
                lambda: w4.lora_add_backward(p.dy, p.x, hidden, p.a, p.b, p.ids, p.scale, dx_base=p.base)):
        with pytest.raises(ValueError):
            bad()
