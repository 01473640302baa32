"""A mixture-of-experts block with 4-bit weights, served and trained through
low-rank adapters.

    h  = x W_p^T + adapters(x)                 one projection, an adapter per request
    router: softmax(h W_r^T), the top k experts of each token
    z  = silu(gate_e(h)) * up_e(h);  y = sum_j p_j * down_e(z)      W4A16 experts

The 4-bit weights are frozen; what is trained are the adapters and the router.
``python examples/moe_adapters.py`` serves a few tokens, checks a training step's
gradients against the same block in 64 bits and trains a few steps."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import bf16_activation_quantized_gb300 as w4  # noqa: E402


class Frozen:
    """``count`` matrices [N, K] of random 4-bit codes, packed, with one scale per 128 weights."""

    def __init__(self, count, N, K, gen):
        codes = torch.randint(0, 256, (count, N, K // 2), device="cuda", dtype=torch.uint8, generator=gen)
        self.packed = torch.stack([w4.pack(c) for c in codes])
        spread = torch.rand(count, N, K // 128, device="cuda", generator=gen) + 0.5
        self.scales = (spread * 0.2 * K ** -0.5).bfloat16()

    def dense(self, e, dtype):
        return w4.dequant_fp32(self.packed[e], self.scales[e]).to(dtype)

    def grouped(self, x, sizes):
        return w4.gemm_grouped(x, self.packed, self.scales, sizes)[0]

    def grouped_gradient(self, dy, sizes):
        """dx = dy W, group by group: the library multiplies by W^T only."""
        dx = torch.zeros(dy.shape[0], self.scales.shape[2] * 128, device="cuda", dtype=torch.bfloat16)
        row = 0
        for e, n in enumerate(sizes.tolist()):
            dx[row:row + n] = dy[row:row + n] @ self.dense(e, torch.bfloat16)
            row += n
        return dx


class Block:
    def __init__(self, width=512, inner=256, experts=8, top_k=2, adapters=4, rank=16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, device="cuda", generator=gen) * std).bfloat16()

        self.experts, self.top_k = experts, top_k
        self.proj = Frozen(1, width, width, gen)
        self.up = Frozen(experts, 2 * inner, width, gen)         # gate and up side by side
        self.down = Frozen(experts, width, inner, gen)
        self.lora_a = normal(adapters, rank, width, std=width ** -0.5)
        self.lora_b = normal(adapters, width, rank, std=0.1)
        self.lora_scales = torch.full((adapters,), 2.0, device="cuda")
        self.router = normal(experts, width, std=width ** -0.5)

    def forward(self, x, adapters):
        """y, and what the gradients need."""
        h = w4.gemm(x, self.proj.packed[0], self.proj.scales[0])
        h, hidden = w4.lora_add(x, self.lora_a, self.lora_b, adapters, self.lora_scales, h, out=h, return_hidden=True)
        probs, ids = torch.topk((h @ self.router.T).float().softmax(-1), self.top_k)
        hs, sizes, slots = w4.dispatch(h, ids, self.experts)
        gu = self.up.grouped(hs, sizes)
        ys = self.down.grouped(swiglu(gu), sizes)
        return w4.combine(ys, slots, probs), (x, adapters, hidden, h, ids, probs, sizes, slots, gu, ys)

    def backward(self, dy, saved):
        """Gradients of the adapters and the router."""
        x, adapters, hidden, h, ids, probs, sizes, slots, gu, ys = saved
        dys, dprobs = w4.combine_backward(dy, ys, slots, probs)
        dz = self.down.grouped_gradient(dys, sizes)
        with torch.enable_grad():
            leaf = gu.detach().requires_grad_()
            dgu, = torch.autograd.grad(swiglu(leaf), leaf, dz)
            logits = (h @ self.router.T).float().detach().requires_grad_()
            dlogits, = torch.autograd.grad(logits.softmax(-1).gather(1, ids), logits, dprobs)
        dh = w4.dispatch_backward(self.up.grouped_gradient(dgu, sizes), slots)
        dh += (dlogits @ self.router.float()).bfloat16()
        _, da, db = w4.lora_add_backward(dh, x, hidden, self.lora_a, self.lora_b, adapters, self.lora_scales)
        return da, db, dlogits.T @ h.float()

    def plain(self, x, adapters, ids, lora_a, lora_b, router):
        """The block in 64 bits by the formulas, with the experts of each token given."""
        x = x.double()
        a = lora_a[adapters.clamp(min=0).long()], lora_b[adapters.clamp(min=0).long()]
        low = torch.einsum("tnr,tr->tn", a[1], torch.einsum("trk,tk->tr", a[0], x))
        scale = torch.where(adapters >= 0, self.lora_scales.double()[adapters.clamp(min=0).long()], 0.0)
        h = x @ self.proj.dense(0, torch.float64).T + scale[:, None] * low
        probs = (h @ router.T).softmax(-1)
        y = torch.zeros_like(h)
        for e in range(self.experts):
            z = swiglu(h @ self.up.dense(e, torch.float64).T) @ self.down.dense(e, torch.float64).T
            y = y + ((ids == e).sum(1) * probs[:, e])[:, None] * z
        return y


def swiglu(gu):
    gate, up = gu.chunk(2, -1)
    return torch.nn.functional.silu(gate) * up


def relative(got, want):
    return float((got.double() - want).norm() / want.norm())


def step_errors(tokens, block, gen):
    """Relative errors of y and of the gradients of |y - target|^2 / 2."""
    x = torch.randn(tokens, block.lora_a.shape[2], device="cuda", generator=gen).bfloat16()
    target = torch.randn_like(x)
    adapters = torch.randint(-1, block.lora_a.shape[0], (tokens,), device="cuda", dtype=torch.int32, generator=gen)
    y, saved = block.forward(x, adapters)
    grads = block.backward(y - target, saved)
    leaves = [p.double().requires_grad_() for p in (block.lora_a, block.lora_b, block.router)]
    with torch.enable_grad():
        want = block.plain(x, adapters, saved[4], *leaves)
        wanted = torch.autograd.grad(want, leaves, (want - target.double()).detach())
    return [relative(y, want.detach())] + [relative(g, w) for g, w in zip(grads, wanted)]


def train(block, steps=30, tokens=512, rate=0.02, gen=None):
    """Losses of a few normalised gradient steps on one batch; the masters are 32-bit."""
    x = torch.randn(tokens, block.lora_a.shape[2], device="cuda", generator=gen).bfloat16()
    target = 0.1 * torch.randn_like(x)
    adapters = torch.randint(0, block.lora_a.shape[0], (tokens,), device="cuda", dtype=torch.int32, generator=gen)
    names = ("lora_a", "lora_b", "router")
    masters = [getattr(block, n).float() for n in names]
    losses = []
    for _ in range(steps):
        y, saved = block.forward(x, adapters)
        losses.append(float((y - target).float().square().mean()))
        for name, master, grad in zip(names, masters, block.backward(y - target, saved)):
            master -= rate * master.norm() * grad.float() / grad.float().norm()
            setattr(block, name, master.bfloat16())
    return losses


@torch.no_grad()
def main():
    gen = torch.Generator(device="cuda").manual_seed(1)
    block = Block()
    for tokens in (1, 5, 64, 700):
        errors = step_errors(tokens, block, gen)
        print(f"{tokens:4d} tokens: relative error of y {errors[0]:.4f}, of the gradients of "
              f"A {errors[1]:.4f}, B {errors[2]:.4f}, router {errors[3]:.4f}")
    losses = train(block, gen=gen)
    print(f"loss {losses[0]:.5f} -> {losses[-1]:.5f} in {len(losses)} steps")


if __name__ == "__main__":
    main()
