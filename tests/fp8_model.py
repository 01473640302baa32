"""Inputs and the 64-bit model of the products in 8-bit floating point.

Bounds.  A product of two e4m3 values is exact in fp32.  A block's sum of 128 of them and
the sum over B blocks carry, however they are ordered and whether a term is rounded or
cut, at most (128 + B) * 2^-23 of the sum of the magnitudes |x w| xs ws, the products
with the scales 2 * 2^-24 more: (130 + B) * 2^-23 in all.  The result is rounded to bf16
once: 2^-8 of it."""
from __future__ import annotations

import torch


def codes(g, *shape):
    """Finite e4m3 values of all binades: any byte but the two NaNs."""
    b = torch.randint(0, 256, shape, device="cuda", dtype=torch.uint8, generator=g)
    b = torch.where((b & 0x7f) == 0x7f, b & 0x80, b)
    return b.view(torch.float8_e4m3fn)


def scales(g, *shape):
    return torch.exp2(4 * torch.rand(*shape, device="cuda", generator=g) - 8)


def problem(g, M, N, K, transposed, groups=None):
    """x, x_scales, w, w_scales of one product."""
    C = -(-N // 128) * 128 if transposed else K
    lead = () if groups is None else (groups,)
    x = codes(g, M, C)
    return x, scales(g, C // 128, M), codes(g, *lead, N, K), scales(g, *lead, -(-N // 128), K // 128)


def dense_rows(x, xs, dtype=torch.float64):
    return x.to(dtype) * xs.to(dtype).t().repeat_interleave(128, 1)


def dense_weights(w, ws, dtype=torch.float64):
    return w.to(dtype) * ws.to(dtype).repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)


def product(x, xs, w, ws, transposed):
    """(the product in 64 bits, the largest error allowed)."""
    xd, wd = dense_rows(x, xs), dense_weights(w, ws)
    if transposed:
        xd, wd = xd[:, :w.shape[0]], wd.t()
    blocks = -(-xd.shape[1] // 128)
    want = xd @ wd.t()
    return want, 2.0 ** -8 * want.abs() + (130 + blocks) * 2.0 ** -23 * (xd.abs() @ wd.abs().t())


def check(got, want, bound, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{what}: {int(bad.sum())} of {bad.numel()} elements, first at "
                                 f"{torch.nonzero(bad)[0].tolist()}, worst {float((err / bound).nan_to_num(9e9).max())} bounds")
