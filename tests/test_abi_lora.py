"""Argument checks of the adapter entry points, on the host (no GPU)."""
from __future__ import annotations

import ctypes

import pytest

from bf16_activation_quantized_gb300 import _lib
from bf16_activation_quantized_gb300 import build as build_mod

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = 1 << 20    # aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return _lib.lib()


def add(L, X=FAKE, A=FAKE, B=FAKE, ids=FAKE, ib=4, s=FAKE, base=FAKE, Y=FAKE, h=FAKE, T=4, n=2, r=16, N=64, K=128,
        ws=None, wsb=0):
    return L.w4a16_lora_add(X, A, B, ids, ib, s, base, Y, h, T, n, r, N, K, ws, wsb, None)


def grad(L, dY=FAKE, X=FAKE, h=FAKE, A=FAKE, B=FAKE, ids=FAKE, ib=4, s=FAKE, dXb=FAKE, dX=FAKE, dA=FAKE, dB=FAKE,
         T=4, n=2, r=16, N=64, K=128, ws=None, wsb=0):
    return L.w4a16_lora_add_backward(dY, X, h, A, B, ids, ib, s, dXb, dX, dA, dB, T, n, r, N, K, ws, wsb, None)


def ws_bytes(L, T, n, r, backward):
    nb = ctypes.c_size_t(1)
    assert L.w4a16_lora_workspace_bytes(T, n, r, backward, ctypes.byref(nb)) == OK
    return nb.value


SIZES = [dict(T=-1), dict(T=(1 << 24) + 1), dict(n=0), dict(n=1025), dict(N=0), dict(N=(1 << 24) + 1), dict(K=0),
         dict(K=64), dict(K=192), dict(K=(1 << 20) + 128)]


@pytest.mark.parametrize("bad", SIZES + [
    dict(X=None), dict(A=None), dict(B=None), dict(ids=None), dict(s=None), dict(Y=None), dict(X=FAKE + 8),
    dict(A=FAKE + 8), dict(B=FAKE + 2), dict(ids=FAKE + 2), dict(ib=8, ids=FAKE + 4), dict(s=FAKE + 2),
    dict(base=FAKE + 1), dict(Y=FAKE + 1), dict(h=FAKE + 8)])
def test_lora_add_refuses(L, bad):
    assert add(L, **bad) == INVALID


@pytest.mark.parametrize("bad", SIZES + [
    dict(dY=None), dict(X=None), dict(h=None), dict(A=None), dict(B=None), dict(ids=None), dict(s=None),
    dict(dX=None), dict(dA=None), dict(dB=None), dict(dY=FAKE + 1), dict(X=FAKE + 8), dict(h=FAKE + 4),
    dict(dA=FAKE + 8), dict(dB=FAKE + 8), dict(dX=FAKE + 1), dict(dXb=FAKE + 1)])
def test_lora_add_backward_refuses(L, bad):
    assert grad(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(r=4), dict(r=12), dict(r=136), dict(r=0), dict(ib=2)])
def test_unsupported(L, bad):
    assert add(L, **bad) == UNSUPPORTED
    assert grad(L, **bad) == UNSUPPORTED


def test_workspaces(L):
    # few tokens go without; many, and every gradient, need one
    assert ws_bytes(L, 1, 1, 8, 0) == 0 and ws_bytes(L, 0, 4, 64, 0) == 0 and ws_bytes(L, 0, 4, 64, 1) == 0
    for backward, call in ((0, add), (1, grad)):
        need = ws_bytes(L, 4096, 3, 64, backward)
        assert need > 0
        size = dict(T=4096, n=3, r=64)
        assert call(L, **size) == WS_SMALL
        assert call(L, **size, ws=FAKE, wsb=need - 1) == WS_SMALL
        assert call(L, **size, ws=FAKE + 8, wsb=need) == INVALID
    assert ws_bytes(L, 1, 1, 8, 1) > 0
    nb = ctypes.c_size_t(0)
    for bad in ((-1, 1, 8), (1, 0, 8), (1, 1025, 8)):
        assert L.w4a16_lora_workspace_bytes(*bad, 0, ctypes.byref(nb)) == INVALID
    assert L.w4a16_lora_workspace_bytes(1, 1, 9, 0, ctypes.byref(nb)) == UNSUPPORTED
    assert L.w4a16_lora_workspace_bytes(1, 1, 8, 0, None) == INVALID


def test_workspace_grows_with_tokens_and_never_wraps(L):
    # the largest call: 2^24 tokens of rank 128, more than 2^32 bytes
    sizes = [ws_bytes(L, T, 1024, 128, 1) for T in (1, 128, 4096, 1 << 20, 1 << 24)]
    assert sizes == sorted(sizes) and sizes[-1] > 1 << 32


def test_no_tokens(L):
    assert add(L, T=0, X=None, A=None, B=None, ids=None, s=None, Y=None) == OK


def test_python_refuses_cpu_tensors():
    import torch
    import bf16_activation_quantized_gb300 as w4
    x, a, b = (torch.zeros(s, dtype=torch.bfloat16) for s in ((2, 128), (1, 8, 128), (1, 16, 8)))
    ids, s = torch.zeros(2, dtype=torch.int32), torch.ones(1)
    with pytest.raises(ValueError):
        w4.lora_add(x, a, b, ids, s)
    with pytest.raises(ValueError):
        w4.lora_add_backward(torch.zeros(2, 16, dtype=torch.bfloat16), x, torch.zeros(2, 8), a, b, ids, s)
