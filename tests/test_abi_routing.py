"""Argument checks of the dispatch / combine entry points, on the host (no GPU)."""
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


def dispatch(L, X=FAKE, ids=FAKE, ib=4, Xs=FAKE, sizes=FAKE, slots=FAKE, T=4, k=2, W=64, E=8, ws=None, wsb=0):
    return L.w4a16_dispatch(X, ids, ib, Xs, sizes, slots, T, k, W, E, ws, wsb, None)


@pytest.mark.parametrize("bad", [dict(X=None), dict(ids=None), dict(Xs=None), dict(sizes=None),
                                 dict(slots=None), dict(T=-1), dict(k=0), dict(W=0), dict(E=0),
                                 dict(E=1025), dict(X=FAKE + 1), dict(Xs=FAKE + 1), dict(ids=FAKE + 2),
                                 dict(ib=8, ids=FAKE + 4), dict(T=1 << 20, k=17), dict(W=(1 << 20) + 1)])
def test_dispatch_refuses(L, bad):
    assert dispatch(L, **bad) == INVALID


def test_dispatch_id_types_and_workspace(L):
    assert dispatch(L, ib=2) == UNSUPPORTED
    nb = ctypes.c_size_t(1)
    assert L.w4a16_dispatch_workspace_bytes(4, 2, 8, ctypes.byref(nb)) == OK and nb.value == 0
    assert L.w4a16_dispatch_workspace_bytes(8192, 8, 128, ctypes.byref(nb)) == OK and nb.value > 0
    need = nb.value
    assert dispatch(L, T=8192, k=8, E=128) == WS_SMALL
    assert dispatch(L, T=8192, k=8, E=128, ws=FAKE, wsb=need - 1) == WS_SMALL
    assert dispatch(L, T=8192, k=8, E=128, ws=FAKE + 4, wsb=need) == INVALID
    assert L.w4a16_dispatch_workspace_bytes(8192, 8, 0, ctypes.byref(nb)) == INVALID
    assert L.w4a16_dispatch_workspace_bytes(8192, 8, 8, None) == INVALID


def combine(L, Ys=FAKE, slots=FAKE, w=FAKE, wb=4, Y=FAKE, T=4, k=2, W=64):
    return L.w4a16_combine(Ys, slots, w, wb, Y, T, k, W, None)


def test_combine_refuses(L):
    for bad in (dict(Ys=None), dict(slots=None), dict(Y=None), dict(T=-1), dict(k=0), dict(W=0),
                dict(Ys=FAKE + 1), dict(Y=FAKE + 1), dict(slots=FAKE + 2), dict(w=FAKE + 2)):
        assert combine(L, **bad) == INVALID
    assert combine(L, wb=8) == UNSUPPORTED
    assert combine(L, T=0, Ys=None, Y=None) == OK


def test_combine_backward_refuses(L):
    def call(dY=FAKE, Ys=FAKE, slots=FAKE, w=FAKE, wb=4, dYs=FAKE, dW=FAKE, T=4, k=2, W=64):
        return L.w4a16_combine_backward(dY, Ys, slots, w, wb, dYs, dW, T, k, W, None)
    for bad in (dict(dY=None), dict(Ys=None), dict(slots=None), dict(w=None), dict(dYs=None), dict(dW=None),
                dict(T=-1), dict(k=0), dict(W=0), dict(dW=FAKE + 2), dict(dY=FAKE + 1)):
        assert call(**bad) == INVALID
    assert call(wb=0) == UNSUPPORTED
    assert call(T=0, dY=None) == OK


def test_python_refuses_cpu_tensors():
    import torch
    import bf16_activation_quantized_gb300 as w4
    x, ids = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: w4.dispatch(x, ids, 2), lambda: w4.combine(x, ids[:1], torch.zeros(1, 2)),
                 lambda: w4.dispatch_backward(x, ids[:1]),
                 lambda: w4.combine_backward(x, x, ids[:1], torch.zeros(1, 2))):
        with pytest.raises(ValueError):
            call()
