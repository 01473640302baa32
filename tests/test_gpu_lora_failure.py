"""GPU: the failure path of the adapters' kernels for many tokens, made to run without
faulting the GPU.

A build of lora_tensor.cu for this test lets the producers of every other CTA stop
reporting their stages (or tiles) from a given one on, with a wait limit of 1 ms.  The
kernels then have to end on their own, record W4A16_ERROR_WAIT_TIMEOUT, and leave NaN
wherever they did not finish: an element of any output is NaN or the right one, never
what the buffer held before or a sum of part of the terms."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import bf16_activation_quantized_gb300 as w4
from bf16_activation_quantized_gb300 import _lib
from bf16_activation_quantized_gb300 import build as build_mod

from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

DOWN, UP, WGRAD, DOWN_TILE, UP_TILE = 1, 2, 3, 4, 5      # the source's enum Stall


@pytest.fixture(scope="module")
def stalling(tmp_path_factory):
    require_gpu()
    where = tmp_path_factory.mktemp("stalling")
    obj, lib = str(where / "lora_tensor.o"), str(where / "libstalling.so")
    flags = build_mod.ARCH + build_mod.NVCC_FLAGS + ["-DW4A16_TEST_STALL", "-DW4A16_WAIT_LIMIT_NS=1000000ull"]
    subprocess.run([build_mod.nvcc()] + flags + ["-c", os.path.join(build_mod.CSRC, "lora_tensor.cu"), "-o", obj],
                   check=True, capture_output=True)
    others = [os.path.join(build_mod.BUILD, os.path.basename(src) + ".o") for src in build_mod._sources()
              if not src.endswith("lora_tensor.cu")]
    if not all(os.path.exists(o) for o in others):
        build_mod.build(force=True)
    subprocess.run([build_mod.nvcc()] + build_mod.ARCH + ["-shared", "-o", lib, obj] + others
                   + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"], check=True, capture_output=True)
    handle = ctypes.CDLL(lib)
    for name, (res, args) in _lib.SIGNATURES.items():
        getattr(handle, name).restype, getattr(handle, name).argtypes = res, args
    return handle


def right_or_nan(got, want, what):
    wrong = ~torch.isnan(got.float()) & (got != want)
    assert not bool(wrong.any()), f"{what}: {int(wrong.sum())} elements neither right nor NaN"
    return bool(torch.isnan(got.float()).any())


# runs that lie in one tile, with and without a wrap of the rings, and runs over several tiles
@pytest.mark.parametrize("at", [0, 1, 4])
@pytest.mark.parametrize("kernel", [DOWN, UP, WGRAD, DOWN_TILE, UP_TILE])
@pytest.mark.parametrize("T,L,r,N,K", [(5000, 3, 64, 4096, 4096), (60000, 40, 16, 264, 256)])
def test_waits_that_run_out_leave_nan(stalling, monkeypatch, T, L, r, N, K, kernel, at):
    g = torch.Generator(device="cuda").manual_seed(T)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std).bfloat16()

    x, dy, base, dx_base = normal(T, K), normal(T, N), normal(T, N), normal(T, K)
    a, b = normal(L, r, K, std=K ** -0.5), normal(L, N, r, std=0.5 * r ** -0.5)
    ids = torch.randint(-1, L, (T,), device="cuda", dtype=torch.int32, generator=g)
    scale = torch.rand(L, device="cuda", generator=g) + 0.5
    y, hidden = w4.lora_add(x, a, b, ids, scale, base, return_hidden=True)
    grads = w4.lora_add_backward(dy, x, hidden, a, b, ids, scale, dx_base=dx_base)
    torch.cuda.synchronize()
    monkeypatch.setattr(_lib, "_lib", stalling)
    # outputs that torch allocates hold zeros, as far as these calls are concerned
    monkeypatch.setattr(w4, "_empty", lambda shape, dtype, index: torch.zeros(shape, dtype=dtype, device=index))
    monkeypatch.setattr(torch, "empty_like", torch.zeros_like)
    try:
        assert stalling.w4a16_test_stall(kernel, at) == 0
        assert w4.read_error_word(clear=True) == 0
        got, got_hidden = w4.lora_add(x, a, b, ids, scale, base, return_hidden=True)
        lost = [right_or_nan(got, y, "y"), right_or_nan(got_hidden, hidden, "hidden")]
        # a stage that the shorter runs do not have stalls nothing
        assert any(lost) == bool(w4.read_error_word(clear=True) & w4.ERROR_WAIT_TIMEOUT)
        buf = base.clone()
        right_or_nan(w4.lora_add(x, a, b, ids, scale, buf, out=buf), y, "y in place")
        w4.read_error_word(clear=True)
        got = w4.lora_add_backward(dy, x, hidden, a, b, ids, scale, dx_base=dx_base)
        lost += [right_or_nan(v, want, name) for v, want, name in zip(got, grads, ("dx", "dA", "dB"))]
        assert any(lost[2:]) == bool(w4.read_error_word(clear=True) & w4.ERROR_WAIT_TIMEOUT)
        if at == 0:
            assert any(lost)
    finally:
        assert stalling.w4a16_test_stall(0, 0) == 0
    # the context stays usable and the next call is right
    assert torch.equal(w4.lora_add(x, a, b, ids, scale, base), y)
    assert w4.read_error_word(clear=True) == 0
