"""GPU: the failure path of the 8-bit products and of the weights' gradients, made to run
without faulting the GPU.

A build for this test lets the producers of every other pair of CTAs stop issuing copies
from a given stage on, with a wait limit of 1 ms.  The kernels then have to end on their
own, record W4A16_ERROR_WAIT_TIMEOUT, and leave NaN wherever they did not finish: an
element of a result is NaN or the right one, never what the buffer held before or a sum
of part of the terms."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest
import torch

import bf16_activation_quantized_gb300 as w4
from bf16_activation_quantized_gb300 import _lib
from bf16_activation_quantized_gb300 import build as build_mod

from fp8_model import problem
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

UNITS = ("fp8_gemm.cu", "fp8_many.cu", "wgrad.cu")


@pytest.fixture(scope="module")
def stalling(tmp_path_factory):
    require_gpu()
    where = tmp_path_factory.mktemp("stalling_fp8")
    flags = build_mod.ARCH + build_mod.NVCC_FLAGS + ["-DW4A16_TEST_STALL", "-DW4A16_WAIT_LIMIT_NS=1000000ull"]
    objs = [str(where / (u + ".o")) for u in UNITS]
    jobs = [subprocess.Popen([build_mod.nvcc()] + flags + ["-c", os.path.join(build_mod.CSRC, u), "-o", o],
                             stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL) for u, o in zip(UNITS, objs)]
    assert [j.wait() for j in jobs] == [0] * len(jobs)
    others = [os.path.join(build_mod.BUILD, os.path.basename(src) + ".o") for src in build_mod._sources()
              if os.path.basename(src) not in UNITS]
    if not all(os.path.exists(o) for o in others):
        build_mod.build(force=True)
    lib = str(where / "libstalling.so")
    subprocess.run([build_mod.nvcc()] + build_mod.ARCH + ["-shared", "-o", lib] + objs + others
                   + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"], check=True, capture_output=True)
    handle = ctypes.CDLL(lib)
    for name, (res, args) in _lib.SIGNATURES.items():
        getattr(handle, name).restype, getattr(handle, name).argtypes = res, args
    return handle


PRODUCTS = ("w4a16_test_stall_few", "w4a16_test_stall_many")      # whichever form a call takes


def run(stalling, monkeypatch, entries, at, call, shape, dtype):
    want = call(torch.zeros(shape, dtype=dtype, device="cuda"))
    torch.cuda.synchronize()
    monkeypatch.setattr(_lib, "_lib", stalling)

    def stall(stage):
        return sum(getattr(stalling, entry)(stage) for entry in entries)

    try:
        assert stall(at) == 0
        assert w4.read_error_word(clear=True) == 0
        got = call(torch.zeros(shape, dtype=dtype, device="cuda"))
        word = w4.read_error_word(clear=True)
        nan = torch.isnan(got.float())
        wrong = ~nan & (got != want)
        assert not bool(wrong.any()), f"{int(wrong.sum())} elements neither right nor NaN"
        # a stage that no run has stalls nothing
        assert bool(nan.any()) == bool(word & w4.ERROR_WAIT_TIMEOUT)
        if at == 0:
            assert bool(nan.any())
    finally:
        assert stall(-1) == 0
    # the context stays usable and the next call is right
    assert torch.equal(call(torch.zeros(shape, dtype=dtype, device="cuda")), want)
    assert w4.read_error_word(clear=True) == 0


# few rows: one CTA a tile, clusters that share one, several tiles a CTA; many rows: pairs,
# single CTAs, clusters that share a tile
@pytest.mark.parametrize("at", [0, 1, 7])
@pytest.mark.parametrize("M,N,K", [(16, 40000, 640), (3, 2560, 4096), (100, 1024, 4096), (64, 90000, 256),
                                   (4096, 4096, 1280), (300, 9000, 1280), (512, 2560, 9728)])
def test_products(stalling, monkeypatch, M, N, K, at):
    for transposed in (False, True):
        args = problem(torch.Generator(device="cuda").manual_seed(M), M, N, K, transposed)
        run(stalling, monkeypatch, PRODUCTS, at,
            lambda out: w4.gemm_fp8(*args, transposed=transposed, out=out), (M, K if transposed else N), torch.bfloat16)


@pytest.mark.parametrize("at", [0, 2, 9])
@pytest.mark.parametrize("M", [200, 9000])
def test_grouped(stalling, monkeypatch, M, at):
    E, N, K = 16, 1000, 640
    args = problem(torch.Generator(device="cuda").manual_seed(M), M, N, K, False, E)
    ids = torch.randint(0, E, (M,), generator=torch.Generator().manual_seed(1))
    sizes = torch.bincount(ids, minlength=E).to(torch.int32).cuda()
    run(stalling, monkeypatch, PRODUCTS, at, lambda out: w4.gemm_fp8_grouped(*args, sizes, out=out)[0], (M, N),
        torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0, 1, 6])
@pytest.mark.parametrize("sizes,N,K", [([300, 0, 77, 1000], 2000, 2048), ([5000], 512, 512), ([64, 128], 256, 256)])
def test_weight_gradients(stalling, monkeypatch, sizes, N, K, at, dtype):
    g = torch.Generator(device="cuda").manual_seed(N)
    dy = torch.randn(sum(sizes), N, device="cuda", generator=g).bfloat16()
    x = torch.randn(sum(sizes), K, device="cuda", generator=g).bfloat16()
    m = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    call = lambda out: w4.gemm_grouped_wgrad(dy, x, m, dtype=dtype, out=out)[0]  # noqa: E731
    shape = (len(sizes), N, K)
    run(stalling, monkeypatch, ("w4a16_test_stall_wgrad",), at, call, shape, dtype)
