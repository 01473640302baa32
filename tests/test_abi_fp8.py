"""Argument checks of the 8-bit entry points and of the weights' gradients, on the host
(no GPU), and what their sources and resources have to keep."""
from __future__ import annotations

import os
import re

import pytest

from bf16_activation_quantized_gb300 import _lib
from bf16_activation_quantized_gb300 import build as build_mod

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = 1 << 20    # aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    build_mod.build()
    return _lib.lib()


def quantize(L, X=FAKE, c=FAKE, s=FAKE, rows=4, width=128):
    return L.w4a16_quantize_fp8(X, c, s, rows, width, None)


def quantize_blocks(L, W=FAKE, c=FAKE, s=FAKE, G=1, N=4, K=128):
    return L.w4a16_quantize_fp8_blocks(W, c, s, G, N, K, None)


def gemm(L, X=FAKE, xs=FAKE, W=FAKE, ws=FAKE, Y=FAKE, M=4, N=64, K=128, t=0, flags=0):
    return L.w4a16_gemm_fp8(X, xs, W, ws, Y, M, N, K, t, flags, None)


def grouped(L, X=FAKE, xs=FAKE, W=FAKE, ws=FAKE, sizes=FAKE, Y=FAKE, G=2, M=4, N=64, K=128, t=0, status=FAKE):
    return L.w4a16_gemm_fp8_grouped(X, xs, W, ws, sizes, Y, G, M, N, K, t, status, None)


def wgrad(L, dY=FAKE, X=FAKE, sizes=FAKE, dW=FAKE, b=4, G=2, M=4, N=64, K=128, status=FAKE):
    return L.w4a16_gemm_grouped_wgrad(dY, X, sizes, dW, b, G, M, N, K, status, None)


@pytest.mark.parametrize("bad", [dict(X=None), dict(c=None), dict(s=None), dict(X=FAKE + 1), dict(c=FAKE + 8),
                                 dict(s=FAKE + 2), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(width=0),
                                 dict(width=(1 << 20) + 1)])
def test_quantize_refuses(L, bad):
    assert quantize(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(W=None), dict(c=None), dict(s=None), dict(W=FAKE + 8), dict(c=FAKE + 8),
                                 dict(s=FAKE + 2), dict(G=0), dict(G=1025), dict(N=0), dict(N=(1 << 24) + 1),
                                 dict(K=0), dict(K=64), dict(K=200), dict(K=(1 << 20) + 128)])
def test_quantize_blocks_refuses(L, bad):
    assert quantize_blocks(L, **bad) == INVALID


PRODUCT = [dict(X=None), dict(xs=None), dict(W=None), dict(ws=None), dict(Y=None), dict(X=FAKE + 8), dict(W=FAKE + 8),
           dict(xs=FAKE + 2), dict(ws=FAKE + 2), dict(Y=FAKE + 1), dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0),
           dict(N=(1 << 24) + 1), dict(K=0), dict(K=64), dict(K=192), dict(K=(1 << 20) + 128),
           dict(N=(1 << 20) + 1, t=1), dict(M=1 << 24, N=1 << 17)]


@pytest.mark.parametrize("bad", PRODUCT + [dict(flags=2), dict(flags=-1)])
def test_gemm_refuses(L, bad):
    assert gemm(L, **bad) == INVALID


@pytest.mark.parametrize("bad", PRODUCT + [dict(sizes=None), dict(status=None), dict(sizes=FAKE + 2),
                                           dict(status=FAKE + 2), dict(G=0), dict(G=1025)])
def test_grouped_refuses(L, bad):
    assert grouped(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(dY=None), dict(X=None), dict(sizes=None), dict(dW=None), dict(status=None),
                                 dict(dY=FAKE + 8), dict(X=FAKE + 8), dict(dW=FAKE + 8), dict(sizes=FAKE + 2),
                                 dict(status=FAKE + 2), dict(G=0), dict(G=1025), dict(M=-1), dict(M=(1 << 24) + 1),
                                 dict(N=0), dict(K=0), dict(N=1 << 24, K=1 << 18)])
def test_wgrad_refuses(L, bad):
    assert wgrad(L, **bad) == INVALID


@pytest.mark.parametrize("bad", [dict(b=8), dict(b=1), dict(N=68), dict(K=4)])
def test_wgrad_unsupported(L, bad):
    assert wgrad(L, **bad) == UNSUPPORTED


def test_no_rows(L):
    assert quantize(L, rows=0, X=None, c=None, s=None) == OK
    assert gemm(L, M=0, X=None, xs=None, W=None, ws=None, Y=None) == OK


def test_python_refuses():
    import torch
    import bf16_activation_quantized_gb300 as w4
    f8 = torch.float8_e4m3fn
    x, w = torch.zeros(2, 128).to(f8), torch.zeros(4, 128).to(f8)
    xs, ws = torch.zeros(1, 2), torch.zeros(1, 1)
    sizes = torch.zeros(1, dtype=torch.int32)
    rows = torch.zeros(2, 128, dtype=torch.bfloat16)
    for call in (lambda: w4.quantize_fp8(rows), lambda: w4.quantize_fp8(rows, blocks=True),
                 lambda: w4.gemm_fp8(x, xs, w, ws), lambda: w4.gemm_fp8_grouped(x, xs, w[None], ws[None], sizes),
                 lambda: w4.gemm_grouped_wgrad(rows, rows, sizes)):
        with pytest.raises(ValueError):
            call()
    for op in (w4.gemm_fp8, w4.gemm_fp8_grouped):
        assert "Not recorded for autograd" in op.__doc__


# ------------------------------------------------------- sources and resources
def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(build_mod.CSRC, name)).read())


@pytest.fixture(scope="module")
def report():
    build_mod.build()
    path = os.path.join(build_mod.BUILD, "ptxas.log")
    if not os.path.exists(path):
        build_mod.build(force=True)
    out, name = {}, None
    for line in open(path).read().splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            name = m.group(1)
        elif name and "spill stores" in line:
            out.setdefault(name, {})["spill"] = int(re.search(r"(\d+) bytes spill stores", line).group(1))
        elif name and re.search(r"Used \d+ registers", line):
            out.setdefault(name, {})["regs"] = int(re.search(r"Used (\d+) registers", line).group(1))
            name = None
    return out


@pytest.mark.parametrize("kernel", ["quantize_rows_kernel", "quantize_blocks_kernel", "fp8_gemm_kernel", "fp8_many_kernel",
                                    "grouped_wgrad_kernel"])
def test_no_spills(report, kernel):
    hits = {k: v for k, v in report.items() if kernel in k}
    assert hits
    for name, r in hits.items():
        assert r["spill"] == 0, name


@pytest.mark.parametrize("file,threads,kernel", [("fp8_many.cu", "kManyThreads", "fp8_many_kernel"),
                                                 ("wgrad.cu", "kWgThreads", "grouped_wgrad_kernel")])
def test_register_shares_fit_the_launch(report, file, threads, kernel):
    """setmaxnreg waits until the block's registers at launch cover what it asks for: a share
    above them would wait forever."""
    text = source(file)
    threads = int(re.search(threads + r" = (\d+)", text).group(1))
    few, more = (int(v) for v in re.search(r"kRegsIn = (\d+), kRegsAdd = (\d+)", text).groups())
    hits = {k: v["regs"] for k, v in report.items() if kernel in k}
    assert hits
    for name, regs in hits.items():
        assert regs == 168, name
        assert 128 * few + (threads - 128) * more <= regs * threads
    assert text.count("setmaxnreg") == 2


@pytest.mark.parametrize("name,kernels", [("fp8.cu", 2), ("fp8_gemm.cu", 1), ("fp8_many.cu", 1), ("wgrad.cu", 1),
                                          ("groups.cu", 1)])
def test_kernels_wait_before_they_let_the_next_one_start(name, kernels):
    text = source(name)
    starts = [m.start() for m in re.finditer(r"__global__", text)]
    assert len(starts) == kernels
    for at in starts:
        assert 0 < text.index("pdl_wait();", at) < text.index("pdl_launch_dependents();", at)


def test_mma_warps_wait_for_the_sums_before_the_ring():
    """Two warps issue every second block's MMAs.  With an odd ring each meets a ring slot every
    second lap, where the slot's parity alone also fits two laps before; the wait for the
    block kSlots back rules that out, if it comes first and the ring is not shorter."""
    text = source("fp8_gemm.cu")
    part = text[text.index("} else if (warp <= 2) {"):text.index("} else if (warp < kAddWarp0) {")]
    assert part.index("mbar_wait(dempty") < part.index("mbar_wait(full")
    assert "if (a.stages % 2 && a.stages < kSlots) --a.stages;" in text


def walk(ring, slots, seed, waits, blocks=23):
    """The waits of the producer, the two MMA warps and the adding warps on a model of the
    barriers, in a random order that they allow, copies landing in any order: fails where a
    warp passes a wait whose phase is not over.  waits: an MMA warp's, in order."""
    full, empty, dfull, dempty = [0] * ring, [0] * ring, [0] * slots, [0] * slots        # phases over
    loads, add, mma, at, lap, step = 0, 0, [0, 1], [0, 1], [0, 0], [0, 0]
    issued, flying, landed = set(), [], set()

    def over(phases, parity):
        return phases % 2 != parity

    for _ in range(8000):
        seed = (seed * 1103515245 + 12345) % 2**31
        who = (seed >> 16) % 5
        if who == 0 and loads < blocks:
            if loads < ring or over(empty[loads % ring], (loads // ring - 1) % 2):
                assert all(b % ring != loads % ring for b in flying), (ring, loads)
                flying.append(loads)
                loads += 1
        elif who == 4 and flying:
            b = flying.pop((seed >> 8) % len(flying))
            full[b % ring] += 1
            landed.add(b)
        elif who in (1, 2) and mma[who - 1] < blocks:
            w, i = who - 1, mma[who - 1]
            d, s = i % slots, at[w]
            if waits[step[w]] == "dempty":
                step[w] += i < slots or over(dempty[d], (i // slots - 1) % 2)
            else:
                step[w] += over(full[s], lap[w])
            if step[w] == 2:
                assert i in landed, (ring, i)
                issued.add(i)
                empty[s] += 1
                dfull[d] += 1
                step[w], mma[w], at[w] = 0, i + 2, s + 2
                if at[w] >= ring:
                    at[w] -= ring
                    lap[w] ^= 1
        elif who == 3 and add < blocks and over(dfull[add % slots], add // slots % 2):
            assert add in issued, (ring, add)
            dempty[add % slots] += 1
            add += 1
    assert add == blocks, (ring, add)


def test_ring_walks_never_pass_a_landing_copy():
    slots = int(re.search(r"kSlots = (\d+);", source("fp8_gemm.cu")).group(1))
    for ring in (2, 4, 5, 6, 7, 9, 16):
        for order in range(40):
            walk(ring, slots, order * 7919 + ring, ("dempty", "full"))
    # the model sees the other order's fault, and that of a shorter odd ring
    for ring, waits in ((5, ("full", "dempty")), (3, ("dempty", "full"))):
        with pytest.raises(AssertionError):
            for order in range(200):
                walk(ring, slots, order * 7919 + ring, waits)
