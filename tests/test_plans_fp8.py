"""Which form the 8-bit products and the weights' gradients take, asked on the host: the rules
compiled by themselves, and the sizes of the GPU tests that are to reach each form."""
from __future__ import annotations

import ctypes
import subprocess

import pytest

from bf16_activation_quantized_gb300 import build as build_mod

from fp8_forms import GROUPED, PLAIN, WGRAD

SMS = 152


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    where = tmp_path_factory.mktemp("plans")
    src, lib = where / "plans.cc", where / "libplans.so"
    src.write_text("""
#include "split_plan.h"
extern "C" void plan(int M, int out, int blocks, int groups, int grouped, int sms, int *r) {
    const w4a16::Fp8Plan p = w4a16::fp8_plan(M, out, blocks, groups, grouped != 0, sms);
    r[0] = p.size, r[1] = p.pair, r[2] = p.split, r[3] = p.bt, r[4] = p.ctas, r[5] = p.occupancy;
}
extern "C" int wgrad(long long tiles, int pairs, int rows, int groups) {
    return w4a16::wgrad_split(tiles, pairs, rows, groups, 64);
}
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build_mod.CSRC, str(src), "-o", str(lib)],
                   check=True, capture_output=True)
    handle = ctypes.CDLL(str(lib))
    handle.wgrad.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return handle


def plan(rules, M, N, K, transposed, groups=None, sms=SMS):
    """(size, pair, split), rows of x a tile, CTAs."""
    r = (ctypes.c_int * 6)()
    n, k = -(-N // 128), K // 128
    rules.plan(M, K if transposed else N, n if transposed else k, groups or 1, int(groups is not None), sms, r)
    return (r[0], bool(r[1]), r[2]), r[3], r[4]


@pytest.mark.parametrize("form", PLAIN)
def test_plain_sizes_take_their_form(rules, form):
    for transposed, (M, N, K) in enumerate(PLAIN[form]):
        assert plan(rules, M, N, K, transposed)[0] == form
        blocks = -(-N // 128) if transposed else K // 128
        if form[2] > 1 and not form[1]:
            assert blocks % form[2] and blocks >= 2 * form[2]


@pytest.mark.parametrize("form", GROUPED)
def test_grouped_sizes_take_their_form(rules, form):
    for transposed, (M, groups, N, K) in enumerate(GROUPED[form]):
        assert plan(rules, M, N, K, transposed, groups)[0] == form
        blocks = -(-N // 128) if transposed else K // 128
        if form[2] > 1 and not form[1]:
            assert blocks % form[2] and blocks >= 2 * form[2]


@pytest.mark.parametrize("split", WGRAD)
def test_gradients_take_their_form(rules, split):
    for sizes, N, K in WGRAD[split]:
        tiles = len(sizes) * -(-N // 256) * -(-K // 256)
        assert rules.wgrad(tiles, SMS // 2, sum(sizes), len(sizes)) == split


def test_a_cluster_has_one_tile_at_most(rules):
    """Tiles are counted from above before the sizes are known: whatever the sizes, no cluster
    that shares a tile's sum has to take a second one."""
    seed = 1
    shared = 0
    for _ in range(4000):
        seed = (seed * 6364136223846793005 + 1442695040888963407) % 2**64
        groups, M = (1, 2, 3, 8, 40)[seed >> 60 & 3], 1 + (seed >> 20) % 1500
        N, K = 1 + (seed >> 33) % 3000, 128 * (1 + (seed >> 48) % 90)
        form, bt, ctas = plan(rules, M, N, K, False, groups)
        if form[2] == 1 or form[1]:
            continue
        shared += 1
        cols = -(-N // (128 if form[0] else 256))
        worst = 0
        for lead in (1, bt - 1, bt, bt + 1, M // groups, M):     # one group's rows, the rest evenly
            first = min(lead, M)
            rest = M - first
            sizes = [first] + ([rest // (groups - 1)] * (groups - 1) if groups > 1 else [])
            if groups > 1:
                sizes[-1] += M - sum(sizes)
            worst = max(worst, sum(-(-s // bt) for s in sizes) * cols)
        assert worst * form[2] <= ctas, (M, groups, N, K)
    assert shared > 300
