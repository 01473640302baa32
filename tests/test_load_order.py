"""Loads of global memory in inline assembly, read on the host.

A kernel may be started while the one before it on the stream still writes its inputs;
griddepcontrol.wait is what it waits at.  An asm statement without ``volatile`` is to the
compiler a function of its operands alone, which it may move above that wait."""
from __future__ import annotations

import glob
import os
import re

import pytest

from bf16_activation_quantized_gb300 import build as build_mod

FILES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(build_mod.CSRC, "*.cu*")))


def statements(text):
    """(qualifier, text up to the outputs) of every asm statement."""
    text = re.sub(r"//[^\n]*", "", text)
    return re.findall(r"\basm\b\s*(volatile|)\s*\(((?:\s*\"[^\"]*\")+)", text)


@pytest.mark.parametrize("name", FILES)
def test_loads_of_memory_keep_their_place(name):
    found = statements(open(os.path.join(build_mod.CSRC, name)).read())
    loads = [(q, t) for q, t in found if re.search(r"\bld(\.|matrix)", t)]
    assert all(q == "volatile" for q, _ in loads), [t for q, t in loads if q != "volatile"]


def test_the_waits_keep_their_place():
    found = statements(open(os.path.join(build_mod.CSRC, "common.cuh")).read())
    waits = [q for q, t in found if "griddepcontrol" in t]
    assert waits == ["volatile", "volatile"]


def test_the_reader_sees_a_load_without_it():
    text = 'uint4 f() { asm("ld.global.nc.v4.u32 {%0}, [%1];" : "=r"(x) : "l"(p)); asm volatile("ld.global.u32 %0, [%1];" : : ); }'
    assert [q for q, t in statements(text)] == ["", "volatile"]
