"""What the adapter kernels' sources have to keep, read on the host: a breach would
show on a GPU, if at all, as a fault, a hang or a rare wrong value.

Instructions of a whole warp (``.aligned``) stand where its lanes have met: the
cluster barriers, which follow loops whose trip counts differ between lanes, and the
loads from tensor memory in loops whose bodies store under lane-dependent conditions."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from bf16_activation_quantized_gb300 import _lib
from bf16_activation_quantized_gb300 import build as build_mod


def source(name):
    text = open(os.path.join(build_mod.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def enclosing_loop(text, at):
    """The body of the innermost ``for`` around position ``at``."""
    depth, i = 0, at
    while i > 0:
        i -= 1
        if text[i] == "}":
            depth += 1
        elif text[i] == "{":
            if depth == 0:
                head = text[text.rfind("\n", 0, i) + 1:i]
                if head.lstrip().startswith("for ("):
                    break
            else:
                depth -= 1
    start, depth = i + 1, 1
    for j in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[start:j]
    raise AssertionError("unbalanced braces")


@pytest.mark.parametrize("name", ["arrive", "wait"])
def test_lanes_meet_before_a_cluster_barrier(name):
    body = re.search(r"void cluster_%s\(\) \{(.*?)\n\}" % name, source("lora.cuh"), re.S).group(1)
    assert body.index("__syncwarp();") < body.index("barrier.cluster.")


def test_lanes_meet_before_the_next_load_from_tensor_memory():
    text = source("lora_tensor.cu")
    calls = [m.start() for m in re.finditer(r"\btc_ld_\w+\(", text)]
    assert len(calls) >= 5
    for at in calls:
        assert enclosing_loop(text, at).rstrip().endswith("__syncwarp();"), text[at:at + 60]


def test_smoke_takes_both_forms_of_the_adapters():
    """The few-token form takes no workspace, the many-token form does."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "__graft_entry__.py")).read()
    sizes = [int(v) for v in re.search(r"for tokens in \((\d+), (\d+)\)", text).groups()]
    rank, adapters = 16, 3
    assert f"normal({adapters}, {rank}, 256" in text
    build_mod.build()
    need = ctypes.c_size_t(0)
    forms = []
    for tokens in sizes:
        assert _lib.lib().w4a16_lora_workspace_bytes(tokens, adapters, rank, 0, ctypes.byref(need)) == 0
        forms.append(need.value > 0)
    assert forms == [False, True]
