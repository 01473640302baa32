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


def kernel_parts(text, name):
    """The names of the kernel's parameters, and its body."""
    at = re.search(r"\b%s\(([^)]*)\)" % name, text[text.index("__global__"):])
    names = [v.split()[-1].lstrip("*") for v in at.group(1).split(",")]
    start = text.index("{", text.index("__global__") + at.end()) + 1
    depth = 1
    for j in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return names, text[start:j]
    raise AssertionError("unbalanced braces")


# kernel -> the kernel that may run right before it in a call (None: it comes first)
CHAIN = {
    "routing.cu": {"sort_count_kernel": None, "sort_rank_kernel": None, "dispatch_copy_kernel": "sort_rank_kernel",
                   "dispatch_few_kernel": None, "combine_kernel": None, "combine_backward_kernel": None},
    "lora.cu": {"lora_few_kernel": None},
    "lora_tensor.cu": {"lora_down_kernel": "sort_rank_kernel", "lora_sum_kernel": "lora_down_kernel",
                       "lora_up_kernel": "lora_sum_kernel", "lora_wgrad_kernel": "lora_sum_kernel",
                       "wgrad_sum_kernel": "lora_up_kernel"}}


def test_chained_kernels_wait_before_they_let_the_next_one_start():
    """What a kernel reads before its own wait rests on its predecessor having waited
    before letting it start; the two that let it start first are followed by kernels
    that rely on the launch before those alone, which has to have waited."""
    waits_first = {}
    for name, kernels in CHAIN.items():
        text = source(name)
        assert len(re.findall(r"__global__", text)) == len(kernels)
        for kernel, before in kernels.items():
            names, body = kernel_parts(text, kernel)
            wait, trigger = body.index("pdl_wait();"), body.index("pdl_launch_dependents();")
            waits_first[kernel] = wait < trigger
            if before is None:                           # no argument is looked at before the wait
                assert not re.search(r"\b(%s)\b" % "|".join(names), body[:wait]), kernel
    assert {k for k, first in waits_first.items() if not first} == {"lora_sum_kernel", "wgrad_sum_kernel"}
    # the launch before the early one waits first
    for early in ("lora_sum_kernel", "wgrad_sum_kernel"):
        before = next(v[early] for v in CHAIN.values() if early in v)
        assert waits_first[before]
