"""Resource report of the dispatch, combine and adapter kernels (ptxas -v of the
sm_103a build): none may spill, and those launched two to an SM must fit."""
from __future__ import annotations

import os
import re

import pytest

from bf16_activation_quantized_gb300 import build as build_mod


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


@pytest.mark.parametrize("kernel,regs", [
    ("sort_count_kernel", 64), ("sort_rank_kernel", 64), ("dispatch_few_kernel", 64), ("dispatch_copy_kernel", 64),
    ("combine_kernel", 64), ("combine_backward_kernel", 64), ("lora_few_kernelILi16", 128),
    ("lora_few_kernelILi32", 128), ("lora_few_kernel", 255), ("lora_down_kernel", 152), ("lora_sum_kernel", 64),
    ("lora_up_kernel", 152), ("lora_wgrad_kernel", 152), ("wgrad_sum_kernel", 64)])
def test_no_spills(report, kernel, regs):
    hits = {k: v for k, v in report.items() if kernel in k}
    assert hits, kernel
    for name, r in hits.items():
        assert r["spill"] == 0, name
        assert r["regs"] <= regs, (name, r["regs"])
