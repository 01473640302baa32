"""The Python binding of dispatch, combine and the adapters, on the host (no GPU)."""
from __future__ import annotations

import os
import subprocess
import sys

import bf16_activation_quantized_gb300 as w4
from bf16_activation_quantized_gb300 import build as build_mod

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_imports_with_a_torch_that_has_no_cuda():
    """Such a torch lacks the two calls; pack sizes, plans and host checks need neither."""
    code = ("import torch\n"
            "for name in ('_cuda_getCurrentRawStream', '_cuda_getDevice'):\n"
            "    if hasattr(torch._C, name): delattr(torch._C, name)\n"
            "import bf16_activation_quantized_gb300 as w4\n"
            "x = torch.zeros(2, 8, dtype=torch.bfloat16)\n"
            "try:\n"
            "    w4.dispatch(x, torch.zeros(2, 1, dtype=torch.int32), 2)\n"
            "except ValueError:\n"
            "    print('refused')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stdout + r.stderr


def test_sizes_kept_for_calls_are_bounded():
    """A server that meets every token count keeps no entry for each of them."""
    build_mod.build()
    for tokens in range(1, 5001):
        w4._sort_bytes(tokens, 8, 64)
        w4._lora_bytes(tokens, 4, 16, 1)
    for cached in (w4._sort_bytes, w4._lora_bytes):
        assert cached.cache_info().currsize <= 1024


def test_the_operators_say_that_autograd_does_not_see_them():
    for op, gradient in ((w4.dispatch, "dispatch_backward"), (w4.combine, "combine_backward"),
                         (w4.lora_add, "lora_add_backward")):
        assert "Not recorded for autograd" in op.__doc__ and gradient in op.__doc__
    assert "autograd" in w4.__doc__
