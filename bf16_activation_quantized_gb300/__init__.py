"""W4A16 skinny GEMM for GB300 (sm_103a): Python binding of the C ABI.

``Y[M, N] = X[M, K] . dequant(W)[N, K]^T`` with bf16 X and Y, int4 W packed two
codes per byte (low nibble = even k), one bf16 scale per G weights along K
(G = 128, 64 or 32, read off the scales' shape [N, K/G]),
``dequant = scale * (code - 8)``, fp32 accumulation.  Beside the products: rows to the
groups of the grouped product and back (``dispatch``, ``combine``), low-rank
adapters (``lora_add``), and products with rows and weights in 8-bit floating point
(``quantize_fp8``, ``gemm_fp8``, ``gemm_fp8_grouped``), with their gradients.

Every function here only checks tensor metadata, allocates outputs and
workspaces with torch, and calls the C ABI on the current torch stream: all
arithmetic runs in the library's CUDA kernels.  There is no CPU path; a call
with CPU tensors or without the built library raises.  Nothing is recorded for
autograd: results have no gradient function, whatever their inputs require, and a
gradient is what the ``*_backward`` call of an operator returns.
"""
from __future__ import annotations

import ctypes
import functools
import threading

import torch

from . import _lib
from ._lib import Options, PlanInfo, W4A16Error

GROUP = 128                  # default scale group size
GROUP_SIZES = (128, 64, 32)
ARM_AUTO, ARM_DECODE, ARM_TENSOR = 0, 1, 2
_ARMS = {None: ARM_AUTO, "auto": ARM_AUTO, "decode": ARM_DECODE, "tensor": ARM_TENSOR}

__all__ = ["GROUP", "pack", "gemm", "gemm_partials", "gemm_grouped", "gemm_batched", "plan_batched", "dequant_fp32", "dequant_bf16",
           "splitk_reduce", "dispatch", "dispatch_backward", "combine", "combine_backward",
           "lora_add", "lora_add_backward", "quantize_fp8", "gemm_fp8", "gemm_fp8_grouped", "gemm_grouped_wgrad", "plan", "packed_weight_bytes", "layout_version", "read_error_word",
           "ERROR_WAIT_TIMEOUT", "W4A16Error"]


def _stream_ptr(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need_cuda(t: torch.Tensor, name: str, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


FLAG_RESIDENT_WEIGHTS = 1
FLAG_DECODE_WHOLE_K = 2
FLAG_DECODE_K_SLICES = 4
FLAG_ZERO_POINTS = 8
FLAG_TEST_STALL = 16
ERROR_WAIT_TIMEOUT = 1       # error-word bit: a bounded wait in a kernel ran out
_KERNELS = {None: 0, "auto": 0, "whole_k": FLAG_DECODE_WHOLE_K, "k_slices": FLAG_DECODE_K_SLICES}


def _group_size(K: int, cols: int, what: str) -> int:
    """G from K and the scales' last dimension K / G (the library rejects G
    other than 128, 64 and 32)."""
    if cols <= 0 or K % cols or (K // cols) not in GROUP_SIZES:
        raise ValueError(f"{what} must have K/G columns with G in {GROUP_SIZES} (K={K}, got {cols})")
    return K // cols


def _opts(arm, split_k, tile_tokens, resident_weights=False, decode_kernel=None, zero_points=False,
          test_stall=False):
    if arm not in _ARMS:
        raise ValueError(f"arm must be one of {list(_ARMS)}")
    if decode_kernel not in _KERNELS:
        raise ValueError(f"decode_kernel must be one of {list(_KERNELS)}")
    flags = ((FLAG_RESIDENT_WEIGHTS if resident_weights else 0) | _KERNELS[decode_kernel]
             | (FLAG_ZERO_POINTS if zero_points else 0) | (FLAG_TEST_STALL if test_stall else 0))
    return Options(_ARMS[arm], int(split_k), int(tile_tokens), flags)


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def _workspace(device, nbytes: int) -> torch.Tensor:
    """A grow-only scratch buffer per device (contents need no initialisation)."""
    key = torch.device(device).index
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
        return buf


# Host-side answers that depend only on the shape, the options and the device
# (the plan depends on the device's SM count), cached so that a call costs one
# library call.
_plan_cache: dict = {}
_pwb_cache: dict = {}


def _workspace_need(M: int, N: int, K: int, G: int, o: Options, dev_index: int) -> int:
    key = (M, N, K, G, o.arm, o.split_k, o.tile_tokens, o.flags, dev_index)
    need = _plan_cache.get(key)
    if need is None:
        info = PlanInfo()
        _lib.check(_lib.lib().w4a16_plan(M, N, K, G, ctypes.byref(o), ctypes.byref(info)),
                   "w4a16_plan")
        need = int(info.workspace_bytes)
        _plan_cache[key] = need
    return need


def _plan_dict(info: PlanInfo) -> dict:
    return {"arm": {1: "decode", 2: "tensor"}.get(info.arm, info.arm), "split_k": info.split_k,
            "tile_tokens": info.tile_tokens, "ctas": info.ctas,
            "workspace_bytes": int(info.workspace_bytes), "whole_k": bool(info.whole_k)}


def layout_version() -> int:
    return int(_lib.lib().w4a16_layout_version())


def read_error_word(clear: bool = True, device=None) -> int:
    """The device error word (w4a16_read_error_word): OR of the ERROR_* bits
    the kernels recorded since it was last cleared; 0 means no kernel gave up.
    Waits for all work on the device first; ``clear`` resets the word."""
    v = ctypes.c_int(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _lib.check(_lib.lib().w4a16_read_error_word(ctypes.byref(v), 1 if clear else 0),
                   "w4a16_read_error_word")
    return int(v.value)


def packed_weight_bytes(N: int, K: int) -> int:
    key = (N, K)
    nb = _pwb_cache.get(key)
    if nb is None:
        nb = _pwb_cache[key] = int(_lib.lib().w4a16_packed_weight_bytes(N, K))
    return nb


def pack(w_canon: torch.Tensor) -> torch.Tensor:
    """Canonical uint8 [N, K/2] (CUDA) -> packed uint8 buffer for the kernels."""
    _need_cuda(w_canon, "w_canon", torch.uint8)
    N, half_k = w_canon.shape
    K = 2 * half_k
    nbytes = packed_weight_bytes(N, K)
    if nbytes == 0:
        raise ValueError(f"unsupported weight shape N={N} K={K} (K must be a multiple of 128)")
    out = torch.empty(nbytes, dtype=torch.uint8, device=w_canon.device)
    with torch.cuda.device(w_canon.device):
        _lib.check(_lib.lib().w4a16_pack_weights(w_canon.data_ptr(), out.data_ptr(), N, K,
                                                 _stream_ptr(w_canon.device)), "w4a16_pack_weights")
    return out


def plan(M: int, N: int, K: int, arm=None, split_k: int = 0, tile_tokens: int = 0,
         device=None, decode_kernel=None, group_size: int = GROUP,
         zero_points: bool = False, sms: int | None = None) -> dict:
    """What the dispatcher picks for this shape on the (current) device, or,
    with ``sms``, on a device with that many SMs (host only, no GPU needed)."""
    info = PlanInfo()
    o = _opts(arm, split_k, tile_tokens, decode_kernel=decode_kernel, zero_points=zero_points)
    if sms is not None:
        _lib.check(_lib.lib().w4a16_plan_for_sms(int(sms), 1, M, N, K, group_size, ctypes.byref(o),
                                                 ctypes.byref(info)), "w4a16_plan_for_sms")
        return _plan_dict(info)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _lib.check(_lib.lib().w4a16_plan(M, N, K, group_size, ctypes.byref(o), ctypes.byref(info)),
                   "w4a16_plan")
    return _plan_dict(info)


def gemm(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, *, arm=None,
         split_k: int = 0, tile_tokens: int = 0, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, resident_weights: bool = False,
         decode_kernel=None, zeros: torch.Tensor | None = None,
         test_stall: bool = False) -> torch.Tensor:
    """Y = X . dequant(W)^T.  x: bf16 [M, K]; scales: bf16 [N, K/G]; returns bf16 [M, N].

    ``zeros`` (uint8 [N, K/G], low four bits) selects the zero-point variant,
    dequant = scale * (code - z) (w4a16_gemm_zp); without it z is 8.

    ``resident_weights=True`` promises that no kernel still running on the
    current stream writes ``w_packed`` or ``scales`` (W4A16_FLAG_RESIDENT_WEIGHTS):
    the call may then start streaming them before the previous kernel ends.
    ``decode_kernel`` ("whole_k" or "k_slices") forces the decode arm's kernel.
    ``test_stall`` (tests only, W4A16_FLAG_TEST_STALL) makes the decode kernel's
    bounded waits run out: the outputs become NaN and the error word is set."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(scales, "scales", torch.bfloat16)
    _need_cuda(w_packed, "w_packed", torch.uint8)
    M, K = x.shape
    N = scales.shape[0]
    G = _group_size(K, scales.shape[1], "scales [N, K/G]")
    if w_packed.numel() < packed_weight_bytes(N, K):
        raise ValueError("w_packed is smaller than packed_weight_bytes(N, K)")
    if zeros is not None:
        _need_cuda(zeros, "zeros", torch.uint8)
        if tuple(zeros.shape) != tuple(scales.shape):
            raise ValueError("zeros must be uint8 [N, K/G], the shape of scales")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _need_cuda(out, "out", torch.bfloat16)
    o = _opts(arm, split_k, tile_tokens, resident_weights, decode_kernel, zeros is not None,
              test_stall)
    L = _lib.lib()
    dev = x.device
    switch = dev.index != torch.cuda.current_device()
    if switch:
        prev = torch.cuda.current_device()
        torch.cuda.set_device(dev)
    try:
        need = _workspace_need(M, N, K, G, o, dev.index)
        if workspace is None:
            ws = _workspace(dev, need) if need else None
        else:
            ws = workspace
        ws_ptr = ws.data_ptr() if ws is not None else None
        ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
        stream = torch.cuda.current_stream(dev).cuda_stream
        if zeros is None:
            _lib.check(L.w4a16_gemm_ex(x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(),
                                       out.data_ptr(), M, N, K, G, ws_ptr, ws_bytes,
                                       ctypes.byref(o), stream), "w4a16_gemm_ex")
        else:
            _lib.check(L.w4a16_gemm_zp(x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(),
                                       zeros.data_ptr(), out.data_ptr(), M, N, K, G, ws_ptr,
                                       ws_bytes, ctypes.byref(o), stream), "w4a16_gemm_zp")
    finally:
        if switch:
            torch.cuda.set_device(prev)
    return out


def gemm_partials(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, *,
                  out: torch.Tensor, workspace: torch.Tensor, arm=None, split_k: int = 0,
                  tile_tokens: int = 0, resident_weights: bool = False) -> int:
    """First launch of gemm() only (see w4a16_gemm_partials); returns SPLIT_K.

    With SPLIT_K > 1 the fp32 partial sums land in ``workspace`` as
    [SPLIT_K, M, N] and ``out`` is untouched; splitk_reduce() finishes the call."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(scales, "scales", torch.bfloat16)
    _need_cuda(w_packed, "w_packed", torch.uint8)
    _need_cuda(out, "out", torch.bfloat16)
    _need_cuda(workspace, "workspace")
    M, K = x.shape
    N = scales.shape[0]
    G = _group_size(K, scales.shape[1], "scales [N, K/G]")
    o = _opts(arm, split_k, tile_tokens, resident_weights)
    sk = ctypes.c_int(0)
    with torch.cuda.device(x.device):
        _lib.check(_lib.lib().w4a16_gemm_partials(
            x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(), out.data_ptr(), M, N, K, G,
            workspace.data_ptr(), workspace.numel() * workspace.element_size(), ctypes.byref(o),
            ctypes.byref(sk), _stream_ptr(x.device)), "w4a16_gemm_partials")
    return int(sk.value)


def plan_batched(batch: int, M: int, N: int, K: int, arm=None, split_k: int = 0,
                 tile_tokens: int = 0, device=None, decode_kernel=None,
                 group_size: int = GROUP, zero_points: bool = False) -> dict:
    """What the dispatcher picks for a batch of ``batch`` products of shape (M, N, K)."""
    info = PlanInfo()
    o = _opts(arm, split_k, tile_tokens, decode_kernel=decode_kernel, zero_points=zero_points)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _lib.check(_lib.lib().w4a16_plan_batched(batch, M, N, K, group_size, ctypes.byref(o),
                                                 ctypes.byref(info)), "w4a16_plan_batched")
    return _plan_dict(info)


def gemm_batched(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor, *, arm=None,
                 split_k: int = 0, tile_tokens: int = 0, out: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, resident_weights: bool = False,
                 decode_kernel=None, zeros: torch.Tensor | None = None) -> torch.Tensor:
    """Y[b] = X[b] . dequant(W[b])^T for every b in one launch.

    x: bf16 [B, M, K]; w_packed: uint8 [B, packed_weight_bytes(N, K)] (or the same
    bytes flat); scales: bf16 [B, N, K/G]; returns bf16 [B, M, N].  ``zeros``
    (uint8 [B, N, K/G]) selects the zero-point variant (w4a16_gemm_batched_zp)."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(scales, "scales", torch.bfloat16)
    _need_cuda(w_packed, "w_packed", torch.uint8)
    if x.dim() != 3 or scales.dim() != 3:
        raise ValueError("x must be [B, M, K] and scales [B, N, K/G]")
    B, M, K = x.shape
    N = scales.shape[1]
    if scales.shape[0] != B:
        raise ValueError("scales must be [B, N, K/G]")
    G = _group_size(K, scales.shape[2], "scales [B, N, K/G]")
    if w_packed.numel() < B * packed_weight_bytes(N, K):
        raise ValueError("w_packed is smaller than B * packed_weight_bytes(N, K)")
    if out is None:
        out = torch.empty((B, M, N), dtype=torch.bfloat16, device=x.device)
    else:
        _need_cuda(out, "out", torch.bfloat16)
    if zeros is not None:
        _need_cuda(zeros, "zeros", torch.uint8)
        if tuple(zeros.shape) != tuple(scales.shape):
            raise ValueError("zeros must be uint8 [B, N, K/G], the shape of scales")
    o = _opts(arm, split_k, tile_tokens, resident_weights, decode_kernel, zeros is not None)
    with torch.cuda.device(x.device):
        info = PlanInfo()
        _lib.check(_lib.lib().w4a16_plan_batched(B, M, N, K, G, ctypes.byref(o), ctypes.byref(info)),
                   "w4a16_plan_batched")
        need = int(info.workspace_bytes)
        ws = workspace if workspace is not None else (_workspace(x.device, need) if need else None)
        args = (ws.data_ptr() if ws is not None else None,
                ws.numel() * ws.element_size() if ws is not None else 0, ctypes.byref(o),
                _stream_ptr(x.device))
        if zeros is None:
            _lib.check(_lib.lib().w4a16_gemm_batched(
                x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(), out.data_ptr(), B, M, N, K, G,
                *args), "w4a16_gemm_batched")
        else:
            _lib.check(_lib.lib().w4a16_gemm_batched_zp(
                x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                out.data_ptr(), B, M, N, K, G, *args), "w4a16_gemm_batched_zp")
    return out


def gemm_grouped(x: torch.Tensor, w_packed: torch.Tensor, scales: torch.Tensor,
                 m_sizes: torch.Tensor, *, out: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, zeros: torch.Tensor | None = None):
    """Grouped product in one launch.

    x: bf16 [M_total, K]; w_packed: num_groups packed blocks; scales: bf16
    [num_groups, N, K/G]; m_sizes: int32 [num_groups] on the device (never
    read on the host).  ``zeros`` (uint8 [num_groups, N, K/G]) selects the
    zero-point variant (w4a16_gemm_grouped_zp).  Returns (Y bf16 [M_total, N],
    status int32 tensor whose element 0 the kernel sets; 0 = sizes consistent)."""
    _need_cuda(x, "x", torch.bfloat16)
    _need_cuda(scales, "scales", torch.bfloat16)
    _need_cuda(w_packed, "w_packed", torch.uint8)
    _need_cuda(m_sizes, "m_sizes", torch.int32)
    M_total, K = x.shape
    NG, N, kg = scales.shape
    if m_sizes.numel() != NG:
        raise ValueError("scales must be [num_groups, N, K/G] and m_sizes [num_groups]")
    G = _group_size(K, kg, "scales [num_groups, N, K/G]")
    if w_packed.numel() < NG * packed_weight_bytes(N, K):
        raise ValueError("w_packed is smaller than num_groups * packed_weight_bytes(N, K)")
    if out is None:
        out = torch.empty((M_total, N), dtype=torch.bfloat16, device=x.device)
    L = _lib.lib()
    with torch.cuda.device(x.device):
        nb = ctypes.c_size_t(0)
        _lib.check(L.w4a16_grouped_workspace_bytes(NG, M_total, N, K, G, ctypes.byref(nb)),
                   "w4a16_grouped_workspace_bytes")
        if status is None:
            status = torch.empty(max(4, (nb.value + 3) // 4), dtype=torch.int32, device=x.device)
        if zeros is None:
            _lib.check(L.w4a16_gemm_grouped(x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(),
                                            m_sizes.data_ptr(), out.data_ptr(), NG, M_total, N, K,
                                            G, status.data_ptr(), status.numel() * 4,
                                            _stream_ptr(x.device)), "w4a16_gemm_grouped")
        else:
            _need_cuda(zeros, "zeros", torch.uint8)
            if tuple(zeros.shape) != tuple(scales.shape):
                raise ValueError("zeros must be uint8 [num_groups, N, K/G], the shape of scales")
            _lib.check(L.w4a16_gemm_grouped_zp(x.data_ptr(), w_packed.data_ptr(), scales.data_ptr(),
                                               zeros.data_ptr(), m_sizes.data_ptr(), out.data_ptr(),
                                               NG, M_total, N, K, G, status.data_ptr(),
                                               status.numel() * 4, _stream_ptr(x.device)),
                       "w4a16_gemm_grouped_zp")
    return out, status


def dequant_fp32(w_packed: torch.Tensor, scales: torch.Tensor,
                 group_size: int = GROUP, zeros: torch.Tensor | None = None) -> torch.Tensor:
    """fp32 [N, K] = scale * (code - 8), computed by the kernels' bit trick;
    scales bf16 [N, K/G] with G = group_size; with ``zeros`` (uint8 [N, K/G])
    scale * (code - z)."""
    _need_cuda(w_packed, "w_packed", torch.uint8)
    _need_cuda(scales, "scales", torch.bfloat16)
    N, kg = scales.shape
    K = kg * group_size
    out = torch.empty((N, K), dtype=torch.float32, device=scales.device)
    with torch.cuda.device(scales.device):
        if zeros is None:
            _lib.check(_lib.lib().w4a16_dequant_fp32(w_packed.data_ptr(), scales.data_ptr(),
                                                     out.data_ptr(), N, K, group_size,
                                                     _stream_ptr(scales.device)), "w4a16_dequant_fp32")
        else:
            _need_cuda(zeros, "zeros", torch.uint8)
            _lib.check(_lib.lib().w4a16_dequant_zp_fp32(w_packed.data_ptr(), scales.data_ptr(),
                                                        zeros.data_ptr(), out.data_ptr(), N, K,
                                                        group_size, _stream_ptr(scales.device)),
                       "w4a16_dequant_zp_fp32")
    return out


def dequant_bf16(w_packed: torch.Tensor, scales: torch.Tensor,
                 group_size: int = GROUP, zeros: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [N, K] = round_nearest_even(scale * (code - 8)): the tensor arm's
    operand; scales bf16 [N, K/G] with G = group_size; with ``zeros``
    scale * (code - z)."""
    _need_cuda(w_packed, "w_packed", torch.uint8)
    _need_cuda(scales, "scales", torch.bfloat16)
    N, kg = scales.shape
    K = kg * group_size
    out = torch.empty((N, K), dtype=torch.bfloat16, device=scales.device)
    with torch.cuda.device(scales.device):
        if zeros is None:
            _lib.check(_lib.lib().w4a16_dequant_bf16(w_packed.data_ptr(), scales.data_ptr(),
                                                     out.data_ptr(), N, K, group_size,
                                                     _stream_ptr(scales.device)), "w4a16_dequant_bf16")
        else:
            _need_cuda(zeros, "zeros", torch.uint8)
            _lib.check(_lib.lib().w4a16_dequant_zp_bf16(w_packed.data_ptr(), scales.data_ptr(),
                                                        zeros.data_ptr(), out.data_ptr(), N, K,
                                                        group_size, _stream_ptr(scales.device)),
                       "w4a16_dequant_zp_bf16")
    return out


def splitk_reduce(ws: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [M, N] = sum over slices of fp32 ws [S, M, N] (slices in order)."""
    _need_cuda(ws, "ws", torch.float32)
    S, M, N = ws.shape
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=ws.device)
    with torch.cuda.device(ws.device):
        _lib.check(_lib.lib().w4a16_splitk_reduce(ws.data_ptr(), out.data_ptr(), S, M, N,
                                                  _stream_ptr(ws.device)), "w4a16_splitk_reduce")
    return out


# The current stream's handle and the current device without the objects around
# them: a call of a few microseconds spends a third of its time there otherwise.
# (A torch without CUDA has neither; its tensors never get past the checks.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _empty(shape, dtype, index: int) -> torch.Tensor:
    return torch.empty(shape, dtype=dtype, device=index)


def _launch(name: str, index: int, *args) -> None:
    """One library call on the current torch stream of device ``index``."""
    fn = getattr(_lib._lib or _lib.lib(), name)
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(status, name)


def _need_int32(*sizes: int) -> None:
    """The C ABI takes sizes as 32-bit integers; ctypes would drop the upper bits."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"a size is past 32 bits: {sizes}")


def _need_on(index: int, t: torch.Tensor, name: str, dtype=None) -> None:
    """``t`` is a contiguous tensor of ``dtype`` on CUDA device ``index``."""
    if (isinstance(t, torch.Tensor) and (dtype is None or t.dtype == dtype) and t.is_contiguous()
            and t.get_device() == index):
        return
    _need_cuda(t, name, dtype)
    raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _index_of(t: torch.Tensor, name: str, dtype) -> int:
    """The CUDA device of ``t``, a contiguous tensor of ``dtype``."""
    _need_cuda(t, name, dtype)
    return t.get_device()


# The workspaces' sizes are kept for the sizes used last: a call then costs one library
# call, and a server that meets every token count holds no entry for each.
@functools.lru_cache(maxsize=1024)
def _sort_bytes(tokens: int, top_k: int, num_groups: int) -> int:
    nb = ctypes.c_size_t(0)
    _lib.check(_lib.lib().w4a16_dispatch_workspace_bytes(tokens, top_k, num_groups, ctypes.byref(nb)),
               "w4a16_dispatch_workspace_bytes")
    return int(nb.value)


def dispatch(x: torch.Tensor, ids: torch.Tensor, num_groups: int):
    """Copy every token's row to the groups (experts) its ids name, in group order.

    x: bf16 [T, K]; ids: int32 or int64 [T, k], an id outside [0, num_groups)
    drops its slot.  Returns (xs bf16 [T*k, K], m_sizes int32 [num_groups],
    slots int32 [T, k]): xs and m_sizes are what gemm_grouped takes; slots[t, j]
    is the row of xs that holds the copy, or ~row (negative) for a dropped slot,
    whose row lies past the groups and holds zeros.  The order is stable: inside
    a group rows stand by token, then slot.  Not recorded for autograd: xs's
    gradient goes through dispatch_backward."""
    dev = _index_of(x, "x", torch.bfloat16)
    _need_on(dev, ids, "ids")
    if x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError("x must be [T, K] and ids [T, k]")
    if ids.dtype not in _ID_DTYPES:
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    T, K = x.shape
    k = ids.shape[1]
    _need_int32(T, k, K, num_groups)
    need = _sort_bytes(T, k, num_groups)
    ws = _empty(need, torch.uint8, dev) if need else None
    xs = _empty((T * k, K), torch.bfloat16, dev)
    m_sizes = _empty(num_groups, torch.int32, dev)
    slots = _empty((T, k), torch.int32, dev)
    _launch("w4a16_dispatch", dev, x.data_ptr(), ids.data_ptr(), ids.element_size(), xs.data_ptr(),
            m_sizes.data_ptr(), slots.data_ptr(), T, k, K, num_groups,
            ws.data_ptr() if need else None, need)
    return xs, m_sizes, slots


_ID_DTYPES = (torch.int32, torch.int64)
_WEIGHT_DTYPES = (torch.float32, torch.bfloat16)


def _need_slots(rows: torch.Tensor, slots: torch.Tensor, weights, name: str) -> int:
    dev = _index_of(rows, name, torch.bfloat16)
    _need_on(dev, slots, "slots", torch.int32)
    if rows.dim() != 2 or slots.dim() != 2 or rows.shape[0] != slots.numel():
        raise ValueError(f"{name} must be [T*k, N] for slots [T, k]")
    _need_int32(*slots.shape, rows.shape[1])
    if weights is not None:
        _need_on(dev, weights, "weights")
        if weights.dtype not in _WEIGHT_DTYPES or weights.shape != slots.shape:
            raise ValueError("weights must be float32 or bfloat16 with the shape of slots")
    return dev


def _combine(ys, slots, weights, name) -> torch.Tensor:
    dev = _need_slots(ys, slots, weights, name)
    T, k = slots.shape
    N = ys.shape[1]
    y = _empty((T, N), torch.bfloat16, dev)
    _launch("w4a16_combine", dev, ys.data_ptr(), slots.data_ptr(),
            None if weights is None else weights.data_ptr(),
            0 if weights is None else weights.element_size(), y.data_ptr(), T, k, N)
    return y


def combine(ys: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
    """y[t] = sum over j of weights[t, j] * ys[slots[t, j]] (dropped slots left out).

    ys: bf16 [T*k, N], rows in group order (the grouped product of dispatch's
    rows); slots: from dispatch; weights: float32 or bfloat16 [T, k].  fp32 sums,
    rounded once; returns bf16 [T, N].  Not recorded for autograd: the gradients are
    combine_backward's."""
    if weights is None:
        raise ValueError("weights must be a CUDA tensor")
    return _combine(ys, slots, weights, "ys")


def dispatch_backward(dxs: torch.Tensor, slots: torch.Tensor) -> torch.Tensor:
    """The gradient of dispatch: dx[t] = sum over the kept slots of dxs[slots[t, j]].

    dxs: bf16 [T*k, K]; returns bf16 [T, K] (fp32 sums, rounded once)."""
    return _combine(dxs, slots, None, "dxs")


def combine_backward(dy: torch.Tensor, ys: torch.Tensor, slots: torch.Tensor, weights: torch.Tensor):
    """The gradients of combine: (dys bf16 [T*k, N], dweights [T, k] in the weights' type).

    dys[slots[t, j]] = weights[t, j] * dy[t], zeros in the rows of dropped slots;
    dweights[t, j] = <dy[t], ys[slots[t, j]]>, 0 for a dropped slot."""
    if weights is None:
        raise ValueError("weights must be a CUDA tensor")
    dev = _need_slots(ys, slots, weights, "ys")
    T, k = slots.shape
    N = ys.shape[1]
    _need_on(dev, dy, "dy", torch.bfloat16)
    if dy.shape != (T, N):
        raise ValueError("dy must be [T, N]")
    dys = torch.empty_like(ys)
    dweights = torch.empty_like(weights)
    _launch("w4a16_combine_backward", dev, dy.data_ptr(), ys.data_ptr(), slots.data_ptr(),
            weights.data_ptr(), weights.element_size(), dys.data_ptr(), dweights.data_ptr(), T, k, N)
    return dys, dweights


@functools.lru_cache(maxsize=1024)
def _lora_bytes(tokens: int, adapters: int, rank: int, backward: int) -> int:
    nb = ctypes.c_size_t(0)
    _lib.check(_lib.lib().w4a16_lora_workspace_bytes(tokens, adapters, rank, backward, ctypes.byref(nb)),
               "w4a16_lora_workspace_bytes")
    return int(nb.value)


def _lora_workspace(index: int, tokens: int, adapters: int, rank: int, backward: int):
    need = _lora_bytes(tokens, adapters, rank, backward)
    return (_empty(need, torch.uint8, index) if need else None), need


def _need_lora(x, lora_a, lora_b, adapters, lora_scales):
    """Checks of what lora_add and its gradient share: (device, T, L, r, N, K)."""
    dev = _index_of(x, "x", torch.bfloat16)
    _need_on(dev, lora_a, "lora_a", torch.bfloat16)
    _need_on(dev, lora_b, "lora_b", torch.bfloat16)
    _need_on(dev, adapters, "adapters")
    _need_on(dev, lora_scales, "lora_scales", torch.float32)
    if x.dim() != 2 or lora_a.dim() != 3 or lora_b.dim() != 3:
        raise ValueError("x must be [T, K], lora_a [L, r, K] and lora_b [L, N, r]")
    T, K = x.shape
    L, r, ka = lora_a.shape
    lb, N, rb = lora_b.shape
    if ka != K or lb != L or rb != r:
        raise ValueError("lora_a must be [L, r, K] and lora_b [L, N, r] for x [T, K]")
    if adapters.dtype not in _ID_DTYPES or adapters.shape != (T,):
        raise ValueError("adapters must be int32 or int64 [T]")
    if lora_scales.shape != (L,):
        raise ValueError("lora_scales must be float32 [L]")
    _need_int32(T, L, r, N, K)
    return dev, T, L, r, N, K


def _need_rows(index, t, name, shape, dtype=torch.bfloat16):
    _need_on(index, t, name, dtype)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")


def lora_add(x: torch.Tensor, lora_a: torch.Tensor, lora_b: torch.Tensor, adapters: torch.Tensor,
             lora_scales: torch.Tensor, base: torch.Tensor | None = None, *,
             out: torch.Tensor | None = None, return_hidden: bool = False):
    """y[t] = base[t] + s_a * B_a . (A_a . x[t]), a = adapters[t]: the low-rank
    adapters of many requests at once, beside a shared projection's result.

    x: bf16 [T, K]; lora_a: bf16 [L, r, K]; lora_b: bf16 [L, N, r] (r a multiple
    of 8, at most 128); adapters: int32 or int64 [T], an id outside [0, L) leaves
    the token as it is; lora_scales: float32 [L]; base: bf16 [T, N] (gemm's
    result) or None for zeros.  ``out`` may be base itself.  Returns y bf16
    [T, N], with ``return_hidden`` also A . x (float32 [T, r]), which
    lora_add_backward takes.  Not recorded for autograd: the gradients are
    lora_add_backward's."""
    dev, T, L, r, N, K = _need_lora(x, lora_a, lora_b, adapters, lora_scales)
    if base is not None:
        _need_rows(dev, base, "base", (T, N))
    if out is None:
        out = _empty((T, N), torch.bfloat16, dev)
    else:
        _need_rows(dev, out, "out", (T, N))
    hidden = _empty((T, r), torch.float32, dev) if return_hidden else None
    ws, need = _lora_workspace(dev, T, L, r, 0)
    _launch("w4a16_lora_add", dev, x.data_ptr(), lora_a.data_ptr(), lora_b.data_ptr(), adapters.data_ptr(),
            adapters.element_size(), lora_scales.data_ptr(), None if base is None else base.data_ptr(),
            out.data_ptr(), hidden.data_ptr() if return_hidden else None, T, L, r, N, K,
            ws.data_ptr() if need else None, need)
    return (out, hidden) if return_hidden else out


def lora_add_backward(dy: torch.Tensor, x: torch.Tensor, hidden: torch.Tensor, lora_a: torch.Tensor,
                      lora_b: torch.Tensor, adapters: torch.Tensor, lora_scales: torch.Tensor, *,
                      dx_base: torch.Tensor | None = None):
    """The gradients of lora_add: (dx bf16 [T, K], d_lora_a, d_lora_b), the latter
    in the shapes and type of the adapters, zeros for an adapter without tokens.

    dy: bf16 [T, N]; hidden: what lora_add returned; dx_base: bf16 [T, K], the
    shared projection's own gradient, which the adapters' part is added to.
    base's gradient is dy."""
    dev, T, L, r, N, K = _need_lora(x, lora_a, lora_b, adapters, lora_scales)
    _need_rows(dev, dy, "dy", (T, N))
    _need_rows(dev, hidden, "hidden", (T, r), torch.float32)
    if dx_base is not None:
        _need_rows(dev, dx_base, "dx_base", (T, K))
    dx = torch.empty_like(x)
    da, db = torch.empty_like(lora_a), torch.empty_like(lora_b)
    ws, need = _lora_workspace(dev, T, L, r, 1)
    _launch("w4a16_lora_add_backward", dev, dy.data_ptr(), x.data_ptr(), hidden.data_ptr(), lora_a.data_ptr(),
            lora_b.data_ptr(), adapters.data_ptr(), adapters.element_size(), lora_scales.data_ptr(),
            None if dx_base is None else dx_base.data_ptr(), dx.data_ptr(), da.data_ptr(), db.data_ptr(),
            T, L, r, N, K, ws.data_ptr() if need else None, need)
    return dx, da, db


FP8_BLOCK = 128              # elements of a row per scale; of weights 128 x 128
_FP8 = torch.float8_e4m3fn


def quantize_fp8(x: torch.Tensor, *, blocks: bool = False):
    """(codes, scales): x in e4m3 with a float32 scale for 128 elements of a row, or,
    with ``blocks``, for a block of 128 x 128: what the 8-bit products take as their
    rows and as their weights.

    x: bf16 [M, K], any K; codes float8_e4m3fn [M, Kp] with Kp = K rounded up to a
    multiple of 128 and zeros past K; scales [Kp/128, M].  With ``blocks`` x is bf16
    [N, K] or [G, N, K] (K a multiple of 128); codes have its shape and scales are
    [N/128 rounded up, K/128], a leading G kept.  A scale is max |x| / 448, a code the
    nearest e4m3 to 448 x / max |x| (ties to even); a block of zeros has scale 0."""
    dev = _index_of(x, "x", torch.bfloat16)
    if not blocks:
        if x.dim() != 2 or x.shape[1] < 1:
            raise ValueError("x must be [M, K]")
        M, K = x.shape
        _need_int32(M, K)
        n = -(-K // FP8_BLOCK)
        codes, scales = _empty((M, n * FP8_BLOCK), _FP8, dev), _empty((n, M), torch.float32, dev)
        _launch("w4a16_quantize_fp8", dev, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K)
        return codes, scales
    if x.dim() not in (2, 3) or x.shape[-1] % FP8_BLOCK or 0 in x.shape:
        raise ValueError("x must be [N, K] or [G, N, K], K a multiple of 128")
    N, K = x.shape[-2:]
    G = x.shape[0] if x.dim() == 3 else 1
    _need_int32(G, N, K)
    codes = _empty(x.shape, _FP8, dev)
    scales = _empty((*x.shape[:-2], -(-N // FP8_BLOCK), K // FP8_BLOCK), torch.float32, dev)
    _launch("w4a16_quantize_fp8_blocks", dev, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), G, N, K)
    return codes, scales


def _need_fp8(x, x_scales, w, w_scales, dims, transposed):
    """Checks of what the 8-bit products share: (device, M, N, K, output columns)."""
    dev = _index_of(x, "x", _FP8)
    _need_on(dev, x_scales, "x_scales", torch.float32)
    _need_on(dev, w, "w", _FP8)
    _need_on(dev, w_scales, "w_scales", torch.float32)
    if x.dim() != 2 or w.dim() != dims:
        raise ValueError(f"x must be [M, C] and w {'[N, K]' if dims == 2 else '[num_groups, N, K]'}")
    N, K = w.shape[-2:]
    M, C = x.shape
    n = -(-N // FP8_BLOCK)
    if K % FP8_BLOCK or C != (n * FP8_BLOCK if transposed else K):
        raise ValueError("K must be a multiple of 128, and x [M, K] or, transposed, [M, N rounded up to one]")
    if x_scales.shape != (C // FP8_BLOCK, M):
        raise ValueError("x_scales must be float32 [C/128, M] for x [M, C]")
    if w_scales.shape != (*w.shape[:-2], n, K // FP8_BLOCK):
        raise ValueError("w_scales must be float32 [N/128 rounded up, K/128], by group as w is")
    _need_int32(M, N, K)
    return dev, M, N, K, K if transposed else N


def gemm_fp8(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, *,
             transposed: bool = False, out: torch.Tensor | None = None,
             resident_weights: bool = False) -> torch.Tensor:
    """Y = X . W^T (bf16 [M, N]) of rows and weights in 8 bits, as quantize_fp8 gives
    them: x [M, K] with x_scales [K/128, M], w [N, K] with w_scales of its blocks.

    ``transposed=True`` multiplies by W instead, from the same weights: x is [M, N]
    (N rounded up to a multiple of 128, the columns past N finite), the result bf16
    [M, K]; with the quantised gradient of Y that is the gradient of X.  Sums over a
    block of 128 are the tensor core's, over the blocks fp32; one rounding.  A row's scale
    times a weight block's has to be a normal float32 or 0 because one of them is 0 (so it
    is where blocks' largest magnitudes are 0 or between 2^-54 and 2^72).
    ``resident_weights`` as for gemm.  Not recorded for autograd."""
    dev, M, N, K, cols = _need_fp8(x, x_scales, w, w_scales, 2, transposed)
    if out is None:
        out = _empty((M, cols), torch.bfloat16, dev)
    else:
        _need_rows(dev, out, "out", (M, cols))
    _launch("w4a16_gemm_fp8", dev, x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
            out.data_ptr(), M, N, K, 1 if transposed else 0, FLAG_RESIDENT_WEIGHTS if resident_weights else 0)
    return out


def _need_groups(dev, m_sizes, groups, status):
    _need_on(dev, m_sizes, "m_sizes", torch.int32)
    if m_sizes.shape != (groups,):
        raise ValueError("m_sizes must be int32 [num_groups]")
    if status is None:
        return _empty(4, torch.int32, dev)
    _need_on(dev, status, "status", torch.int32)
    if status.numel() < 1:
        raise ValueError("status must hold an int32")
    return status


def gemm_fp8_grouped(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                     m_sizes: torch.Tensor, *, transposed: bool = False, out: torch.Tensor | None = None,
                     status: torch.Tensor | None = None):
    """gemm_fp8 by group in one launch: group g owns m_sizes[g] rows of x, in order, and
    w[g] of w [num_groups, N, K].

    m_sizes: int32 [num_groups] on the device (dispatch's), never read on the host.  Rows
    no group covers are left unwritten.  Returns (Y, status), status as gemm_grouped's.
    ``transposed=True``: the gradient of the rows.  Not recorded for autograd."""
    dev, M, N, K, cols = _need_fp8(x, x_scales, w, w_scales, 3, transposed)
    status = _need_groups(dev, m_sizes, w.shape[0], status)
    if out is None:
        out = _empty((M, cols), torch.bfloat16, dev)
    else:
        _need_rows(dev, out, "out", (M, cols))
    _launch("w4a16_gemm_fp8_grouped", dev, x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(),
            m_sizes.data_ptr(), out.data_ptr(), w.shape[0], M, N, K, 1 if transposed else 0, status.data_ptr())
    return out, status


def gemm_grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, m_sizes: torch.Tensor, *,
                       dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                       status: torch.Tensor | None = None):
    """The gradients of the weights of a product by group: dw[g] = dy_g^T . x_g over the
    rows of group g, zeros for a group without rows.

    dy: bf16 [M, N]; x: bf16 [M, K]; m_sizes: int32 [num_groups] on the device; N and K
    multiples of 8.  Returns (dw [num_groups, N, K] in ``dtype`` (float32 or bfloat16),
    status as gemm_grouped's).  fp32 sums, rounded once; rows no group covers are not
    summed."""
    dev = _index_of(dy, "dy", torch.bfloat16)
    _need_on(dev, x, "x", torch.bfloat16)
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [M, N] and x [M, K]")
    M, N = dy.shape
    K = x.shape[1]
    if m_sizes is None or not isinstance(m_sizes, torch.Tensor) or m_sizes.dim() != 1:
        raise ValueError("m_sizes must be int32 [num_groups]")
    G = m_sizes.shape[0]
    status = _need_groups(dev, m_sizes, G, status)
    if dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
    if N % 8 or K % 8:
        raise ValueError("N and K must be multiples of 8")
    _need_int32(M, N, K, G)
    if out is None:
        out = _empty((G, N, K), dtype, dev)
    else:
        _need_rows(dev, out, "out", (G, N, K), dtype)
    _launch("w4a16_gemm_grouped_wgrad", dev, dy.data_ptr(), x.data_ptr(), m_sizes.data_ptr(), out.data_ptr(),
            out.element_size(), G, M, N, K, status.data_ptr())
    return out, status
