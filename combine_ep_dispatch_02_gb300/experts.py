"""The expert-layer operators around dispatch and combine: thin bindings over ``libep.so``.

* ``rms_norm_fp8``: residual addition and RMS norm with e4m3 rows and block scales, the input of an
  ``"fp8"`` plan's dispatch;
* ``sort_by_expert``, ``sorted_rows``, ``return_rows`` and the gradients ``sorted_rows_backward`` and
  ``return_rows_backward``: received rows in compact expert order, and back with routing weights;
* ``matmul_fp8`` and ``matmul_fp8_swiglu``: the block-scaled e4m3 product, dense or by expert.

Every call runs on the device of its first tensor, enqueues on the current stream (or ``stream``) and
returns without waiting.  Outputs and workspaces come from PyTorch's allocator on that stream.
Arguments are checked before any launch (``EpError`` with ``EP_ERR_ARG``); what only the device can
see is recorded in one status word per device, read and cleared by ``op_status``.  The first call on a
device makes that word and waits for it, so a call comes before a graph's capture.

The gradients are calls of their own, for a training step or its ``torch.autograd.Function`` to make: no call
here records itself for autograd, and its results never require a gradient.

The checks and allocations are native (``_ep_binding``, csrc/ep_binding.cpp): these calls are often one
token's, and marshalling in Python would take longer than the kernels.
"""
from __future__ import annotations

import ctypes
import dataclasses
import importlib.util
import os
import sys
from typing import Optional

import torch

from . import EP_BF16, EP_ERR_ARG, EP_FP16, EP_FP8_E4M3, EpError, _PKG, _check, load_library

_package = sys.modules[__package__]

BINDING_PATH = os.path.join(_PKG, "_ep_binding.so")
_OUT_CODES = {"bf16": EP_BF16, "fp16": EP_FP16}
# the C ABI functions the binding calls, in the order of its bind()
_BOUND = ("ep_rms_norm_fp8", "ep_sort_workspace_bytes", "ep_sort_by_expert", "ep_sorted_rows", "ep_return_rows",
          "ep_return_rows_backward", "ep_matmul_fp8", "ep_strerror", "ep_last_error")
_status_words = {}
_binding = None
_bound_to = None


def _native():
    """The native binding, calling whichever build of libep.so the package has loaded."""
    global _binding, _bound_to
    if _bound_to is not None and _package._lib is _bound_to:   # the usual case, without a call
        return _binding
    lib = load_library()
    if lib is not _bound_to:
        if _binding is None:
            if not os.path.exists(BINDING_PATH):
                raise RuntimeError(f"_ep_binding.so not found at {BINDING_PATH}: build it with "
                                   "combine_ep_dispatch_02_gb300.build.build()")
            spec = importlib.util.spec_from_file_location("_ep_binding", BINDING_PATH)
            _binding = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_binding)
        _binding.bind(EpError, _status_address,
                      *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _BOUND))
        _bound_to = lib
    return _binding


@dataclasses.dataclass
class ExpertOrder:
    """Rows sorted by expert: group g's sorted rows are offsets[g] .. offsets[g + 1] - 1."""
    offsets: torch.Tensor                    # [groups + 1] int32
    pos: torch.Tensor                        # [rows][k] (or [W][rows][k]) int32: sorted row of a pair, -1 for none
    src: torch.Tensor                        # [max_rows] int32: row * k + slot of a sorted row, -1 past the last
    counts: Optional[torch.Tensor] = None    # [W] int32: rows held by each rank (None: all of them)


def _status_word(device: torch.device) -> torch.Tensor:
    w = _status_words.get(device.index)
    if w is None:
        with torch.cuda.device(device):
            w = torch.zeros(1, dtype=torch.int32, device=device)
            torch.cuda.synchronize(device)   # other streams may be the first to use it
        _status_words[device.index] = w
    return w


def _status_address(index: int) -> int:
    return _status_word(torch.device("cuda", index)).data_ptr()


def op_status(device=None) -> int:
    """Wait for the device and return the first status its expert-layer calls recorded since the last
    read (0 for none), clearing it: EP_ERR_CAPACITY (more sorted rows than max_rows; the rest were
    left out), EP_ERR_DEVICE_BOUNDS (a position outside its buffer; skipped) or
    EP_ERR_DEVICE_TIMEOUT (a bounded wait of the product ran out; its output is not valid).  The word
    is read and cleared in one step, so a status that another host thread's call records meanwhile stays for
    the next read; but it is the device's, not the caller's: one thread's read takes what another's call
    recorded."""
    index = None if device is None else torch.device(device).index
    dev = torch.device("cuda", torch.cuda.current_device() if index is None else index)
    w = _status_word(dev)
    torch.cuda.synchronize(dev)
    with torch.cuda.device(dev):
        taken = torch.empty(1, dtype=torch.int32, device=dev)
        _check(load_library().ep_take_status(w.data_ptr(), taken.data_ptr(), torch.cuda.current_stream().cuda_stream))
        return int(taken.item())


def _on(stream, call, *args):
    """The call on the current stream, or on the caller's, where its outputs are then allocated too; memory of
    its inputs that is freed is not reused before that stream is done with them."""
    if stream is None:
        return call(*args)
    with torch.cuda.stream(stream):
        out = call(*args)
        for a in args:
            if isinstance(a, torch.Tensor) and a.is_cuda:
                a.record_stream(stream)
        return out


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, want_y: bool = False, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; q, scales = e4m3 codes and one FP32
    scale per 128 elements of y (max|y| / 448, 1 for a block of zeros).  x and residual [rows][hidden]
    BF16 or FP16, hidden a multiple of 16, rows any multiple of 8 elements apart; weight [hidden] of
    x's type or FP32.  Returns (q [rows][hidden] float8_e4m3fn, scales [rows][ceil(hidden/128)],
    h [rows][hidden] or None without a residual, y [rows][hidden] or None unless want_y)."""
    return _on(stream, _native().rms_norm_fp8, x, weight, residual, eps, want_y)


def sort_by_expert(indices: torch.Tensor, experts: int, max_rows: Optional[int] = None,
                   counts: Optional[torch.Tensor] = None, stream=None) -> ExpertOrder:
    """Stable sort of (row, slot) pairs by expert.  indices [rows][k] int32 with ``experts`` experts, or
    [W][rows][k] with ``experts`` per rank, of which a rank's rows keep their own (ids r * experts ..
    (r + 1) * experts - 1); other ids, -1 among them, are left out.  counts [W] int32 on the device: rows
    held by each rank (``Dispatched.recv_count``).  max_rows bounds the sorted rows (default: every
    pair); pairs past it are left out and recorded (``op_status``)."""
    return ExpertOrder(*_on(stream, _native().sort_by_expert, indices, experts, max_rows, counts), counts)


def sorted_rows(order: ExpertOrder, x: torch.Tensor, scales: Optional[torch.Tensor] = None, stream=None):
    """x [rows][hidden] (or [W][rows][hidden]) in expert order: (x_sorted [max_rows][hidden], scales_sorted
    [max_rows][scale_dim] or None).  Any element type whose rows are a multiple of 16 bytes; scales
    FP32.  Rows past order.offsets[-1] hold unspecified data."""
    return _on(stream, _native().sorted_rows, order.pos, order.src, order.counts, x, scales)


def return_rows(order: ExpertOrder, y: torch.Tensor, weights: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Rows back from expert order: out[row] = sum over the row's slots, ascending, of weight * y[pos],
    in FP32, rounded once.  y [max_rows][hidden] BF16 or FP16; weights of order.pos's shape, FP32 (None:
    ones).  A row without a sorted slot becomes zeros; rows past order.counts are not written."""
    return _on(stream, _native().return_rows, order.pos, order.src, order.counts, y, weights)


def sorted_rows_backward(order: ExpertOrder, dx_sorted: torch.Tensor, stream=None) -> torch.Tensor:
    """Gradient of sorted_rows for x: the sum of a row's sorted copies' gradients, in FP32, rounded once."""
    return return_rows(order, dx_sorted, None, stream)


def return_rows_backward(order: ExpertOrder, y: torch.Tensor, weights: torch.Tensor, dout: torch.Tensor, stream=None):
    """Gradients of return_rows: (dy [max_rows][hidden] = weight * dout[row], rounded once; dweights of
    weights' shape = <y[pos], dout[row]> in FP32, 0 where a slot has no sorted row).  Rows of dy past
    order.offsets[-1], and dweights of rows past order.counts, hold unspecified data."""
    return _on(stream, _native().return_rows_backward, order.pos, order.src, order.counts, y, weights, dout)


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, out_dtype: str = "bf16", stream=None) -> torch.Tensor:
    """a @ b^T of e4m3 values with FP32 scales, in FP32, rounded once to out_dtype ("bf16" or "fp16").
    a [rows][inner] with a_scales [rows][ceil(inner/128)]; b [columns][inner] with b_scales
    [ceil(columns/128)][ceil(inner/128)].  With offsets [groups + 1] int32 on the device, b and b_scales
    have a leading [groups] and rows offsets[g] .. offsets[g + 1] - 1 take b[g]; rows outside every group
    are not written.  inner must be a multiple of 16.  The kernel is chosen from a's rows, so a buffer cut to
    about the rows that the groups hold can be faster than one of full capacity."""
    code = _OUT_CODES.get(out_dtype)
    if code is None:
        raise EpError(EP_ERR_ARG, f"out_dtype={out_dtype!r} is neither 'bf16' nor 'fp16'")
    return _on(stream, _native().matmul_fp8, a, a_scales, b, b_scales, offsets, code)


def matmul_fp8_swiglu(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, stream=None):
    """SwiGLU of the product, quantised: b's first half of columns is the gate, the second the up
    projection; z = gate * sigmoid(gate) * up in FP32.  Returns (q [rows][columns/2] float8_e4m3fn,
    scales [rows][ceil(columns/256)]), the a and a_scales of a following matmul_fp8.  Arguments as
    matmul_fp8; columns must be a multiple of 32."""
    return _on(stream, _native().matmul_fp8, a, a_scales, b, b_scales, offsets, EP_FP8_E4M3)
