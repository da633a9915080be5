"""The expert-layer operators around dispatch and combine: thin bindings over ``libep.so``.

* ``rms_norm_fp8``: residual addition and RMS norm with e4m3 rows and block scales, the input of an
  ``"fp8"`` plan's dispatch;
* ``sort_by_expert``, ``sorted_rows``, ``return_rows`` and the gradients ``sorted_rows_backward`` and
  ``return_rows_backward``: received rows in compact expert order, and back with routing weights;
* ``matmul_fp8`` and ``matmul_fp8_swiglu``: the block-scaled e4m3 product, dense or by expert.

Every call runs on the device of its first tensor, enqueues on the current stream (or ``stream``) and
returns without waiting.  Outputs and workspaces come from PyTorch's allocator on that stream.
Arguments are checked before any launch (``EpError`` with ``EP_ERR_ARG``); what only the device can
see is recorded in one status word per device, read and cleared by ``op_status``.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional, Tuple

import torch

from . import EP_BF16, EP_ERR_ARG, EP_FP16, EP_FP8_E4M3, EpError, _check, load_library

_HALF_CODES = {torch.bfloat16: EP_BF16, torch.float16: EP_FP16}
_OUT_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_status_words = {}


@dataclasses.dataclass
class ExpertOrder:
    """Rows sorted by expert: group g's sorted rows are offsets[g] .. offsets[g + 1] - 1."""
    offsets: torch.Tensor                    # [groups + 1] int32
    pos: torch.Tensor                        # [rows][k] (or [W][rows][k]) int32: sorted row of a pair, -1 for none
    src: torch.Tensor                        # [max_rows] int32: row * k + slot of a sorted row, -1 past the last
    counts: Optional[torch.Tensor] = None    # [W] int32: rows held by each rank (None: all of them)


def _bad(msg: str):
    raise EpError(EP_ERR_ARG, msg)


def _arg(t: torch.Tensor, what: str, dtype, shape, device) -> int:
    """Address of a tensor that has to be contiguous, of this type and shape, on this device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    if t.device != device:
        _bad(f"{what} is on {t.device}, the call runs on {device}")
    if t.dtype != dtype:
        _bad(f"{what} is {t.dtype}, the call takes {dtype}")
    if tuple(t.shape) != tuple(shape):
        _bad(f"{what} has shape {tuple(t.shape)}, the call takes {tuple(shape)}")
    _bad(f"{what} is not contiguous")


def _device(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        _bad(f"{what} is on {t.device}, not a CUDA device")
    return t.device


def _status_word(device: torch.device) -> torch.Tensor:
    w = _status_words.get(device.index)
    if w is None:
        with torch.cuda.device(device):
            w = torch.zeros(1, dtype=torch.int32, device=device)
            torch.cuda.synchronize(device)   # other streams may be the first to use it
        _status_words[device.index] = w
    return w


def op_status(device=None) -> int:
    """Wait for the device and return the first status its expert-layer calls recorded since the last
    read (0 for none), clearing it: EP_ERR_CAPACITY (more sorted rows than max_rows; the rest were
    left out), EP_ERR_DEVICE_BOUNDS (a position outside its buffer; skipped) or
    EP_ERR_DEVICE_TIMEOUT (a bounded wait of the product ran out; its output is not valid)."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else torch.device(device).index or 0)
    w = _status_word(dev)
    torch.cuda.synchronize(dev)
    v = int(w.item())
    if v:
        w.zero_()
        torch.cuda.synchronize(dev)
    return v


@contextlib.contextmanager
def _other_place(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


_here = contextlib.nullcontext()


def _place(device: torch.device, stream):
    """Context in which outputs are allocated and the call is enqueued: the tensors' device and the
    caller's stream, so that the allocator ties the memory to the stream that uses it."""
    if stream is None and device.index == torch.cuda.current_device():
        return _here
    return _other_place(device, stream)


# the current stream's handle without building a torch.cuda.Stream around it: 2 us less per call
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _raw_stream(device: torch.device) -> int:
    return _current_raw_stream(device.index)


def rms_norm_fp8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, want_y: bool = False, stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight; q, scales = e4m3 codes and one FP32
    scale per 128 elements of y (max|y| / 448, 1 for a block of zeros).  x and residual [rows][hidden]
    BF16 or FP16, hidden a multiple of 16, rows any multiple of 8 elements apart; weight [hidden] of
    x's type or FP32.  Returns (q [rows][hidden] float8_e4m3fn, scales [rows][ceil(hidden/128)],
    h [rows][hidden] or None without a residual, y [rows][hidden] or None unless want_y)."""
    dev = _device(x, "x")
    code = _HALF_CODES.get(x.dtype)
    if code is None:
        _bad(f"x is {x.dtype}, the call takes bfloat16 or float16")
    if x.dim() != 2:
        _bad(f"x has {x.dim()} dimensions, the call takes [rows][hidden]")
    rows, hidden = x.shape
    if x.stride(1) != 1 and hidden > 1:
        _bad("x: the elements of a row are not consecutive")
    rp, rs = None, 0
    if residual is not None:
        if residual.device != dev or residual.dtype != x.dtype or residual.shape != x.shape:
            _bad(f"residual is {residual.dtype} {tuple(residual.shape)} on {residual.device}, x is {x.dtype} "
                 f"{tuple(x.shape)} on {dev}")
        if residual.stride(1) != 1 and hidden > 1:
            _bad("residual: the elements of a row are not consecutive")
        rp, rs = residual.data_ptr(), residual.stride(0) if rows > 1 else hidden
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        _bad(f"weight is {weight.dtype}, the call takes {x.dtype} or float32")
    wp = _arg(weight, "weight", weight.dtype, (hidden,), dev)
    with _place(dev, stream):
        q = torch.empty((rows, hidden), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((rows, -(-hidden // 128)), dtype=torch.float32, device=dev)
        h = torch.empty((rows, hidden), dtype=x.dtype, device=dev) if residual is not None else None
        y = torch.empty((rows, hidden), dtype=x.dtype, device=dev) if want_y else None
        _check(load_library().ep_rms_norm_fp8(
            x.data_ptr(), x.stride(0) if rows > 1 else hidden, rp, rs, wp, weight.dtype == torch.float32, code, rows,
            hidden, eps, q.data_ptr(), scales.data_ptr(), h.data_ptr() if h is not None else None,
            y.data_ptr() if y is not None else None, _raw_stream(dev)))
    return q, scales, h, y


def _rows_shape(shape) -> Tuple[int, int]:
    """(W, rows per rank) of the leading dimensions [rows] or [W][rows]."""
    return (1, shape[0]) if len(shape) == 1 else (shape[0], shape[1])


def sort_by_expert(indices: torch.Tensor, experts: int, max_rows: Optional[int] = None,
                   counts: Optional[torch.Tensor] = None, stream=None) -> ExpertOrder:
    """Stable sort of (row, slot) pairs by expert.  indices [rows][k] int32 with ``experts`` experts, or
    [W][rows][k] with ``experts`` per rank, of which a rank's rows keep their own (ids r * experts ..
    (r + 1) * experts - 1); other ids, -1 among them, are left out.  counts [W] int32 on the device: rows
    held by each rank (``Dispatched.recv_count``).  max_rows bounds the sorted rows (default: every
    pair); pairs past it are left out and recorded (``op_status``)."""
    dev = _device(indices, "indices")
    if indices.dim() not in (2, 3):
        _bad(f"indices has {indices.dim()} dimensions, the call takes [rows][k] or [W][rows][k]")
    W, rows = _rows_shape(indices.shape[:-1])
    k = indices.shape[-1]
    ip = _arg(indices, "indices", torch.int32, indices.shape, dev)
    cp = None if counts is None else _arg(counts, "counts", torch.int32, (W,), dev)
    if max_rows is None:
        max_rows = W * rows * k
    if max_rows < 0:
        _bad(f"max_rows={max_rows} < 0")
    lib = load_library()
    status = _status_word(dev)
    with _place(dev, stream):
        need = lib.ep_sort_workspace_bytes(W, rows, k, experts)
        work = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        offsets = torch.empty(max(0, W * experts) + 1, dtype=torch.int32, device=dev)
        pos = torch.empty_like(indices)
        src = torch.empty(max_rows, dtype=torch.int32, device=dev)
        _check(lib.ep_sort_by_expert(ip, cp, W, rows, k, experts, max_rows, offsets.data_ptr(), pos.data_ptr(),
                                     src.data_ptr(), work.data_ptr() if need else None, need, status.data_ptr(),
                                     _raw_stream(dev)))
    return ExpertOrder(offsets, pos, src, counts)


def _order_args(order: ExpertOrder, lead, dev):
    """(W, rows, k, max_rows, pos, counts) of an order whose pairs belong to rows of shape ``lead``."""
    if order.pos.dim() not in (2, 3) or tuple(order.pos.shape[:-1]) != tuple(lead):
        _bad(f"order.pos has shape {tuple(order.pos.shape)}, the rows are {tuple(lead)}")
    W, rows = _rows_shape(lead)
    pp = _arg(order.pos, "order.pos", torch.int32, order.pos.shape, dev)
    cp = None if order.counts is None else _arg(order.counts, "order.counts", torch.int32, (W,), dev)
    return W, rows, order.pos.shape[-1], order.src.shape[0], pp, cp


def sorted_rows(order: ExpertOrder, x: torch.Tensor, scales: Optional[torch.Tensor] = None, stream=None):
    """x [rows][hidden] (or [W][rows][hidden]) in expert order: (x_sorted [max_rows][hidden], scales_sorted
    [max_rows][scale_dim] or None).  Any element type whose rows are a multiple of 16 bytes; scales
    FP32.  Rows past order.offsets[-1] hold unspecified data."""
    dev = _device(x, "x")
    lead = x.shape[:-1]
    W, rows, k, max_rows, pp, cp = _order_args(order, lead, dev)
    xp = _arg(x, "x", x.dtype, x.shape, dev)
    sd, sp = 0, None
    if scales is not None:
        sd = scales.shape[-1]
        sp = _arg(scales, "scales", torch.float32, (*lead, sd), dev)
    status = _status_word(dev)
    with _place(dev, stream):
        out = torch.empty((max_rows, x.shape[-1]), dtype=x.dtype, device=dev)
        out_s = torch.empty((max_rows, sd), dtype=torch.float32, device=dev) if scales is not None else None
        _check(load_library().ep_sorted_rows(
            xp, sp, pp, cp, W, rows, k, max_rows, x.shape[-1] * x.element_size(), sd, out.data_ptr(),
            out_s.data_ptr() if sd else None, status.data_ptr(), _raw_stream(dev)))
    return out, out_s


def _sorted_arg(order, y, what, dev):
    if y.dtype not in _HALF_CODES:
        _bad(f"{what} is {y.dtype}, the call takes bfloat16 or float16")
    if y.dim() != 2:
        _bad(f"{what} has {y.dim()} dimensions, the call takes [max_rows][hidden]")
    return _arg(y, what, y.dtype, (order.src.shape[0], y.shape[1]), dev), _HALF_CODES[y.dtype]


def return_rows(order: ExpertOrder, y: torch.Tensor, weights: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Rows back from expert order: out[row] = sum over the row's slots, ascending, of weight * y[pos],
    in FP32, rounded once.  y [max_rows][hidden] BF16 or FP16; weights of order.pos's shape, FP32 (None:
    ones).  A row without a sorted slot becomes zeros; rows past order.counts are not written."""
    dev = _device(y, "y")
    yp, code = _sorted_arg(order, y, "y", dev)
    lead = order.pos.shape[:-1]
    W, rows, k, max_rows, pp, cp = _order_args(order, lead, dev)
    wp = None if weights is None else _arg(weights, "weights", torch.float32, order.pos.shape, dev)
    status = _status_word(dev)
    with _place(dev, stream):
        out = torch.empty((*lead, y.shape[1]), dtype=y.dtype, device=dev)
        _check(load_library().ep_return_rows(yp, wp, pp, cp, W, rows, k, max_rows, y.shape[1], code, out.data_ptr(),
                                             status.data_ptr(), _raw_stream(dev)))
    return out


def sorted_rows_backward(order: ExpertOrder, dx_sorted: torch.Tensor, stream=None) -> torch.Tensor:
    """Gradient of sorted_rows for x: the sum of a row's sorted copies' gradients, in FP32, rounded once."""
    return return_rows(order, dx_sorted, None, stream)


def return_rows_backward(order: ExpertOrder, y: torch.Tensor, weights: torch.Tensor, dout: torch.Tensor, stream=None):
    """Gradients of return_rows: (dy [max_rows][hidden] = weight * dout[row], rounded once; dweights of
    weights' shape = <y[pos], dout[row]> in FP32, 0 where a slot has no sorted row).  Rows of dy past
    order.offsets[-1], and dweights of rows past order.counts, hold unspecified data."""
    dev = _device(y, "y")
    yp, code = _sorted_arg(order, y, "y", dev)
    lead = order.pos.shape[:-1]
    W, rows, k, max_rows, pp, cp = _order_args(order, lead, dev)
    wp = _arg(weights, "weights", torch.float32, order.pos.shape, dev)
    dp = _arg(dout, "dout", y.dtype, (*lead, y.shape[1]), dev)
    status = _status_word(dev)
    with _place(dev, stream):
        dy = torch.empty_like(y)
        dw = torch.empty_like(weights)
        _check(load_library().ep_return_rows_backward(
            yp, wp, dp, pp, cp, W, rows, k, max_rows, y.shape[1], code, dy.data_ptr(), dw.data_ptr(),
            status.data_ptr(), _raw_stream(dev)))
    return dy, dw


def _product_args(a, a_scales, b, b_scales, offsets):
    dev = _device(a, "a")
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if a.dim() != 2:
        _bad(f"a has {a.dim()} dimensions, the call takes [rows][inner]")
    rows, inner = a.shape
    if b.dim() != (2 if offsets is None else 3) or b.shape[-1] != inner:
        _bad(f"b has shape {tuple(b.shape)}, the call takes "
             f"{'[columns]' if offsets is None else '[groups][columns]'}[{inner}]")
    groups = 1 if offsets is None else b.shape[0]
    columns, kb = b.shape[-2], -(-inner // 128)
    scale_shape = (-(-columns // 128), kb) if offsets is None else (groups, -(-columns // 128), kb)
    args = (_arg(a, "a", f8, a.shape, dev), _arg(a_scales, "a_scales", f32, (rows, kb), dev),
            _arg(b, "b", f8, b.shape, dev), _arg(b_scales, "b_scales", f32, scale_shape, dev),
            None if offsets is None else _arg(offsets, "offsets", torch.int32, (groups + 1,), dev))
    return dev, args, rows, groups, columns, inner


def matmul_fp8(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, out_dtype: str = "bf16", stream=None) -> torch.Tensor:
    """a @ b^T of e4m3 values with FP32 scales, in FP32, rounded once to out_dtype ("bf16" or "fp16").
    a [rows][inner] with a_scales [rows][ceil(inner/128)]; b [columns][inner] with b_scales
    [ceil(columns/128)][ceil(inner/128)].  With offsets [groups + 1] int32 on the device, b and b_scales
    have a leading [groups] and rows offsets[g] .. offsets[g + 1] - 1 take b[g]; rows outside every group
    are not written.  inner must be a multiple of 16."""
    dev, args, rows, groups, columns, inner = _product_args(a, a_scales, b, b_scales, offsets)
    t = _OUT_TYPES.get(out_dtype)
    if t is None:
        _bad(f"out_dtype={out_dtype!r} is neither 'bf16' nor 'fp16'")
    status = _status_word(dev)
    with _place(dev, stream):
        out = torch.empty((rows, columns), dtype=t, device=dev)
        _check(load_library().ep_matmul_fp8(*args, rows, groups, columns, inner, 0, _HALF_CODES[t], out.data_ptr(),
                                            None, status.data_ptr(), _raw_stream(dev)))
    return out


def matmul_fp8_swiglu(a: torch.Tensor, a_scales: torch.Tensor, b: torch.Tensor, b_scales: torch.Tensor,
                      offsets: Optional[torch.Tensor] = None, stream=None):
    """SwiGLU of the product, quantised: b's first half of columns is the gate, the second the up
    projection; z = gate * sigmoid(gate) * up in FP32.  Returns (q [rows][columns/2] float8_e4m3fn,
    scales [rows][ceil(columns/256)]), the a and a_scales of a following matmul_fp8.  Arguments as
    matmul_fp8; columns must be a multiple of 32."""
    dev, args, rows, groups, columns, inner = _product_args(a, a_scales, b, b_scales, offsets)
    status = _status_word(dev)
    with _place(dev, stream):
        q = torch.empty((rows, columns // 2), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((rows, -(-(columns // 2) // 128)), dtype=torch.float32, device=dev)
        _check(load_library().ep_matmul_fp8(*args, rows, groups, columns, inner, 1, EP_FP8_E4M3, q.data_ptr(),
                                            scales.data_ptr(), status.data_ptr(), _raw_stream(dev)))
    return q, scales
