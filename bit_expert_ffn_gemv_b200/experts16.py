"""16-bit experts on torch tensors: grouped products and their gradients, SwiGLU and its gradient.

Thin wrappers of the C calls (moe_grouped_matmul, moe_grouped_wgrad, moe_swiglu, moe_swiglu_backward in
include/moe.h): they check types, shapes and strides, allocate missing results with torch and enqueue on ``stream``
(default: the current stream of the tensors' device).  No call synchronises.  There is no autograd: the gradients
are calls of their own.

Rows are (token, expert) pairs sorted by expert; ``offsets`` (int32 [E + 1], on the device) gives each expert's row
range.  An expert FFN and its gradient, for gate/up matrices w1 [E, 2f, d] and down matrices w2 [E, d, f]:

    gu = grouped_matmul(x, w1, offsets)                       # [rows, 2f]
    h = swiglu(gu, row_weights)                               # [rows, f]
    y = grouped_matmul(h, w2, offsets)                        # [rows, d]

    dh = grouped_matmul(dy, w2, offsets, transpose=True)
    dgu, h, d_row_weights = swiglu_backward(gu, dh, row_weights, with_h=True)
    dx = grouped_matmul(dgu, w1, offsets, transpose=True)
    dw1 = grouped_matmul_wgrad(dgu, x, offsets)
    dw2 = grouped_matmul_wgrad(dy, h, offsets)

Rows outside every group are left as they were in a given ``out``, and are unset in an allocated one.
"""
from __future__ import annotations

import ctypes

import torch

from . import MOE_ACCUMULATE, MOE_OP_FP16, MOE_OP_TRANSPOSE, MOE_OUT_FP32, MoeAdapterArgs, _check, lib

__all__ = ["grouped_matmul", "grouped_matmul_wgrad", "swiglu", "swiglu_backward", "adapter_project"]

# Checks are written for the host's time: at the smallest sizes a call's kernels take a few microseconds, so
# every tensor attribute is read once and devices are compared by index.
_FP32, _INT32, _FP16, _BF16 = torch.float32, torch.int32, torch.float16, torch.bfloat16
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fail(what: str):
    raise ValueError(what)


def _operand(t, name: str):
    """(device index, type, rows, columns, pitch) of the matrix that sets a call's type and device."""
    dt = t.dtype
    if t.dim() != 2 or not t.is_cuda or (dt is not _BF16 and dt is not _FP16):
        _fail(f"{name}: a bf16 or fp16 CUDA matrix")
    dev = t.get_device()
    rows, cols = t.shape
    return dev, dt, rows, cols, _matrix(t, name, dev, dt, rows, cols)


def _matrix(t, name: str, dev: int, dt, rows: int, cols: int) -> int:
    """Row pitch of a [rows x cols] matrix of type dt on device dev with contiguous rows."""
    if t.dim() != 2 or t.get_device() != dev or t.dtype is not dt:
        _fail(f"{name}: a matrix of {dt} on cuda:{dev} is expected")
    if tuple(t.shape) != (rows, cols):
        _fail(f"{name}: shape {tuple(t.shape)}, {(rows, cols)} expected")
    if rows <= 1:  # (torch leaves the stride of one row arbitrary)
        if rows and cols > 1 and t.stride(1) != 1:
            _fail(f"{name}: columns must be contiguous")
        return (cols + 7) // 8 * 8
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        _fail(f"{name}: columns must be contiguous")
    return pitch


def _block(t, name: str, dev: int, dt, shape):
    if t.get_device() != dev or t.dtype is not dt or tuple(t.shape) != shape or not t.is_contiguous():
        _fail(f"{name}: a contiguous {shape} tensor of {dt} on cuda:{dev} is expected")


def _vector(t, name: str, dev: int, dt, n: int) -> int:
    if t.dim() != 1 or t.get_device() != dev or t.dtype is not dt or t.shape[0] != n or not t.is_contiguous():
        _fail(f"{name}: {n} contiguous values of {dt} on cuda:{dev} are expected")
    return t.data_ptr()


def _enqueue(dev: int, stream, what: str, fn, *args):
    """fn(*args, stream) with `dev` the current device."""
    if stream is not None:
        s = stream.cuda_stream
    elif _raw_stream is not None:
        s = _raw_stream(dev)
    else:
        s = torch.cuda.current_stream(dev).cuda_stream
    if torch.cuda.current_device() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st:
        _check(st, what)


def grouped_matmul(x, w, offsets, out=None, transpose=False, out_dtype=None, stream=None):
    """x [rows, k] times each group's W_e^T -> [rows, n]; w [E, n, k] contiguous.  With transpose: x [rows, n] times
    W_e -> [rows, k].  out (or out_dtype): x's type or fp32."""
    dev, dt, rows, xc, ldx = _operand(x, "x")
    if w.dim() != 3:
        _fail("w: a contiguous [E, n, k] tensor")
    E, n, k = w.shape
    _block(w, "w", dev, dt, (E, n, k))
    if xc != (n if transpose else k):
        _fail(f"x: {xc} columns do not match w {(E, n, k)}")
    off = _vector(offsets, "offsets", dev, _INT32, E + 1)
    cols = k if transpose else n
    if out is None:
        out = (x.new_empty((rows, cols)) if out_dtype is None
               else torch.empty((rows, cols), dtype=out_dtype, device=x.device))
    odt = out.dtype
    if (odt is not dt and odt is not _FP32) or (out_dtype is not None and odt is not out_dtype):
        _fail(f"out: {odt}")
    ldy = _matrix(out, "out", dev, odt, rows, cols)
    flags = ((MOE_OP_FP16 if dt is _FP16 else 0) | (MOE_OP_TRANSPOSE if transpose else 0)
             | (MOE_OUT_FP32 if odt is _FP32 else 0))
    _enqueue(dev, stream, "moe_grouped_matmul", lib().moe_grouped_matmul, x.data_ptr(), ldx, rows, w.data_ptr(), off, E,
             n, k, out.data_ptr(), ldy, flags)
    return out


def grouped_matmul_wgrad(dy, x, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """dy_e^T x_e of each group: dy [rows, n], x [rows, k] -> [E, n, k] of dy's type or fp32; accumulate adds to an
    fp32 out."""
    dev, dt, rows, n, lddy = _operand(dy, "dy")
    if x.dim() != 2:
        _fail("x: a matrix")
    k = x.shape[1]
    ldx = _matrix(x, "x", dev, dt, rows, k)
    E = offsets.numel() - 1
    if E < 1:
        _fail("offsets: at least one group")
    off = _vector(offsets, "offsets", dev, _INT32, E + 1)
    if accumulate and out is None:
        _fail("accumulate adds to a given out")
    if out is None:
        out = torch.empty((E, n, k), dtype=out_dtype or dt, device=dy.device)
    odt = out.dtype
    if (odt is not dt and odt is not _FP32) or (out_dtype is not None and odt is not out_dtype):
        _fail(f"out: {odt}")
    _block(out, "out", dev, odt, (E, n, k))
    flags = ((MOE_OP_FP16 if dt is _FP16 else 0) | (MOE_OUT_FP32 if odt is _FP32 else 0)
             | (MOE_ACCUMULATE if accumulate else 0))
    _enqueue(dev, stream, "moe_grouped_wgrad", lib().moe_grouped_wgrad, dy.data_ptr(), lddy, x.data_ptr(), ldx, rows, off,
             E, n, k, out.data_ptr(), flags)
    return out


def _gate_up(gu):
    dev, dt, rows, cols, ld = _operand(gu, "gu")
    if cols % 2:
        _fail("gu: gate and up values, an even number of columns")
    return dev, dt, rows, cols // 2, ld


def swiglu(gu, row_weights=None, out=None, n_rows=None, stream=None):
    """row_weights * silu(g) * u for gu = [g | u] [rows, 2f] -> [rows, f].  n_rows: int32 device tensor of one value,
    rows from it on are left as they were."""
    dev, dt, rows, f, ld = _gate_up(gu)
    rw = _vector(row_weights, "row_weights", dev, _FP32, rows) if row_weights is not None else None
    nr = _vector(n_rows, "n_rows", dev, _INT32, 1) if n_rows is not None else None
    if out is None:
        out = gu.new_empty((rows, f))
    ldh = _matrix(out, "out", dev, dt, rows, f)
    _enqueue(dev, stream, "moe_swiglu", lib().moe_swiglu, gu.data_ptr(), ld, rows, f, rw, nr, out.data_ptr(), ldh,
             MOE_OP_FP16 if dt is _FP16 else 0)
    return out


def swiglu_backward(gu, dh, row_weights=None, dgu=None, h=None, drw=None, with_h=False, n_rows=None, stream=None):
    """Gradient of swiglu: (dgu [rows, 2f], h or None, d_row_weights or None).  h, the forward's result again, is
    written when given or with_h; d_row_weights when row_weights is given."""
    dev, dt, rows, f, ld = _gate_up(gu)
    lddh = _matrix(dh, "dh", dev, dt, rows, f)
    if dgu is None:
        dgu = torch.empty((rows, 2 * f), dtype=dt, device=gu.device)
    lddgu = _matrix(dgu, "dgu", dev, dt, rows, 2 * f)
    if h is None and with_h:
        h = torch.empty((rows, f), dtype=dt, device=gu.device)
    ldh = _matrix(h, "h", dev, dt, rows, f) if h is not None else 0
    if row_weights is None and drw is not None:
        _fail("drw: needs row_weights")
    rw = dw = None
    if row_weights is not None:
        rw = _vector(row_weights, "row_weights", dev, _FP32, rows)
        if drw is None:
            drw = torch.empty(rows, dtype=_FP32, device=gu.device)
        dw = _vector(drw, "drw", dev, _FP32, rows)
    nr = _vector(n_rows, "n_rows", dev, _INT32, 1) if n_rows is not None else None
    _enqueue(dev, stream, "moe_swiglu_backward", lib().moe_swiglu_backward, gu.data_ptr(), ld, dh.data_ptr(), lddh, rows,
             f, rw, nr, dgu.data_ptr(), lddgu, h.data_ptr() if h is not None else None, ldh, dw,
             MOE_OP_FP16 if dt is _FP16 else 0)
    return dgu, h, drw


def adapter_project(x, a, b, ids, w=None, scale=None, out=None, flags=0, stream=None):
    """[w x_t +] scale[i] * b[i] (a[i] x_t) for every token t with its adapter i = ids[t]: x [T, k], a [L, rank, k],
    b [L, n, rank], ids int32 [T], w [n, k], scale fp32 [L] -> [T, n], x's type, or fp32 with MOE_OUT_FP32 in flags.
    With MOE_ACCUMULATE the result is added to out.  An id outside [0, L): no adapter."""
    dev, dt, T, k, ldx = _operand(x, "x")
    if a.dim() != 3 or b.dim() != 3:
        _fail("a, b: contiguous [L, rank, k] and [L, n, rank] tensors")
    L, rank = a.shape[0], a.shape[1]
    n = b.shape[1]
    _block(a, "a", dev, dt, (L, rank, k))
    _block(b, "b", dev, dt, (L, n, rank))
    id_ptr = _vector(ids, "ids", dev, _INT32, T)
    wp = sp = None
    if w is not None:
        _block(w, "w", dev, dt, (n, k))
        wp = w.data_ptr()
    if scale is not None:
        sp = _vector(scale, "scale", dev, _FP32, L)
    odt = _FP32 if flags & MOE_OUT_FP32 else dt
    if out is None:
        if flags & MOE_ACCUMULATE:
            _fail("MOE_ACCUMULATE adds to a given out")
        out = x.new_empty((T, n)) if odt is dt else torch.empty((T, n), dtype=odt, device=x.device)
    ldy = _matrix(out, "out", dev, odt, T, n)
    L_ = lib()
    size = L_.moe_adapter_workspace(T, rank)
    ws = x.new_empty(size // 2)  # (16-bit values)
    if stream is not None:
        ws.record_stream(stream)  # freed below, possibly before the call has run on its stream
    args = MoeAdapterArgs(x.data_ptr(), ldx, T, n, k, wp, a.data_ptr(), b.data_ptr(), sp, id_ptr, L, rank,
                          out.data_ptr(), ldy, ws.data_ptr(), size)
    _enqueue(dev, stream, "moe_adapter_project", L_.moe_adapter_project, args,
             flags | (MOE_OP_FP16 if dt is _FP16 else 0))
    return out
