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

_TYPES = (torch.bfloat16, torch.float16)


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _matrix(t, name: str, like, cols=None, rows=None, dtypes=None):
    """A 2-D device matrix with unit column stride, of like's device (and type unless dtypes is given)."""
    _need(t.dim() == 2 and t.is_cuda and t.device == like.device, f"{name}: a matrix on {like.device}")
    _need(t.dtype in dtypes if dtypes else t.dtype == like.dtype, f"{name}: type {t.dtype}")
    _need(cols is None or t.shape[1] == cols, f"{name}: {t.shape[1]} columns, {cols} expected")
    _need(rows is None or t.shape[0] == rows, f"{name}: {t.shape[0]} rows, {rows} expected")
    _need(t.stride(1) == 1 or t.shape[1] <= 1 or t.shape[0] == 0, f"{name}: columns must be contiguous")


def _pitch(t) -> int:
    """Row pitch in values (of one row: its length rounded up, torch leaves the stride arbitrary)."""
    return t.stride(0) if t.shape[0] > 1 else -(-t.shape[1] // 8) * 8


def _vector(t, name: str, like, dtype, n=None):
    _need(t.is_cuda and t.device == like.device and t.dtype == dtype and t.is_contiguous(),
          f"{name}: contiguous {dtype} on {like.device}")
    _need(n is None or t.numel() == n, f"{name}: {t.numel()} values, {n} expected")


def _operand(x, name: str):
    _need(x.is_cuda and x.dim() == 2 and x.dtype in _TYPES, f"{name}: a bf16 or fp16 CUDA matrix")
    _matrix(x, name, x)


def _enqueue(dev, stream, what: str, fn, *args):
    """fn(*args, stream) with `dev` the current device."""
    s = (torch.cuda.current_stream(dev) if stream is None else stream).cuda_stream
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    _check(st, what)


def _type_flag(t) -> int:
    return MOE_OP_FP16 if t.dtype == torch.float16 else 0


def _groups(w, offsets, like):
    _vector(offsets, "offsets", like, torch.int32)
    _need(offsets.dim() == 1 and offsets.numel() == w + 1, f"offsets: {offsets.numel()} values, {w + 1} expected")


def grouped_matmul(x, w, offsets, out=None, transpose=False, out_dtype=None, stream=None):
    """x [rows, k] times each group's W_e^T -> [rows, n]; w [E, n, k] contiguous.  With transpose: x [rows, n] times
    W_e -> [rows, k].  out (or out_dtype): x's type or fp32."""
    _operand(x, "x")
    _need(w.dim() == 3 and w.is_cuda and w.device == x.device and w.dtype == x.dtype and w.is_contiguous(),
          "w: a contiguous [E, n, k] tensor of x's type and device")
    E, n, k = w.shape
    _need(x.shape[1] == (n if transpose else k), f"x: {x.shape[1]} columns do not match w {tuple(w.shape)}")
    _groups(E, offsets, x)
    cols = k if transpose else n
    if out is None:
        out = torch.empty((x.shape[0], cols), dtype=out_dtype or x.dtype, device=x.device)
    _matrix(out, "out", x, cols, x.shape[0], (x.dtype, torch.float32))
    _need(out_dtype is None or out.dtype == out_dtype, "out and out_dtype differ")
    flags = _type_flag(x) | (MOE_OP_TRANSPOSE if transpose else 0) | (MOE_OUT_FP32 if out.dtype == torch.float32 else 0)
    _enqueue(x.device, stream, "moe_grouped_matmul", lib().moe_grouped_matmul, x.data_ptr(), _pitch(x), x.shape[0],
             w.data_ptr(), offsets.data_ptr(), E, n, k, out.data_ptr(), _pitch(out), flags)
    return out


def grouped_matmul_wgrad(dy, x, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """dy_e^T x_e of each group: dy [rows, n], x [rows, k] -> [E, n, k] of dy's type or fp32; accumulate adds to an
    fp32 out."""
    _operand(dy, "dy")
    _matrix(x, "x", dy, rows=dy.shape[0])
    _need(offsets.numel() >= 2, "offsets: at least one group")
    E, n, k = offsets.numel() - 1, dy.shape[1], x.shape[1]
    _groups(E, offsets, dy)
    _need(not accumulate or out is not None, "accumulate adds to a given out")
    if out is None:
        out = torch.empty((E, n, k), dtype=out_dtype or dy.dtype, device=dy.device)
    _need(tuple(out.shape) == (E, n, k) and out.is_cuda and out.device == dy.device and out.is_contiguous()
          and out.dtype in (dy.dtype, torch.float32), f"out: a contiguous {(E, n, k)} tensor of dy's type or fp32")
    _need(out_dtype is None or out.dtype == out_dtype, "out and out_dtype differ")
    flags = (_type_flag(dy) | (MOE_OUT_FP32 if out.dtype == torch.float32 else 0)
             | (MOE_ACCUMULATE if accumulate else 0))
    _enqueue(dy.device, stream, "moe_grouped_wgrad", lib().moe_grouped_wgrad, dy.data_ptr(), _pitch(dy), x.data_ptr(),
             _pitch(x), dy.shape[0], offsets.data_ptr(), E, n, k, out.data_ptr(), flags)
    return out


def _ptr(t):
    return t.data_ptr() if t is not None else None


def swiglu(gu, row_weights=None, out=None, n_rows=None, stream=None):
    """row_weights * silu(g) * u for gu = [g | u] [rows, 2f] -> [rows, f].  n_rows: int32 device tensor of one value,
    rows from it on are left as they were."""
    _operand(gu, "gu")
    _need(gu.shape[1] % 2 == 0, "gu: gate and up values, an even number of columns")
    rows, f = gu.shape[0], gu.shape[1] // 2
    if row_weights is not None:
        _vector(row_weights, "row_weights", gu, torch.float32, rows)
    if n_rows is not None:
        _vector(n_rows, "n_rows", gu, torch.int32, 1)
    if out is None:
        out = torch.empty((rows, f), dtype=gu.dtype, device=gu.device)
    _matrix(out, "out", gu, f, rows)
    _enqueue(gu.device, stream, "moe_swiglu", lib().moe_swiglu, gu.data_ptr(), _pitch(gu), rows, f, _ptr(row_weights),
             _ptr(n_rows), out.data_ptr(), _pitch(out), _type_flag(gu))
    return out


def swiglu_backward(gu, dh, row_weights=None, dgu=None, h=None, drw=None, with_h=False, n_rows=None, stream=None):
    """Gradient of swiglu: (dgu [rows, 2f], h or None, d_row_weights or None).  h, the forward's result again, is
    written when given or with_h; d_row_weights when row_weights is given."""
    _operand(gu, "gu")
    _need(gu.shape[1] % 2 == 0, "gu: gate and up values, an even number of columns")
    rows, f = gu.shape[0], gu.shape[1] // 2
    _matrix(dh, "dh", gu, f, rows)
    if dgu is None:
        dgu = torch.empty((rows, 2 * f), dtype=gu.dtype, device=gu.device)
    _matrix(dgu, "dgu", gu, 2 * f, rows)
    if h is None and with_h:
        h = torch.empty((rows, f), dtype=gu.dtype, device=gu.device)
    if h is not None:
        _matrix(h, "h", gu, f, rows)
    _need(row_weights is not None or drw is None, "drw: needs row_weights")
    if row_weights is not None:
        _vector(row_weights, "row_weights", gu, torch.float32, rows)
        if drw is None:
            drw = torch.empty(rows, dtype=torch.float32, device=gu.device)
        _vector(drw, "drw", gu, torch.float32, rows)
    if n_rows is not None:
        _vector(n_rows, "n_rows", gu, torch.int32, 1)
    _enqueue(gu.device, stream, "moe_swiglu_backward", lib().moe_swiglu_backward, gu.data_ptr(), _pitch(gu),
             dh.data_ptr(), _pitch(dh), rows, f, _ptr(row_weights), _ptr(n_rows), dgu.data_ptr(), _pitch(dgu), _ptr(h),
             _pitch(h) if h is not None else 0, _ptr(drw), _type_flag(gu))
    return dgu, h, drw


def adapter_project(x, a, b, ids, w=None, scale=None, out=None, flags=0, stream=None):
    """[w x_t +] scale[i] * b[i] (a[i] x_t) for every token t with its adapter i = ids[t]: x [T, k], a [L, rank, k],
    b [L, n, rank], ids int32 [T], w [n, k], scale fp32 [L] -> [T, n], x's type, or fp32 with MOE_OUT_FP32 in flags.
    With MOE_ACCUMULATE the result is added to out.  An id outside [0, L): no adapter."""
    _operand(x, "x")
    for t, name in ((a, "a"), (b, "b")):
        _need(t.dim() == 3 and t.is_cuda and t.device == x.device and t.dtype == x.dtype and t.is_contiguous(),
              f"{name}: a contiguous 3-D tensor of x's type and device")
    T, k = x.shape
    L, rank, n = a.shape[0], a.shape[1], b.shape[1]
    _need(a.shape[2] == k and tuple(b.shape) == (L, n, rank), f"a {tuple(a.shape)}, b {tuple(b.shape)} and x do not match")
    _vector(ids, "ids", x, torch.int32, T)
    if w is not None:
        _need(tuple(w.shape) == (n, k) and w.device == x.device and w.dtype == x.dtype and w.is_contiguous(),
              f"w: a contiguous {(n, k)} tensor of x's type and device")
    if scale is not None:
        _vector(scale, "scale", x, torch.float32, L)
    dt = torch.float32 if flags & MOE_OUT_FP32 else x.dtype
    _need(out is not None or not flags & MOE_ACCUMULATE, "MOE_ACCUMULATE adds to a given out")
    if out is None:
        out = torch.empty((T, n), dtype=dt, device=x.device)
    _matrix(out, "out", x, n, T, (dt,))
    size = lib().moe_adapter_workspace(T, rank)
    ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    if stream is not None:
        ws.record_stream(stream)  # freed below, possibly before the call has run on its stream
    args = MoeAdapterArgs(x.data_ptr(), _pitch(x), T, n, k, _ptr(w), a.data_ptr(), b.data_ptr(), _ptr(scale),
                          ids.data_ptr(), L, rank, out.data_ptr(), _pitch(out), ws.data_ptr(), size)
    _enqueue(x.device, stream, "moe_adapter_project", lib().moe_adapter_project, ctypes.byref(args),
             flags | _type_flag(x))
    return out
