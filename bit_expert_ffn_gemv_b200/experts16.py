"""16-bit experts on torch tensors: grouped products and their gradients, SwiGLU and its gradient, adapters.

Wrappers of the C calls (moe_grouped_matmul, moe_grouped_wgrad, moe_swiglu, moe_swiglu_backward and
moe_adapter_project in include/moe.h).  The checks of types, shapes and strides, the results' allocation and the call
are in csrc/binding.cpp (module _ops16): ValueError for tensors that do not fit, MoeError for what the library
refuses.  Work is enqueued on ``stream`` (a torch.cuda.Stream; default: the current stream of the tensors' device),
and a result that is not given is allocated for that stream.  No call synchronises.  There is no autograd: the
gradients are calls of their own, and while gradients are recorded a tensor that requires one is refused (detach it,
or call under torch.no_grad()).

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

from . import MoeError, lib

lib()  # libmoe.so, which the binding links against; raises with the build's command if it is absent
try:
    from . import _ops16
except ImportError as e:
    raise ImportError(f"the torch binding is missing: build it with `python -m bit_expert_ffn_gemv_b200.build` ({e})") from e
_ops16.set_error(MoeError)

__all__ = ["grouped_matmul", "grouped_matmul_wgrad", "swiglu", "swiglu_backward", "adapter_project"]


def grouped_matmul(x, w, offsets, out=None, transpose=False, out_dtype=None, stream=None):
    """x [rows, k] times each group's W_e^T -> [rows, n]; w [E, n, k] contiguous.  With transpose: x [rows, n] times
    W_e -> [rows, k].  out (or out_dtype): x's type or fp32."""
    return _ops16.grouped_matmul(x, w, offsets, out, transpose, out_dtype, stream)


def grouped_matmul_wgrad(dy, x, offsets, out=None, out_dtype=None, accumulate=False, stream=None):
    """dy_e^T x_e of each group: dy [rows, n], x [rows, k] -> [E, n, k] of dy's type or fp32; accumulate adds to an
    fp32 out."""
    return _ops16.grouped_wgrad(dy, x, offsets, out, out_dtype, accumulate, stream)


def swiglu(gu, row_weights=None, out=None, n_rows=None, stream=None):
    """row_weights * silu(g) * u for gu = [g | u] [rows, 2f] -> [rows, f].  n_rows: int32 device tensor of one value,
    rows from it on are left as they were."""
    return _ops16.swiglu(gu, row_weights, out, n_rows, stream)


def swiglu_backward(gu, dh, row_weights=None, dgu=None, h=None, drw=None, with_h=False, n_rows=None, stream=None):
    """Gradient of swiglu: (dgu [rows, 2f], h or None, d_row_weights or None).  h, the forward's result again, is
    written when given or with_h; d_row_weights when row_weights is given.  dgu may be gu itself (in place)."""
    return _ops16.swiglu_backward(gu, dh, row_weights, dgu, h, drw, with_h, n_rows, stream)


def adapter_project(x, a, b, ids, w=None, scale=None, out=None, flags=0, stream=None):
    """[w x_t +] scale[i] * b[i] (a[i] x_t) for every token t with its adapter i = ids[t]: x [T, k], a [L, rank, k],
    b [L, n, rank], ids int32 [T], w [n, k], scale fp32 [L] -> [T, n], x's type, or fp32 with MOE_OUT_FP32 in flags.
    With MOE_ACCUMULATE the result is added to out; no other flag is taken (the type is x's).  An id outside [0, L): no adapter."""
    return _ops16.adapter_project(x, a, b, ids, w, scale, out, flags, stream)
