// binding.cpp -- the 16-bit expert operators on torch tensors (module _ops16).
//
// At the smallest sizes an operator's kernels take two to six microseconds, as
// long as one pass of argument checks in Python takes by itself, so the checks,
// the results' allocation and the call of the C ABI are here: about one
// microsecond beside the launches.  experts16.py holds the documented signatures
// and passes every argument by position.  Wrong shapes, types and devices raise
// ValueError before anything is enqueued; a status of the library raises
// MoeError.  No call synchronises.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>

#include "moe.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_moe_error = nullptr;

// a failed status as MoeError(status, what)
PyObject* raise_status(moe_status s, const char* what) {
    PyObject* e = PyObject_CallFunction(g_moe_error, "is", (int)s, what);
    if (e) {
        PyErr_SetObject(g_moe_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, ": a tensor is expected");
    const Tensor& t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(!(t.requires_grad() && at::GradMode::is_enabled()), name,
                      ": requires a gradient, and this call records none (detach it, or call under torch.no_grad())");
    return t;
}

struct Operand {  // the matrix that sets a call's type and device
    const Tensor& t;
    int dev;
    ScalarType type;
    int64_t rows, cols, ld;
};

// Row pitch of a [rows x cols] matrix with contiguous columns (of one row: its
// length rounded up, torch leaves that stride arbitrary).
int64_t pitch(const Tensor& t, const char* name) {
    const int64_t rows = t.size(0), cols = t.size(1);
    TORCH_CHECK_VALUE(rows == 0 || cols <= 1 || t.stride(1) == 1, name, ": columns must be contiguous");
    return rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
}

void on_device(const Tensor& t, const char* name, int dev) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == dev, name, ": a tensor on cuda:", dev, " is expected");
}

int64_t matrix(const Tensor& t, const char* name, int dev, ScalarType type, int64_t rows, int64_t cols) {
    on_device(t, name, dev);
    TORCH_CHECK_VALUE(t.dim() == 2 && t.scalar_type() == type && t.size(0) == rows && t.size(1) == cols, name,
                      ": a [", rows, ", ", cols, "] matrix of ", type, " is expected, not ", t.sizes(), " of ",
                      t.scalar_type());
    return pitch(t, name);
}

Operand operand(PyObject* o, const char* name) {
    const Tensor& t = tensor(o, name);
    TORCH_CHECK_VALUE(t.is_cuda() && t.dim() == 2 &&
                          (t.scalar_type() == ScalarType::BFloat16 || t.scalar_type() == ScalarType::Half),
                      name, ": a bf16 or fp16 CUDA matrix is expected");
    return {t, (int)t.get_device(), t.scalar_type(), t.size(0), t.size(1), pitch(t, name)};
}

void block(const Tensor& t, const char* name, int dev, ScalarType type, at::IntArrayRef shape) {
    on_device(t, name, dev);
    TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous(), name, ": a contiguous ", shape,
                      " tensor of ", type, " is expected, not ", t.sizes(), " of ", t.scalar_type());
}

// data of an optional vector of n values (None: null)
void* vector(PyObject* o, const char* name, int dev, ScalarType type, int64_t n) {
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    on_device(t, name, dev);
    TORCH_CHECK_VALUE(t.dim() == 1 && t.scalar_type() == type && t.size(0) == n && t.is_contiguous(), name, ": ", n,
                      " contiguous values of ", type, " are expected");
    return t.data_ptr();
}

int32_t int32(int64_t v, const char* name) {
    TORCH_CHECK_VALUE(v >= 0 && v <= INT32_MAX, name, ": ", v, " is out of range");
    return (int32_t)v;
}

// A result: the caller's tensor `o`, or a new one (held by `made`).
struct Result {
    Tensor made;
    const Tensor* t = nullptr;
    PyObject* given = nullptr;
    PyObject* object() {
        if (given) {
            // written behind autograd's back: a graph that saved it has to see that
            if (!t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
            Py_INCREF(given);
            return given;
        }
        return THPVariable_Wrap(std::move(made));
    }
};
Result result(PyObject* o, const char* name, at::IntArrayRef shape, const Tensor& like, ScalarType type) {
    Result r;
    if (o != Py_None) {
        r.t = &tensor(o, name);
        r.given = o;
    } else {
        r.made = at::empty(shape, like.options().dtype(type));
    }
    return r;
}
const Tensor& of(const Result& r) { return r.t ? *r.t : r.made; }

// the type of a result that may be fp32: the given tensor's, else out_dtype's, else the operands'
ScalarType result_type(PyObject* out, PyObject* out_dtype, ScalarType type) {
    ScalarType t = type;
    if (out_dtype != Py_None) {
        TORCH_CHECK_TYPE(THPDtype_Check(out_dtype), "out_dtype: a torch.dtype is expected");
        t = reinterpret_cast<THPDtype*>(out_dtype)->scalar_type;
    }
    if (out != Py_None) {
        const ScalarType have = tensor(out, "out").scalar_type();
        TORCH_CHECK_VALUE(out_dtype == Py_None || have == t, "out and out_dtype differ");
        t = have;
    }
    TORCH_CHECK_VALUE(t == type || t == ScalarType::Float, "out: ", type, " or fp32 is expected, not ", t);
    return t;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v == 1;
}
uint32_t type_flag(ScalarType t) { return t == ScalarType::Half ? MOE_OP_FP16 : 0u; }
uint32_t fp32_flag(ScalarType t) { return t == ScalarType::Float ? MOE_OUT_FP32 : 0u; }

// The device and stream of a call: the given torch.cuda.Stream, or (None) the
// device's current one.  What the call allocates belongs to that stream: memory of
// another stream's pool may still be in use there, and the workspace is freed on
// return, before the call has run.
class Call {
    c10::cuda::CUDAGuard device_;
    std::optional<c10::cuda::CUDAStreamGuard> given_;

    static PyObject* attribute(PyObject* o, const char* name) {
        PyObject* v = PyObject_GetAttrString(o, name);
        if (!v) throw python_error();
        return v;
    }

public:
    void* stream;
    Call(PyObject* o, int dev) : device_((c10::DeviceIndex)dev) {
        if (o == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
            return;
        }
        PyObject* v = attribute(o, "device_index");
        const long on = PyLong_AsLong(v);
        Py_DECREF(v);
        v = attribute(o, "cuda_stream");
        stream = PyLong_AsVoidPtr(v);
        Py_DECREF(v);
        if (PyErr_Occurred()) throw python_error();
        TORCH_CHECK_VALUE(on == dev, "stream: one of cuda:", dev, " is expected, not of cuda:", on);
        given_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)dev));
    }
};

void arguments(Py_ssize_t got, Py_ssize_t want) { TORCH_CHECK_TYPE(got == want, want, " arguments are expected, not ", got); }

// x, w, offsets, out, transpose, out_dtype, stream
PyObject* grouped_matmul(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 7);
    const Operand x = operand(a[0], "x");
    const Tensor& w = tensor(a[1], "w");
    TORCH_CHECK_VALUE(w.dim() == 3, "w: a contiguous [E, n, k] tensor is expected");
    const int64_t E = w.size(0), n = w.size(1), k = w.size(2);
    block(w, "w", x.dev, x.type, {E, n, k});
    const bool tr = truth(a[4]);
    TORCH_CHECK_VALUE(x.cols == (tr ? n : k), "x: ", x.cols, " columns do not match w ", w.sizes());
    TORCH_CHECK_VALUE(a[2] != Py_None, "offsets: a tensor is expected");
    const void* off = vector(a[2], "offsets", x.dev, ScalarType::Int, E + 1);
    const int64_t cols = tr ? k : n;
    const ScalarType type = result_type(a[3], a[5], x.type);
    const Call call(a[6], x.dev);
    Result y = result(a[3], "out", {x.rows, cols}, x.t, type);
    const int64_t ldy = matrix(of(y), "out", x.dev, type, x.rows, cols);
    const moe_status s = moe_grouped_matmul(x.t.data_ptr(), x.ld, int32(x.rows, "rows"), w.data_ptr(),
                                            static_cast<const int32_t*>(off), int32(E, "E"), int32(n, "n"), int32(k, "k"),
                                            of(y).data_ptr(), ldy,
                                            type_flag(x.type) | fp32_flag(type) | (tr ? MOE_OP_TRANSPOSE : 0u),
                                            call.stream);
    if (s != MOE_OK) return raise_status(s, "moe_grouped_matmul");
    return y.object();
    END_HANDLE_TH_ERRORS
}

// dy, x, offsets, out, out_dtype, accumulate, stream
PyObject* grouped_wgrad(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 7);
    const Operand dy = operand(a[0], "dy");
    const Tensor& x = tensor(a[1], "x");
    TORCH_CHECK_VALUE(x.dim() == 2, "x: a matrix is expected");
    const int64_t n = dy.cols, k = x.size(1), ldx = matrix(x, "x", dy.dev, dy.type, dy.rows, k);
    const int64_t E = tensor(a[2], "offsets").numel() - 1;
    TORCH_CHECK_VALUE(E >= 1, "offsets: at least one group is expected");
    const void* off = vector(a[2], "offsets", dy.dev, ScalarType::Int, E + 1);
    const bool add = truth(a[5]);
    TORCH_CHECK_VALUE(!add || a[3] != Py_None, "accumulate adds to a given out");
    const ScalarType type = result_type(a[3], a[4], dy.type);
    const Call call(a[6], dy.dev);
    Result dw = result(a[3], "out", {E, n, k}, dy.t, type);
    block(of(dw), "out", dy.dev, type, {E, n, k});
    const moe_status s = moe_grouped_wgrad(dy.t.data_ptr(), dy.ld, x.data_ptr(), ldx, int32(dy.rows, "rows"),
                                           static_cast<const int32_t*>(off), int32(E, "E"), int32(n, "n"), int32(k, "k"),
                                           of(dw).data_ptr(),
                                           type_flag(dy.type) | fp32_flag(type) | (add ? MOE_ACCUMULATE : 0u),
                                           call.stream);
    if (s != MOE_OK) return raise_status(s, "moe_grouped_wgrad");
    return dw.object();
    END_HANDLE_TH_ERRORS
}

int64_t half_cols(const Operand& gu) {
    TORCH_CHECK_VALUE(gu.cols % 2 == 0, "gu: gate and up values, an even number of columns, are expected");
    return gu.cols / 2;
}

// gu, row_weights, out, n_rows, stream
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 5);
    const Operand gu = operand(a[0], "gu");
    const int64_t f = half_cols(gu);
    const void* rw = vector(a[1], "row_weights", gu.dev, ScalarType::Float, gu.rows);
    const void* nr = vector(a[3], "n_rows", gu.dev, ScalarType::Int, 1);
    const Call call(a[4], gu.dev);
    Result h = result(a[2], "out", {gu.rows, f}, gu.t, gu.type);
    const int64_t ldh = matrix(of(h), "out", gu.dev, gu.type, gu.rows, f);
    const moe_status s = moe_swiglu(gu.t.data_ptr(), gu.ld, int32(gu.rows, "rows"), int32(f, "f"),
                                    static_cast<const float*>(rw), static_cast<const int32_t*>(nr), of(h).data_ptr(), ldh,
                                    type_flag(gu.type), call.stream);
    if (s != MOE_OK) return raise_status(s, "moe_swiglu");
    return h.object();
    END_HANDLE_TH_ERRORS
}

// gu, dh, row_weights, dgu, h, drw, with_h, n_rows, stream
PyObject* swiglu_backward(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 9);
    const Operand gu = operand(a[0], "gu");
    const int64_t f = half_cols(gu);
    const Tensor& dh = tensor(a[1], "dh");
    const int64_t lddh = matrix(dh, "dh", gu.dev, gu.type, gu.rows, f);
    const bool weighted = a[2] != Py_None, want_h = a[4] != Py_None || truth(a[6]);
    TORCH_CHECK_VALUE(weighted || a[5] == Py_None, "drw: needs row_weights");
    const void* rw = vector(a[2], "row_weights", gu.dev, ScalarType::Float, gu.rows);
    const void* nr = vector(a[7], "n_rows", gu.dev, ScalarType::Int, 1);
    const Call call(a[8], gu.dev);
    Result dgu = result(a[3], "dgu", {gu.rows, 2 * f}, gu.t, gu.type), h, drw;
    const int64_t lddgu = matrix(of(dgu), "dgu", gu.dev, gu.type, gu.rows, 2 * f);
    int64_t ldh = 0;
    if (want_h) {
        h = result(a[4], "h", {gu.rows, f}, gu.t, gu.type);
        ldh = matrix(of(h), "h", gu.dev, gu.type, gu.rows, f);
    }
    float* dw = nullptr;
    if (weighted) {
        dw = static_cast<float*>(vector(a[5], "drw", gu.dev, ScalarType::Float, gu.rows));
        drw = result(a[5], "drw", {gu.rows}, gu.t, ScalarType::Float);
        if (!dw) dw = static_cast<float*>(of(drw).data_ptr());
    }
    const moe_status s = moe_swiglu_backward(gu.t.data_ptr(), gu.ld, dh.data_ptr(), lddh, int32(gu.rows, "rows"),
                                             int32(f, "f"), static_cast<const float*>(rw), static_cast<const int32_t*>(nr),
                                             of(dgu).data_ptr(), lddgu, want_h ? of(h).data_ptr() : nullptr, ldh, dw,
                                             type_flag(gu.type), call.stream);
    if (s != MOE_OK) return raise_status(s, "moe_swiglu_backward");
    PyObject *o1 = dgu.object(), *o2 = want_h ? h.object() : Py_NewRef(Py_None),
             *o3 = weighted ? drw.object() : Py_NewRef(Py_None);
    PyObject* out = PyTuple_Pack(3, o1, o2, o3);
    Py_DECREF(o1);
    Py_DECREF(o2);
    Py_DECREF(o3);
    return out;
    END_HANDLE_TH_ERRORS
}

// The arguments of an adapter call but its result and workspace, checked.
struct Adapter {
    const Operand x;
    moe_adapter_args p{};
    uint32_t flags;
    ScalarType type;  // of the result
};
uint32_t adapter_flags(PyObject* o) {
    const unsigned long flags = PyLong_AsUnsignedLong(o);  // (the type is the tensors': MOE_OP_FP16 is none of them)
    TORCH_CHECK_VALUE(!PyErr_Occurred() && !(flags & ~(unsigned long)(MOE_OUT_FP32 | MOE_ACCUMULATE)),
                      "flags: a sum of MOE_OUT_FP32 and MOE_ACCUMULATE is expected");
    return (uint32_t)flags;
}
Adapter adapter(PyObject* ox, PyObject* oa, PyObject* ob, PyObject* oids, PyObject* ow, PyObject* oscale, uint32_t flags) {
    Adapter r{operand(ox, "x"), {}, 0, ScalarType::Float};
    const Operand& x = r.x;
    const Tensor &A = tensor(oa, "a"), &B = tensor(ob, "b");
    TORCH_CHECK_VALUE(A.dim() == 3 && B.dim() == 3, "a, b: contiguous [L, rank, k] and [L, n, rank] tensors are expected");
    const int64_t L = A.size(0), rank = A.size(1), n = B.size(1), k = x.cols;
    block(A, "a", x.dev, x.type, {L, rank, k});
    block(B, "b", x.dev, x.type, {L, n, rank});
    TORCH_CHECK_VALUE(oids != Py_None, "ids: a tensor is expected");
    moe_adapter_args& p = r.p;
    p.ids = static_cast<const int32_t*>(vector(oids, "ids", x.dev, ScalarType::Int, x.rows));
    if (ow != Py_None) {
        const Tensor& w = tensor(ow, "w");
        block(w, "w", x.dev, x.type, {n, k});
        p.w = w.data_ptr();
    }
    p.scale = static_cast<const float*>(vector(oscale, "scale", x.dev, ScalarType::Float, L));
    p.x = x.t.data_ptr();
    p.ldx = x.ld;
    p.tokens = int32(x.rows, "tokens");
    p.n = int32(n, "n");
    p.k = int32(k, "k");
    p.a = A.data_ptr();
    p.b = B.data_ptr();
    p.n_adapters = int32(L, "L");
    p.rank = int32(rank, "rank");
    p.workspace_bytes = moe_adapter_workspace(p.tokens, p.rank);
    r.flags = flags | type_flag(x.type);
    r.type = (flags & MOE_OUT_FP32) ? ScalarType::Float : x.type;
    return r;
}

// x, a, b, ids, w, scale, out, flags, stream
PyObject* adapter_project(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 9);
    const uint32_t flags = adapter_flags(a[7]);
    Adapter c = adapter(a[0], a[1], a[2], a[3], a[4], a[5], flags);
    moe_adapter_args& p = c.p;
    TORCH_CHECK_VALUE(!(flags & MOE_ACCUMULATE) || a[6] != Py_None, "MOE_ACCUMULATE adds to a given out");
    const Call call(a[8], c.x.dev);
    Result y = result(a[6], "out", {c.x.rows, p.n}, c.x.t, c.type);
    p.ldy = matrix(of(y), "out", c.x.dev, c.type, c.x.rows, p.n);
    p.y = of(y).data_ptr();
    const Tensor workspace = at::empty({(int64_t)p.workspace_bytes}, c.x.t.options().dtype(ScalarType::Byte));
    p.workspace = workspace.data_ptr();
    const moe_status s = moe_adapter_project(&p, c.flags, call.stream);
    if (s != MOE_OK) return raise_status(s, "moe_adapter_project");
    return y.object();
    END_HANDLE_TH_ERRORS
}

// What MoeLayer.forward_adapted needs before the layer writes y: x [T, d] bf16 and y (or None) [T, d] contiguous, and
// adapters of this shape that the operator takes.
// x, a, b, ids, scale, y, flags, d, stream
PyObject* adapter_beside(PyObject*, PyObject* const* a, Py_ssize_t count) {
    HANDLE_TH_ERRORS
    arguments(count, 9);
    Adapter c = adapter(a[0], a[1], a[2], a[3], Py_None, a[4], adapter_flags(a[6]));
    moe_adapter_args& p = c.p;
    const int64_t d = PyLong_AsLongLong(a[7]);
    TORCH_CHECK_VALUE(c.x.type == ScalarType::BFloat16 && c.x.cols == d && c.x.t.is_contiguous(),
                      "x: a contiguous [T, ", d, "] bf16 tensor is expected, not ", c.x.t.sizes(), " of ", c.x.t.scalar_type());
    TORCH_CHECK_VALUE(p.n == d, "b: ", d, " features are expected, not ", p.n);
    p.ldy = d;
    p.y = reinterpret_cast<void*>(16);  // (these two are allocated later: aligned)
    p.workspace = reinterpret_cast<void*>(32);
    if (a[5] != Py_None) {
        const Tensor& y = tensor(a[5], "y");
        block(y, "y", c.x.dev, c.type, {c.x.rows, d});
        if (y.data_ptr() != p.x) p.y = y.data_ptr();  // (y may be x, where the adapters read the normalised copy)
    }
    const Call call(a[8], c.x.dev);  // (a stream of another device)
    const moe_status s = moe_adapter_check(&p, c.flags);
    if (s != MOE_OK) return raise_status(s, "moe_adapter_check");
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_INCREF(cls);
    Py_XSETREF(g_moe_error, cls);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{"grouped_matmul", FAST(grouped_matmul), nullptr},
                          {"grouped_wgrad", FAST(grouped_wgrad), nullptr},
                          {"swiglu", FAST(swiglu), nullptr},
                          {"swiglu_backward", FAST(swiglu_backward), nullptr},
                          {"adapter_project", FAST(adapter_project), nullptr},
                          {"adapter_beside", FAST(adapter_beside), nullptr},
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ops16", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops16() { return PyModule_Create(&kModule); }
