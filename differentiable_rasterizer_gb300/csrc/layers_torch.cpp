// layers_torch.cpp -- the decoder layers on torch tensors, natively: argument checks,
// allocation of outputs and scratch on the current stream, and the calls of the C ABI
// (include/gs.h).  layers.py is its Python face and states what each function takes.
//
// A layer call is a few microseconds of GPU work for single tokens; the same steps in
// Python cost the host 12 (linear) to 30 microseconds (its gradients).
//
// The C ABI's functions come from the library that abi.py has loaded (bind); torch is
// used for device memory and streams alone.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/gs.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Library {
    decltype(&gs_rms_norm) rms_norm;
    decltype(&gs_rms_norm_bwd) rms_norm_bwd;
    decltype(&gs_quantize_rows) quantize_rows;
    decltype(&gs_linear) linear;
    decltype(&gs_linear_bwd) linear_bwd;
    decltype(&gs_glu) glu;
    decltype(&gs_glu_bwd) glu_bwd;
};
Library lib = {};
PyObject* gs_error = nullptr;   // abi.GsError

// ------------------------------------------------------------------ refusals
struct Refusal {
    std::string what;
};
struct Failure {   // a status of the library
    const char* call;
    int status;
};
[[noreturn]] void refuse(const std::string& what) { throw Refusal{what}; }

std::string shape_of(const Tensor& t)
{
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    s += "] strides [";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
    return s + "]";
}

constexpr unsigned kF32 = 1u << GS_F32, kBf16 = 1u << GS_BF16, kF16 = 1u << GS_F16, kE4m3 = 1u << GS_E4M3;
constexpr unsigned kHalf = kBf16 | kF16, kFloat = kF32 | kHalf;

int type_code(ScalarType t)   // -1: not one of the layers'
{
    switch (t) {
        case ScalarType::Float: return GS_F32;
        case ScalarType::BFloat16: return GS_BF16;
        case ScalarType::Half: return GS_F16;
        case ScalarType::Float8_e4m3fn: return GS_E4M3;
        default: return -1;
    }
}
ScalarType scalar_type(int code)
{
    return code == GS_F32    ? ScalarType::Float
           : code == GS_BF16 ? ScalarType::BFloat16
           : code == GS_F16  ? ScalarType::Half
                             : ScalarType::Float8_e4m3fn;
}
std::string types_of(unsigned mask)
{
    std::string s;
    for (int c = 0; c < 4; ++c)
        if (mask >> c & 1) s += (s.empty() ? "" : ", ") + std::string(c10::toString(scalar_type(c)));
    return s;
}

const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
    const Tensor& t = THPVariable_Unpack(o);
    // results have no grad_fn: a gradient would be lost without a word
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(std::string(name) + ": requires grad, which the layers do not record; call under torch.no_grad() or detach it, "
                                   "and take the gradients from the *_backward functions");
    return t;
}

// The device of a call: its first tensor's, made current while the call runs.
int cuda_device(const Tensor& t, const char* name)
{
    if (!t.is_cuda()) refuse(std::string(name) + ": expected a CUDA tensor, got one on " + t.device().str());
    return t.get_device();
}

void check_kind(const Tensor& t, const char* name, unsigned types, int dev)
{
    const int c = type_code(t.scalar_type());
    if (c < 0 || !(types >> c & 1))
        refuse(std::string(name) + ": expected " + types_of(types) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_cuda() || t.get_device() != dev)
        refuse(std::string(name) + ": on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
}

// A tensor as rows of its last dimension: the leading dimensions merge into one stride.
struct Rows {
    void* p = nullptr;
    int64_t ld = 0, rows = 0, cols = 0;
    int type = 0;
};

Rows rows_of(const Tensor& t, const char* name, unsigned types, int dev, int64_t cols = -1, int64_t rows = -1)
{
    check_kind(t, name, types, dev);
    const int64_t d = t.dim();
    if (d == 0) refuse(std::string(name) + ": needs at least one dimension");
    Rows r;
    r.type = type_code(t.scalar_type());
    r.cols = t.size(d - 1);
    r.rows = 1;
    for (int64_t i = 0; i + 1 < d; ++i) r.rows *= t.size(i);
    if (cols >= 0 && r.cols != cols)
        refuse(std::string(name) + ": " + std::to_string(r.cols) + " columns, expected " + std::to_string(cols));
    if (rows >= 0 && r.rows != rows)
        refuse(std::string(name) + ": " + std::to_string(r.rows) + " rows, expected " + std::to_string(rows));
    if (r.cols > 1 && t.stride(d - 1) != 1)
        refuse(std::string(name) + ": the last dimension is not contiguous, " + shape_of(t));
    // the pitch of a single row is never used: one that keeps the row aligned
    r.ld = (r.cols + 15) / 16 * 16;
    if (r.rows > 1) {
        int64_t stride = -1, count = 1;   // of the merged leading dimensions, from the innermost out
        for (int64_t i = d - 2; i >= 0; --i) {
            if (t.size(i) == 1) continue;
            if (stride < 0) stride = t.stride(i);
            else if (t.stride(i) != stride * count)
                refuse(std::string(name) + ": leading dimensions do not merge into one stride, " + shape_of(t));
            count *= t.size(i);
        }
        if (stride < r.cols) refuse(std::string(name) + ": rows overlap, " + shape_of(t));
        r.ld = stride;
    }
    r.p = t.data_ptr();
    return r;
}

// A contiguous vector, or nullptr for None.
void* vector_of(PyObject* o, const char* name, unsigned types, int dev, int64_t size, int* type = nullptr)
{
    if (o == Py_None) return nullptr;
    const Tensor& t = tensor(o, name);
    check_kind(t, name, types, dev);
    if (t.numel() != size || !t.is_contiguous())
        refuse(std::string(name) + ": expected " + std::to_string(size) + " contiguous values, got " + shape_of(t));
    if (type) *type = type_code(t.scalar_type());
    return t.data_ptr();
}
void* required(void* p, const char* name, int64_t size)
{
    if (!p && size > 0) refuse(std::string(name) + ": required");
    return p;
}

int type_arg(PyObject* o, const char* name, unsigned types, int fallback)
{
    if (o == Py_None) return fallback;
    if (!THPDtype_Check(o)) refuse(std::string(name) + ": expected a torch.dtype, got " + Py_TYPE(o)->tp_name);
    const ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
    const int c = type_code(t);
    if (c < 0 || !(types >> c & 1))
        refuse(std::string(name) + ": " + c10::toString(t) + " is not one of " + types_of(types));
    return c;
}

bool flag(PyObject* o, const char* name)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        refuse(std::string(name) + ": expected a truth value, got " + Py_TYPE(o)->tp_name);
    }
    return v == 1;
}
float number(PyObject* o, const char* name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + ": expected a number, got " + Py_TYPE(o)->tp_name);
    }
    return (float)v;
}
int code(PyObject* o) { return (int)PyLong_AsLong(o); }   // of layers.py's own table

// ------------------------------------------------------------------ outputs
// [*lead, cols] like `like`'s leading dimensions, rows padded to 16 bytes.
struct Out {
    Tensor t;
    Rows r;
};
Out output(const Tensor& like, int64_t rows, int64_t cols, int type)
{
    const int64_t per = type == GS_F32 ? 4 : (type == GS_E4M3 ? 16 : 8), ld = (cols + per - 1) / per * per;
    c10::SmallVector<int64_t, 5> shape(like.sizes().begin(), like.sizes().end());
    shape.back() = ld;
    Out o;
    o.t = at::empty(shape, like.options().dtype(scalar_type(type)));
    o.r.p = o.t.data_ptr();
    o.r.ld = ld, o.r.rows = rows, o.r.cols = cols, o.r.type = type;
    if (ld != cols) o.t = o.t.narrow(-1, 0, cols);
    return o;
}
Tensor row_values(const Tensor& like)   // one fp32 value a row
{
    return at::empty(like.sizes().slice(0, like.dim() - 1), like.options().dtype(ScalarType::Float));
}
Tensor plain(const Tensor& like, at::IntArrayRef shape, int type)
{
    return at::empty(shape, like.options().dtype(scalar_type(type)));
}

PyObject* wrap(const Tensor& t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}
template <class... T>
PyObject* result(const T&... t)
{
    PyObject* items[] = {wrap(t)...};
    PyObject* r = PyTuple_New(sizeof...(T));
    for (size_t i = 0; i < sizeof...(T); ++i) PyTuple_SET_ITEM(r, (Py_ssize_t)i, items[i]);
    return r;
}

void check(const char* call, gs_status s)
{
    if (s != GS_OK) throw Failure{call, (int)s};
}

// A call with the scratch that it asks for.  first: it mostly needs none.
template <class F, class Args>
void with_scratch(const char* name, F f, const Args& args, const Tensor& like, int dev, bool first)
{
    void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    if (first) {
        const gs_status s = f(&args, nullptr, nullptr, stream);
        if (s == GS_OK) return;
        if (s != GS_ERR_INVALID_ARG) throw Failure{name, (int)s};   // else it needs scratch, or the query says why not
    }
    size_t bytes = 0;
    check(name, f(&args, nullptr, &bytes, nullptr));
    if (bytes == 0) {
        check(name, f(&args, nullptr, nullptr, stream));
        return;
    }
    const Tensor ws = at::empty({(int64_t)bytes}, like.options().dtype(ScalarType::Byte));
    check(name, f(&args, ws.data_ptr(), &bytes, stream));
}

// Runs f, turning refusals into ValueError and the library's statuses into abi.GsError.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f)
{
    HANDLE_TH_ERRORS
    if (got != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
        return nullptr;
    }
    try {
        return f();
    } catch (const Refusal& r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const Failure& e) {
        if (PyObject* x = PyObject_CallFunction(gs_error, "si", e.call, e.status)) {
            PyErr_SetObject(gs_error, x);
            Py_DECREF(x);
        }
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ the layers
// (x, weight, residual, eps, out_dtype, need_backward) -> (y, scale, s, rstd)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 6, [&] {
        const Tensor& x = tensor(a[0], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kFloat, dev);
        gs_rms_norm_args g = {};
        g.rows = rx.rows, g.cols = rx.cols, g.x = rx.p, g.ldx = rx.ld, g.type = rx.type;
        g.weight = required(vector_of(a[1], "weight", kFloat, dev, rx.cols, &g.weight_type), "weight", 1);
        g.eps = number(a[3], "eps");
        g.y_type = type_arg(a[4], "out_dtype", kFloat | kE4m3, rx.type);
        Tensor s = x, scale, rstd;
        if (a[2] != Py_None) {
            const Rows r = rows_of(tensor(a[2], "residual"), "residual", 1u << rx.type, dev, rx.cols, rx.rows);
            const Out o = output(x, rx.rows, rx.cols, rx.type);
            g.residual = r.p, g.ldr = r.ld, g.sum = o.r.p, g.lds = o.r.ld;
            s = o.t;
        }
        const Out y = output(x, rx.rows, rx.cols, g.y_type);
        g.y = y.r.p, g.ldy = y.r.ld;
        if (g.y_type == GS_E4M3) g.y_scale = (scale = row_values(x)).data_ptr<float>();
        if (flag(a[5], "need_backward")) g.rstd = (rstd = row_values(x)).data_ptr<float>();
        if (rx.rows) check("gs_rms_norm", lib.rms_norm(&g, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()));
        return result(y.t, scale, s, rstd);
    });
}

// (dy, s, weight, rstd, ds) -> (dx, dweight)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 5, [&] {
        const Tensor& s = tensor(a[1], "s");
        const int dev = cuda_device(s, "s");
        const c10::cuda::OptionalCUDAGuard guard(s.device());
        const Rows rs = rows_of(s, "s", kFloat, dev);
        const Rows dy = rows_of(tensor(a[0], "dy"), "dy", kFloat, dev, rs.cols, rs.rows);
        gs_rms_norm_bwd_args g = {};
        g.rows = rs.rows, g.cols = rs.cols, g.dy = dy.p, g.lddy = dy.ld, g.dy_type = dy.type;
        g.sum = rs.p, g.lds = rs.ld, g.type = rs.type;
        g.weight = required(vector_of(a[2], "weight", kFloat, dev, rs.cols, &g.weight_type), "weight", 1);
        g.rstd = (const float*)required(vector_of(a[3], "rstd", kF32, dev, rs.rows), "rstd (rms_norm's with need_backward)", rs.rows);
        if (a[4] != Py_None) {
            const Rows ds = rows_of(tensor(a[4], "ds"), "ds", 1u << rs.type, dev, rs.cols, rs.rows);
            g.dsum = ds.p, g.ldds = ds.ld;
        }
        const Out dx = output(s, rs.rows, rs.cols, rs.type);
        g.dx = dx.r.p, g.lddx = dx.r.ld;
        const Tensor dw = plain(s, THPVariable_Unpack(a[2]).sizes(), g.weight_type);
        g.dweight = dw.data_ptr();
        with_scratch("gs_rms_norm_bwd", lib.rms_norm_bwd, g, s, dev, false);
        return result(dx.t, dw);
    });
}

// (x) -> (q, scale)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 1, [&] {
        const Tensor& x = tensor(a[0], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kFloat, dev);
        const Out q = output(x, rx.rows, rx.cols, GS_E4M3);
        const Tensor scale = row_values(x);
        gs_quantize_rows_args g = {};
        g.rows = rx.rows, g.cols = rx.cols, g.x = rx.p, g.ldx = rx.ld, g.type = rx.type;
        g.q = q.r.p, g.ldq = q.r.ld, g.scale = scale.data_ptr<float>();
        if (rx.rows)
            check("gs_quantize_rows", lib.quantize_rows(&g, c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()));
        return result(q.t, scale);
    });
}

// (x, w, bias, x_scale, w_scale, act, residual, out, out_dtype, need_backward) -> (y, z)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const Tensor& x = tensor(a[0], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kHalf | kE4m3, dev);
        const Rows w = rows_of(tensor(a[1], "w"), "w", 1u << rx.type, dev, rx.cols);
        gs_linear_args g = {};
        g.rows = rx.rows, g.in_features = rx.cols, g.out_features = w.rows;
        g.x = rx.p, g.ldx = rx.ld, g.w = w.p, g.ldw = w.ld, g.type = rx.type;
        g.bias = vector_of(a[2], "bias", kFloat, dev, w.rows, &g.bias_type);
        g.x_scale = (const float*)vector_of(a[3], "x_scale", kF32, dev, rx.rows);
        g.w_scale = (const float*)vector_of(a[4], "w_scale", kF32, dev, w.rows);
        g.act = code(a[5]);
        int type = rx.type == GS_E4M3 ? GS_BF16 : rx.type;
        if (a[6] != Py_None) type = type_code(tensor(a[6], "residual").scalar_type());
        if (a[7] != Py_None) type = type_code(tensor(a[7], "out").scalar_type());
        if (type < 0 || !(kFloat >> type & 1)) refuse("out, residual: expected " + types_of(kFloat));
        g.out_type = type_arg(a[8], "out_dtype", kFloat, type);
        if (a[6] != Py_None) {
            const Rows r = rows_of(tensor(a[6], "residual"), "residual", 1u << g.out_type, dev, w.rows, rx.rows);
            g.residual = r.p, g.ldr = r.ld;
        }
        Tensor y, z;
        if (a[7] != Py_None) {
            y = tensor(a[7], "out");
            const Rows r = rows_of(y, "out", 1u << g.out_type, dev, w.rows, rx.rows);
            g.y = r.p, g.ldy = r.ld;
        } else {
            const Out o = output(x, rx.rows, w.rows, g.out_type);
            y = o.t;
            g.y = o.r.p, g.ldy = o.r.ld;
        }
        if (flag(a[9], "need_backward") && g.act != GS_ACT_NONE) {
            if (rx.type == GS_E4M3) refuse("need_backward: 8-bit operands have no gradients");
            const Out o = output(x, rx.rows, w.rows, rx.type);
            z = o.t;
            g.z = o.r.p, g.ldz = o.r.ld;
        }
        with_scratch("gs_linear", lib.linear, g, x, dev, true);
        // written in place: autograd has to see it where y is saved for a backward
        if (a[7] != Py_None && !y.is_inference()) y.unsafeGetTensorImpl()->bump_version();
        return result(y, z);
    });
}

// (dy, x, w, z, act, bias, need_dx, need_dw, dw_dtype, db_dtype) -> (dx, dw, db)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const Tensor& x = tensor(a[1], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kHalf, dev);
        const Rows w = rows_of(tensor(a[2], "w"), "w", 1u << rx.type, dev, rx.cols);
        const Rows dy = rows_of(tensor(a[0], "dy"), "dy", kFloat, dev, w.rows, rx.rows);
        gs_linear_bwd_args g = {};
        g.rows = rx.rows, g.in_features = rx.cols, g.out_features = w.rows;
        g.dy = dy.p, g.lddy = dy.ld, g.dy_type = dy.type;
        g.x = rx.p, g.ldx = rx.ld, g.w = w.p, g.ldw = w.ld, g.type = rx.type;
        g.act = code(a[4]);
        if (g.act != GS_ACT_NONE) {
            if (a[3] == Py_None) refuse("z: required with an activation (linear's with need_backward)");
            const Rows z = rows_of(tensor(a[3], "z"), "z", 1u << rx.type, dev, w.rows, rx.rows);
            g.z = z.p, g.ldz = z.ld;
        }
        g.dw_type = type_arg(a[8], "dw_dtype", 1u << rx.type | kF32, rx.type);
        g.db_type = type_arg(a[9], "db_dtype", kFloat, rx.type);
        Tensor dx, dw, db;
        if (flag(a[6], "need_dx")) {
            const Out o = output(x, rx.rows, rx.cols, rx.type);
            dx = o.t;
            g.dx = o.r.p, g.lddx = o.r.ld;
        }
        if (flag(a[7], "need_dw")) {
            dw = plain(x, {w.rows, rx.cols}, g.dw_type);
            g.dw = dw.data_ptr(), g.lddw = rx.cols;
        }
        if (flag(a[5], "bias")) g.db = (db = plain(x, {w.rows}, g.db_type)).data_ptr();
        with_scratch("gs_linear_bwd", lib.linear_bwd, g, x, dev, false);
        return result(dx, dw, db);
    });
}

// (x, w_gate, w_up, x_scale, gate_scale, up_scale, act, out_dtype, save) -> (h, g, u)
PyObject* glu(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 9, [&] {
        const Tensor& x = tensor(a[0], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kHalf | kE4m3, dev);
        const Rows wg = rows_of(tensor(a[1], "w_gate"), "w_gate", 1u << rx.type, dev, rx.cols);
        const Rows wu = rows_of(tensor(a[2], "w_up"), "w_up", 1u << rx.type, dev, rx.cols, wg.rows);
        gs_glu_args g = {};
        g.rows = rx.rows, g.in_features = rx.cols, g.hidden = wg.rows;
        g.x = rx.p, g.ldx = rx.ld, g.type = rx.type;
        g.w_gate = wg.p, g.ldwg = wg.ld, g.w_up = wu.p, g.ldwu = wu.ld;
        g.x_scale = (const float*)vector_of(a[3], "x_scale", kF32, dev, rx.rows);
        g.gate_scale = (const float*)vector_of(a[4], "gate_scale", kF32, dev, wg.rows);
        g.up_scale = (const float*)vector_of(a[5], "up_scale", kF32, dev, wg.rows);
        g.act = code(a[6]);
        g.out_type = type_arg(a[7], "out_dtype", rx.type == GS_E4M3 ? kHalf : 1u << rx.type,
                              rx.type == GS_E4M3 ? GS_BF16 : rx.type);
        const Out h = output(x, rx.rows, wg.rows, g.out_type);
        g.h = h.r.p, g.ldh = h.r.ld;
        Tensor gate, up;
        if (flag(a[8], "save")) {
            if (rx.type == GS_E4M3) refuse("need_backward: 8-bit operands have no gradients");
            const Out og = output(x, rx.rows, wg.rows, g.out_type), ou = output(x, rx.rows, wg.rows, g.out_type);
            gate = og.t, up = ou.t;
            g.g = og.r.p, g.ldg = og.r.ld, g.u = ou.r.p, g.ldu = ou.r.ld;
        }
        with_scratch("gs_glu", lib.glu, g, x, dev, true);
        return result(h.t, gate, up);
    });
}

// (dh, x, w_gate, w_up, g, u, act, need_dx, need_dw, dw_dtype) -> (dx, dw_gate, dw_up)
PyObject* glu_backward(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    return guarded(n, 10, [&] {
        const Tensor& x = tensor(a[1], "x");
        const int dev = cuda_device(x, "x");
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const Rows rx = rows_of(x, "x", kHalf, dev);
        const unsigned type = 1u << rx.type;
        const Rows wg = rows_of(tensor(a[2], "w_gate"), "w_gate", type, dev, rx.cols);
        const Rows wu = rows_of(tensor(a[3], "w_up"), "w_up", type, dev, rx.cols, wg.rows);
        const Rows dh = rows_of(tensor(a[0], "dh"), "dh", type, dev, wg.rows, rx.rows);
        gs_glu_bwd_args g = {};
        g.rows = rx.rows, g.in_features = rx.cols, g.hidden = wg.rows;
        g.dh = dh.p, g.lddh = dh.ld, g.x = rx.p, g.ldx = rx.ld, g.type = rx.type;
        g.w_gate = wg.p, g.ldwg = wg.ld, g.w_up = wu.p, g.ldwu = wu.ld;
        if (a[4] != Py_None || a[5] != Py_None) {
            const Rows rg = rows_of(tensor(a[4], "g"), "g", type, dev, wg.rows, rx.rows);
            const Rows ru = rows_of(tensor(a[5], "u"), "u", type, dev, wg.rows, rx.rows);
            g.g = rg.p, g.ldg = rg.ld, g.u = ru.p, g.ldu = ru.ld;
        }
        g.act = code(a[6]);
        g.dw_type = type_arg(a[9], "dw_dtype", type | kF32, rx.type);
        Tensor dx, dwg, dwu;
        if (flag(a[7], "need_dx")) {
            const Out o = output(x, rx.rows, rx.cols, rx.type);
            dx = o.t;
            g.dx = o.r.p, g.lddx = o.r.ld;
        }
        if (flag(a[8], "need_dw")) {
            dwg = plain(x, {wg.rows, rx.cols}, g.dw_type);
            dwu = plain(x, {wg.rows, rx.cols}, g.dw_type);
            g.dw_gate = dwg.data_ptr(), g.lddwg = rx.cols, g.dw_up = dwu.data_ptr(), g.lddwu = rx.cols;
        }
        with_scratch("gs_glu_bwd", lib.glu_bwd, g, x, dev, false);
        return result(dx, dwg, dwu);
    });
}

// bind(GsError, address of gs_rms_norm, ..._bwd, quantize_rows, linear, linear_bwd, glu, glu_bwd)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n)
{
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "bind: 8 arguments");
        return nullptr;
    }
    void* f[7];
    for (int i = 0; i < 7; ++i) {
        f[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!f[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function");
            return nullptr;
        }
    }
    lib.rms_norm = reinterpret_cast<decltype(lib.rms_norm)>(f[0]);
    lib.rms_norm_bwd = reinterpret_cast<decltype(lib.rms_norm_bwd)>(f[1]);
    lib.quantize_rows = reinterpret_cast<decltype(lib.quantize_rows)>(f[2]);
    lib.linear = reinterpret_cast<decltype(lib.linear)>(f[3]);
    lib.linear_bwd = reinterpret_cast<decltype(lib.linear_bwd)>(f[4]);
    lib.glu = reinterpret_cast<decltype(lib.glu)>(f[5]);
    lib.glu_bwd = reinterpret_cast<decltype(lib.glu_bwd)>(f[6]);
    Py_INCREF(a[0]);
    Py_XDECREF(gs_error);
    gs_error = a[0];
    Py_RETURN_NONE;
}

#define GS_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {GS_FAST(bind),          GS_FAST(rms_norm), GS_FAST(rms_norm_backward), GS_FAST(quantize_rows),
                         GS_FAST(linear),        GS_FAST(linear_backward), GS_FAST(glu),       GS_FAST(glu_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_torch() { return PyModule_Create(&module); }
