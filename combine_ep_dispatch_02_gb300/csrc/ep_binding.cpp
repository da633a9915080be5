// ep_binding.cpp -- native half of the Python binding of the expert-layer operators: checks tensors,
// allocates outputs and workspaces on the current stream, and calls the C ABI of libep.so.
//
// These calls are often one token's, a few microseconds on the GPU, so marshalling must not cost more than
// that.  The module holds no logic of the operators; libep.so is reached through the addresses given
// to bind(), so whichever build of the library the package has loaded is the one that runs.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "ep.h"

namespace {

decltype(&ep_rms_norm_fp8) g_norm;
decltype(&ep_sort_workspace_bytes) g_sort_bytes;
decltype(&ep_sort_by_expert) g_sort;
decltype(&ep_sorted_rows) g_rows;
decltype(&ep_return_rows) g_return;
decltype(&ep_return_rows_backward) g_back;
decltype(&ep_matmul_fp8) g_matmul;
decltype(&ep_strerror) g_strerror;
decltype(&ep_last_error) g_last_error;
PyObject* g_error;         // the package's EpError
PyObject* g_make_status;   // device index -> address of its status word
int32_t* g_status[64];

// A Python exception is set: unwinds to the entry point.
struct Raised {};

[[noreturn]] void raise(int code, const char* msg)
{
    PyObject* e = PyObject_CallFunction(g_error, "is", code, msg);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

[[noreturn]] void refuse(const char* fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    raise(EP_ERR_ARG, msg);
}

void check(int rc)
{
    if (rc != EP_OK) raise(rc, (std::string(g_strerror(rc)) + ": " + g_last_error()).c_str());
}

std::string shape_text(at::IntArrayRef s)
{
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char* type_text(at::ScalarType t) { return c10::toString(t); }

const at::Tensor& tensor(PyObject* o, const char* what)
{
    if (!THPVariable_Check(o)) refuse("%s is a %s, not a tensor", what, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

// The tensor that decides where the call runs.
const at::Tensor& lead_tensor(PyObject* o, const char* what)
{
    const at::Tensor& t = tensor(o, what);
    if (!t.is_cuda()) refuse("%s is on %s, not a CUDA device", what, t.device().str().c_str());
    return t;
}

// Address of a tensor that has to be contiguous, of this type and shape, on this device.
void* data(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape, at::Device device)
{
    if (t.device() != device)
        refuse("%s is on %s, the call runs on %s", what, t.device().str().c_str(), device.str().c_str());
    if (t.scalar_type() != type) refuse("%s is %s, the call takes %s", what, type_text(t.scalar_type()), type_text(type));
    if (t.sizes() != shape)
        refuse("%s has shape %s, the call takes %s", what, shape_text(t.sizes()).c_str(), shape_text(shape).c_str());
    if (!t.is_contiguous()) refuse("%s is not contiguous", what);
    return t.data_ptr();
}

void* data_or_null(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, at::Device device)
{
    return o == Py_None ? nullptr : data(tensor(o, what), what, type, shape, device);
}

int half_code(const at::Tensor& t, const char* what)
{
    if (t.scalar_type() == at::kBFloat16) return EP_BF16;
    if (t.scalar_type() == at::kHalf) return EP_FP16;
    refuse("%s is %s, the call takes BFloat16 or Half", what, type_text(t.scalar_type()));
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device device)
{
    return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

int32_t* status(at::Device device)
{
    const int i = device.index();
    if (i < 0 || i >= 64) refuse("device index %d outside 0..63", i);
    if (!g_status[i]) {
        PyObject* a = PyObject_CallFunction(g_make_status, "i", i);
        if (!a) throw Raised{};
        g_status[i] = (int32_t*)PyLong_AsVoidPtr(a);
        Py_DECREF(a);
        if (PyErr_Occurred()) throw Raised{};
    }
    return g_status[i];
}

void* stream(at::Device device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

int64_t whole(PyObject* o, const char* what)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("%s is not a whole number of 64 bits", what);
    }
    return v;
}

int small(PyObject* o, const char* what)
{
    const int64_t v = whole(o, what);
    if (v < INT32_MIN || v > INT32_MAX) refuse("%s=%lld outside 32 bits", what, (long long)v);
    return (int)v;
}

// Sizes go to the C ABI as int; it refuses what is out of its range, so a larger one becomes the largest.
int clamp_int(int64_t v) { return v > INT32_MAX ? INT32_MAX : (int)v; }

PyObject* wrap(at::Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); }

PyObject* pack(std::initializer_list<at::Tensor> ts)
{
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    Py_ssize_t i = 0;
    for (const at::Tensor& t : ts) {
        PyObject* o = r ? wrap(t) : nullptr;
        if (!o) {
            Py_XDECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

void* get(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

// (x, weight, residual, eps, want_y)
PyObject* rms_norm(PyObject* const* v)
{
    const at::Tensor& x = lead_tensor(v[0], "x");
    const int code = half_code(x, "x");
    if (x.dim() != 2) refuse("x has %lld dimensions, the call takes [rows][hidden]", (long long)x.dim());
    const at::Device dev = x.device();
    const int64_t rows = x.size(0), hidden = x.size(1);
    if (hidden > 1 && x.stride(1) != 1) refuse("x: the elements of a row are not consecutive");
    const void* rp = nullptr;
    int64_t pitch = rows > 1 ? x.stride(0) : hidden, rpitch = hidden;
    if (v[2] != Py_None) {
        const at::Tensor& r = tensor(v[2], "residual");
        if (r.device() != dev || r.scalar_type() != x.scalar_type() || r.sizes() != x.sizes())
            refuse("residual is %s %s on %s, x is %s %s on %s", type_text(r.scalar_type()), shape_text(r.sizes()).c_str(),
                   r.device().str().c_str(), type_text(x.scalar_type()), shape_text(x.sizes()).c_str(), dev.str().c_str());
        if (hidden > 1 && r.stride(1) != 1) refuse("residual: the elements of a row are not consecutive");
        rp = r.data_ptr();
        if (rows > 1) rpitch = r.stride(0);
    }
    const at::Tensor& w = tensor(v[1], "weight");
    const bool wide = w.scalar_type() == at::kFloat;
    const void* wp = data(w, "weight", wide ? at::kFloat : x.scalar_type(), {hidden}, dev);
    const double eps = PyFloat_AsDouble(v[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const int want_y = PyObject_IsTrue(v[4]);
    if (want_y < 0) throw Raised{};
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor q = empty(x.sizes(), at::kFloat8_e4m3fn, dev), s = empty({rows, (hidden + 127) / 128}, at::kFloat, dev), h, y;
    if (rp) h = empty(x.sizes(), x.scalar_type(), dev);
    if (want_y) y = empty(x.sizes(), x.scalar_type(), dev);
    check(g_norm(x.data_ptr(), pitch, rp, rpitch, wp, wide, code, rows, clamp_int(hidden), (float)eps, q.data_ptr(),
                 (float*)s.data_ptr(), get(h), get(y), stream(dev)));
    return pack({q, s, h, y});
}

// (indices, experts, max_rows or None, counts)
PyObject* sort_by_expert(PyObject* const* v)
{
    const at::Tensor& idx = lead_tensor(v[0], "indices");
    const int64_t dims = idx.dim();
    if (dims != 2 && dims != 3)
        refuse("indices has %lld dimensions, the call takes [rows][k] or [W][rows][k]", (long long)dims);
    const at::Device dev = idx.device();
    const int64_t W = dims == 3 ? idx.size(0) : 1, rows = idx.size(dims - 2), k = idx.size(dims - 1);
    const void* ip = data(idx, "indices", at::kInt, idx.sizes(), dev);
    const void* cp = data_or_null(v[3], "counts", at::kInt, {W}, dev);
    const int experts = small(v[1], "experts");
    const int64_t max_rows = v[2] == Py_None ? W * rows * k : whole(v[2], "max_rows");
    if (max_rows < 0) refuse("max_rows=%lld < 0", (long long)max_rows);
    const c10::cuda::CUDAGuard guard(dev);
    const size_t need = g_sort_bytes(clamp_int(W), rows, clamp_int(k), experts);
    at::Tensor work;
    if (need) work = empty({(int64_t)need}, at::kByte, dev);
    // an order that the C ABI refuses gets no storage for its groups
    const int64_t groups = experts > 0 && W * (int64_t)experts < (int64_t)1 << 31 ? W * experts : 0;
    at::Tensor offsets = empty({groups + 1}, at::kInt, dev), pos = empty(idx.sizes(), at::kInt, dev),
               src = empty({max_rows}, at::kInt, dev);
    check(g_sort((const int32_t*)ip, (const int32_t*)cp, clamp_int(W), rows, clamp_int(k), experts, max_rows,
                 (int32_t*)offsets.data_ptr(), (int32_t*)pos.data_ptr(), (int32_t*)src.data_ptr(), get(work), need,
                 status(dev), stream(dev)));
    return pack({offsets, pos, src});
}

// An order's pos, src and counts, for rows of shape lead.
struct Order {
    int64_t W, rows, k, max_rows;
    const int32_t *pos, *counts;
};

Order order_args(PyObject* pos_o, PyObject* src_o, PyObject* counts_o, at::IntArrayRef lead, at::Device dev)
{
    const at::Tensor& pos = tensor(pos_o, "order.pos");
    const at::Tensor& src = tensor(src_o, "order.src");
    if ((pos.dim() != 2 && pos.dim() != 3) || pos.sizes().slice(0, pos.dim() - 1) != lead)
        refuse("order.pos has shape %s, the rows are %s", shape_text(pos.sizes()).c_str(), shape_text(lead).c_str());
    if (src.dim() != 1) refuse("order.src has %lld dimensions, the call takes [max_rows]", (long long)src.dim());
    Order o;
    o.W = pos.dim() == 3 ? pos.size(0) : 1;
    o.rows = pos.size(pos.dim() - 2);
    o.k = pos.size(pos.dim() - 1);
    o.max_rows = src.size(0);
    o.pos = (const int32_t*)data(pos, "order.pos", at::kInt, pos.sizes(), dev);
    o.counts = (const int32_t*)data_or_null(counts_o, "order.counts", at::kInt, {o.W}, dev);
    return o;
}

// (pos, src, counts, x, scales)
PyObject* sorted_rows(PyObject* const* v)
{
    const at::Tensor& x = lead_tensor(v[3], "x");
    if (x.dim() < 2) refuse("x has %lld dimensions, the call takes [rows][hidden] or [W][rows][hidden]", (long long)x.dim());
    const at::Device dev = x.device();
    const at::IntArrayRef lead = x.sizes().slice(0, x.dim() - 1);
    const Order o = order_args(v[0], v[1], v[2], lead, dev);
    const void* xp = data(x, "x", x.scalar_type(), x.sizes(), dev);
    const int64_t width = x.size(-1);
    int64_t sd = 0;
    const void* sp = nullptr;
    if (v[4] != Py_None) {
        const at::Tensor& s = tensor(v[4], "scales");
        if (s.dim() < 1) refuse("scales has no dimensions");
        sd = s.size(-1);
        std::vector<int64_t> shape(lead.begin(), lead.end());
        shape.push_back(sd);
        sp = data(s, "scales", at::kFloat, shape, dev);
    }
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out = empty({o.max_rows, width}, x.scalar_type(), dev), out_s;
    if (v[4] != Py_None) out_s = empty({o.max_rows, sd}, at::kFloat, dev);
    check(g_rows(xp, (const float*)sp, o.pos, o.counts, clamp_int(o.W), o.rows, clamp_int(o.k), o.max_rows,
                 width * (int64_t)x.element_size(), clamp_int(sd), out.data_ptr(), sd ? (float*)out_s.data_ptr() : nullptr,
                 status(dev), stream(dev)));
    return pack({out, out_s});
}

// y [max_rows][hidden] of a 16-bit type, and the shape of the rows it returns to
const at::Tensor& sorted_arg(PyObject* o, const char* what, PyObject* pos_o, at::IntArrayRef& lead, int& code)
{
    const at::Tensor& y = lead_tensor(o, what);
    code = half_code(y, what);
    if (y.dim() != 2) refuse("%s has %lld dimensions, the call takes [max_rows][hidden]", what, (long long)y.dim());
    const at::Tensor& pos = tensor(pos_o, "order.pos");
    if (pos.dim() < 1) refuse("order.pos has no dimensions");
    lead = pos.sizes().slice(0, pos.dim() - 1);
    return y;
}

// (pos, src, counts, y, weights)
PyObject* return_rows(PyObject* const* v)
{
    at::IntArrayRef lead;
    int code;
    const at::Tensor& y = sorted_arg(v[3], "y", v[0], lead, code);
    const at::Device dev = y.device();
    const Order o = order_args(v[0], v[1], v[2], lead, dev);
    const int64_t hidden = y.size(1);
    const void* yp = data(y, "y", y.scalar_type(), {o.max_rows, hidden}, dev);
    const void* wp = data_or_null(v[4], "weights", at::kFloat, THPVariable_Unpack(v[0]).sizes(), dev);
    std::vector<int64_t> shape(lead.begin(), lead.end());
    shape.push_back(hidden);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out = empty(shape, y.scalar_type(), dev);
    check(g_return(yp, (const float*)wp, o.pos, o.counts, clamp_int(o.W), o.rows, clamp_int(o.k), o.max_rows,
                   clamp_int(hidden), code, out.data_ptr(), status(dev), stream(dev)));
    return wrap(out);
}

// (pos, src, counts, y, weights, dout)
PyObject* return_rows_backward(PyObject* const* v)
{
    at::IntArrayRef lead;
    int code;
    const at::Tensor& y = sorted_arg(v[3], "y", v[0], lead, code);
    const at::Device dev = y.device();
    const Order o = order_args(v[0], v[1], v[2], lead, dev);
    const int64_t hidden = y.size(1);
    const void* yp = data(y, "y", y.scalar_type(), {o.max_rows, hidden}, dev);
    const at::IntArrayRef pairs = THPVariable_Unpack(v[0]).sizes();
    const void* wp = data(tensor(v[4], "weights"), "weights", at::kFloat, pairs, dev);
    std::vector<int64_t> shape(lead.begin(), lead.end());
    shape.push_back(hidden);
    const void* dp = data(tensor(v[5], "dout"), "dout", y.scalar_type(), shape, dev);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor dy = empty(y.sizes(), y.scalar_type(), dev), dw = empty(pairs, at::kFloat, dev);
    check(g_back(yp, (const float*)wp, dp, o.pos, o.counts, clamp_int(o.W), o.rows, clamp_int(o.k), o.max_rows,
                 clamp_int(hidden), code, dy.data_ptr(), (float*)dw.data_ptr(), status(dev), stream(dev)));
    return pack({dy, dw});
}

// (a, a_scales, b, b_scales, offsets, out type: EP_BF16, EP_FP16, or EP_FP8_E4M3 for SwiGLU)
PyObject* matmul(PyObject* const* v)
{
    const at::Tensor& a = lead_tensor(v[0], "a");
    const at::Device dev = a.device();
    if (a.dim() != 2) refuse("a has %lld dimensions, the call takes [rows][inner]", (long long)a.dim());
    const at::Tensor& b = tensor(v[2], "b");
    const bool grouped = v[4] != Py_None;
    const int64_t rows = a.size(0), inner = a.size(1);
    if (b.dim() != (grouped ? 3 : 2) || b.size(-1) != inner)
        refuse("b has shape %s, the call takes %s[columns][%lld]", shape_text(b.sizes()).c_str(), grouped ? "[groups]" : "",
               (long long)inner);
    const int64_t groups = grouped ? b.size(0) : 1, columns = b.size(-2), kb = (inner + 127) / 128, nb = (columns + 127) / 128;
    const int64_t scale_shape[3] = {groups, nb, kb};
    const at::IntArrayRef bs_shape = grouped ? at::IntArrayRef(scale_shape, 3) : at::IntArrayRef(scale_shape + 1, 2);
    const void* ap = data(a, "a", at::kFloat8_e4m3fn, a.sizes(), dev);
    const void* asp = data(tensor(v[1], "a_scales"), "a_scales", at::kFloat, {rows, kb}, dev);
    const void* bp = data(b, "b", at::kFloat8_e4m3fn, b.sizes(), dev);
    const void* bsp = data(tensor(v[3], "b_scales"), "b_scales", at::kFloat, bs_shape, dev);
    const void* op = data_or_null(v[4], "offsets", at::kInt, {groups + 1}, dev);
    const int type = small(v[5], "the output's type");
    const bool swiglu = type == EP_FP8_E4M3;
    const int64_t half = columns / 2;
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor out = swiglu ? empty({rows, half}, at::kFloat8_e4m3fn, dev)
                            : empty({rows, columns}, type == EP_FP16 ? at::kHalf : at::kBFloat16, dev);
    at::Tensor scales;
    if (swiglu) scales = empty({rows, (half + 127) / 128}, at::kFloat, dev);
    check(g_matmul(ap, (const float*)asp, bp, (const float*)bsp, (const int32_t*)op, rows, clamp_int(groups),
                   clamp_int(columns), clamp_int(inner), swiglu, type, out.data_ptr(), (float*)get(scales), status(dev),
                   stream(dev)));
    return swiglu ? pack({out, scales}) : wrap(out);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N || !g_error) {
        PyErr_Format(PyExc_TypeError, "%d arguments wanted, after bind()", N);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// bind(EpError, make_status, addresses of the C ABI functions in the order below)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    void* f[9];
    if (n != 11) {
        PyErr_SetString(PyExc_TypeError, "bind takes EpError, make_status and nine addresses");
        return nullptr;
    }
    for (int i = 0; i < 9; ++i) {
        f[i] = PyLong_AsVoidPtr(args[2 + i]);
        if (PyErr_Occurred()) return nullptr;
        if (!f[i]) {
            PyErr_SetString(PyExc_ValueError, "bind: a function's address is 0");
            return nullptr;
        }
    }
    Py_XDECREF(g_error);
    Py_XDECREF(g_make_status);
    g_error = Py_NewRef(args[0]);
    g_make_status = Py_NewRef(args[1]);
    g_norm = (decltype(g_norm))f[0];
    g_sort_bytes = (decltype(g_sort_bytes))f[1];
    g_sort = (decltype(g_sort))f[2];
    g_rows = (decltype(g_rows))f[3];
    g_return = (decltype(g_return))f[4];
    g_back = (decltype(g_back))f[5];
    g_matmul = (decltype(g_matmul))f[6];
    g_strerror = (decltype(g_strerror))f[7];
    g_last_error = (decltype(g_last_error))f[8];
    Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", (PyCFunction)(void (*)())bind, METH_FASTCALL, nullptr},
    {"rms_norm_fp8", (PyCFunction)(void (*)())entry<rms_norm, 5>, METH_FASTCALL, nullptr},
    {"sort_by_expert", (PyCFunction)(void (*)())entry<sort_by_expert, 4>, METH_FASTCALL, nullptr},
    {"sorted_rows", (PyCFunction)(void (*)())entry<sorted_rows, 5>, METH_FASTCALL, nullptr},
    {"return_rows", (PyCFunction)(void (*)())entry<return_rows, 5>, METH_FASTCALL, nullptr},
    {"return_rows_backward", (PyCFunction)(void (*)())entry<return_rows_backward, 6>, METH_FASTCALL, nullptr},
    {"matmul_fp8", (PyCFunction)(void (*)())entry<matmul, 6>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ep_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ep_binding(void) { return PyModule_Create(&g_module); }
