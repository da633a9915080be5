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
#include <cstring>
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
decltype(&ep_rms_norm_join) g_join;
decltype(&ep_rms_norm_join_workspace_bytes) g_join_bytes;
decltype(&ep_rms_norm_join_backward) g_join_back;
decltype(&ep_swiglu_saved) g_swiglu;
decltype(&ep_swiglu_saved_backward) g_swiglu_back;
decltype(&ep_moe_few_workspace_bytes) g_few_bytes;
decltype(&ep_moe_few_rows) g_few;
decltype(&ep_matmul_fp8_weight_gradient) g_gradient;
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

// Address of a 2-D tensor of rows, of this type and shape on this device, whose rows may be a stride apart.
void* row_data(const at::Tensor& t, const char* what, at::ScalarType type, at::IntArrayRef shape, at::Device device,
               int64_t& stride)
{
    if (t.device() != device)
        refuse("%s is on %s, the call runs on %s", what, t.device().str().c_str(), device.str().c_str());
    if (t.scalar_type() != type) refuse("%s is %s, the call takes %s", what, type_text(t.scalar_type()), type_text(type));
    if (t.sizes() != shape)
        refuse("%s has shape %s, the call takes %s", what, shape_text(t.sizes()).c_str(), shape_text(shape).c_str());
    if (t.size(1) > 1 && t.stride(1) != 1) refuse("%s: the elements of a row are not consecutive", what);
    stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
    return t.data_ptr();
}

// A vector along the channels, of `type` or FP32; NULL for None.
const void* channels(PyObject* o, const char* what, at::ScalarType type, int64_t hidden, at::Device dev, int& fp32)
{
    if (o == Py_None) return nullptr;
    const at::Tensor& w = tensor(o, what);
    fp32 = w.scalar_type() == at::kFloat;
    return data(w, what, fp32 ? at::kFloat : type, {hidden}, dev);
}

double number(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

// The arguments that the join and its gradient share.
ep_join join_args(PyObject* y_o, PyObject* post_o, PyObject* gate_o, PyObject* pre_o, PyObject* scale_o)
{
    const at::Tensor& y = lead_tensor(y_o, "y");
    ep_join j{};
    j.dtype = half_code(y, "y");
    if (y.dim() != 2) refuse("y has %lld dimensions, the call takes [rows][hidden]", (long long)y.dim());
    const at::Device dev = y.device();
    const int64_t hidden = y.size(1);
    j.rows = y.size(0);
    j.hidden = clamp_int(hidden);
    j.y = row_data(y, "y", y.scalar_type(), y.sizes(), dev, j.y_stride);
    j.post_weight = channels(post_o, "post_weight", y.scalar_type(), hidden, dev, j.post_fp32);
    j.pre_weight = channels(pre_o, "pre_weight", y.scalar_type(), hidden, dev, j.pre_fp32);
    j.residual_scale = (float)number(scale_o);
    if (gate_o != Py_None) {
        const at::Tensor& g = tensor(gate_o, "gate");
        if (g.dim() == 1) {
            j.gate_kind = EP_GATE_CHANNEL;
            j.gate = channels(gate_o, "gate", y.scalar_type(), hidden, dev, j.gate_fp32);
        } else if (g.dim() == 2 && g.size(1) == 1) {
            j.gate_kind = EP_GATE_ROW;
            j.gate = data(g, "gate", at::kFloat, {j.rows, 1}, dev);
        } else {
            j.gate_kind = EP_GATE_ELEMENT;
            if (g.dim() != 2)
                refuse("gate has shape %s, the call takes [hidden], [rows][1] or [rows][hidden]", shape_text(g.sizes()).c_str());
            j.gate = row_data(g, "gate", y.scalar_type(), y.sizes(), dev, j.gate_stride);
        }
    }
    return j;
}

bool truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

// (y, residual, post_weight, gate, pre_weight, residual_scale, eps, fp8, want_n)
PyObject* join(PyObject* const* v)
{
    ep_join j = join_args(v[0], v[2], v[3], v[4], v[5]);
    const at::Tensor& y = THPVariable_Unpack(v[0]);
    const at::Device dev = y.device();
    j.eps = (float)number(v[6]);
    const bool fp8 = truth(v[7]), want_n = truth(v[8]);
    if (!j.pre_weight && (fp8 || want_n)) refuse("n or its codes are wanted without pre_weight");
    int64_t rs = 0;
    const void* r = row_data(tensor(v[1], "residual"), "residual", y.scalar_type(), y.sizes(), dev, rs);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor h = empty(y.sizes(), y.scalar_type(), dev), n, q, s, post, pre;
    if (want_n) n = empty(y.sizes(), y.scalar_type(), dev);
    if (fp8) {
        q = empty(y.sizes(), at::kFloat8_e4m3fn, dev);
        s = empty({j.rows, (y.size(1) + 127) / 128}, at::kFloat, dev);
    }
    if (j.post_weight) post = empty({j.rows}, at::kFloat, dev);
    if (j.pre_weight) pre = empty({j.rows}, at::kFloat, dev);
    check(g_join(&j, r, rs, h.data_ptr(), get(n), get(q), (float*)get(s), (float*)get(post), (float*)get(pre), stream(dev)));
    return pack({h, n, q, s, post, pre});
}

// (y, h, post_rstd, pre_rstd, dh, dn, post_weight, gate, pre_weight, residual_scale)
PyObject* join_backward(PyObject* const* v)
{
    const ep_join j = join_args(v[0], v[6], v[7], v[8], v[9]);
    const at::Tensor& y = THPVariable_Unpack(v[0]);
    const at::Device dev = y.device();
    const at::ScalarType type = y.scalar_type();
    int64_t dh_stride = 0, dn_stride = 0;
    const void* dh = v[4] == Py_None ? nullptr : row_data(tensor(v[4], "dh"), "dh", type, y.sizes(), dev, dh_stride);
    const void* dn = v[5] == Py_None ? nullptr : row_data(tensor(v[5], "dn"), "dn", type, y.sizes(), dev, dn_stride);
    if ((v[5] != Py_None) != (v[8] != Py_None)) refuse("dn and pre_weight are not both given, nor both None");
    if (v[4] == Py_None && v[5] == Py_None) refuse("neither dh nor dn is given");
    const void *h = nullptr, *post = nullptr, *pre = nullptr;
    if (j.pre_weight) {
        h = data(tensor(v[1], "joined.h"), "joined.h", type, y.sizes(), dev);
        pre = data(tensor(v[3], "joined.pre_rstd"), "joined.pre_rstd", at::kFloat, {j.rows}, dev);
    }
    if (j.post_weight) post = data(tensor(v[2], "joined.post_rstd"), "joined.post_rstd", at::kFloat, {j.rows}, dev);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor dy = empty(y.sizes(), type, dev), dres = empty(y.sizes(), type, dev), dpost, dgate, dpre, work;
    if (j.post_weight) dpost = empty({y.size(1)}, at::kFloat, dev);
    if (j.pre_weight) dpre = empty({y.size(1)}, at::kFloat, dev);
    if (j.gate_kind != EP_GATE_NONE)
        dgate = empty(THPVariable_Unpack(v[7]).sizes(), j.gate_kind == EP_GATE_ELEMENT ? type : at::kFloat, dev);
    const size_t need = g_join_bytes(j.rows, j.hidden);
    if (need) work = empty({(int64_t)need}, at::kByte, dev);
    check(g_join_back(&j, h, (const float*)post, (const float*)pre, dh, dh_stride, dn, dn_stride, dy.data_ptr(),
                      dres.data_ptr(), (float*)get(dpost), get(dgate), (float*)get(dpre), get(work), need, stream(dev)));
    return pack({dy, dres, dpost, dgate, dpre});
}

// The last of a sort's offsets, past which a buffer's rows hold nothing; NULL for None.
const int32_t* rows_end(PyObject* offsets, at::Device dev)
{
    if (offsets == Py_None) return nullptr;
    const at::Tensor& t = tensor(offsets, "offsets");
    if (t.dim() != 1 || t.size(0) < 1) refuse("offsets has shape %s, the call takes [groups + 1]", shape_text(t.sizes()).c_str());
    return (const int32_t*)data(t, "offsets", at::kInt, t.sizes(), dev) + t.size(0) - 1;
}

// (gate_up, offsets)
PyObject* swiglu_saved(PyObject* const* v)
{
    const at::Tensor& x = lead_tensor(v[0], "gate_up");
    const int code = half_code(x, "gate_up");
    if (x.dim() != 2 || x.size(1) % 2 != 0)
        refuse("gate_up has shape %s, the call takes [rows][2 * inner]", shape_text(x.sizes()).c_str());
    const at::Device dev = x.device();
    const int64_t rows = x.size(0), inner = x.size(1) / 2;
    int64_t stride = 0;
    const void* xp = row_data(x, "gate_up", x.scalar_type(), x.sizes(), dev, stride);
    const int32_t* end = rows_end(v[1], dev);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor q = empty({rows, inner}, at::kFloat8_e4m3fn, dev), s = empty({rows, (inner + 127) / 128}, at::kFloat, dev),
               saved = empty({rows, 2 * inner}, at::kFloat8_e4m3fn, dev),
               saved_s = empty({rows, (2 * inner + 127) / 128}, at::kFloat, dev);
    check(g_swiglu(xp, stride, code, rows, clamp_int(inner), end, q.data_ptr(), (float*)s.data_ptr(), saved.data_ptr(),
                   (float*)saved_s.data_ptr(), stream(dev)));
    return pack({q, s, saved, saved_s});
}

// (saved, saved_scales, dz, offsets, fp8)
PyObject* swiglu_saved_backward(PyObject* const* v)
{
    const at::Tensor& dz = lead_tensor(v[2], "dz");
    const int code = half_code(dz, "dz");
    if (dz.dim() != 2) refuse("dz has %lld dimensions, the call takes [rows][inner]", (long long)dz.dim());
    const at::Device dev = dz.device();
    const int64_t rows = dz.size(0), inner = dz.size(1), blocks = (2 * inner + 127) / 128;
    const void* saved = data(tensor(v[0], "saved"), "saved", at::kFloat8_e4m3fn, {rows, 2 * inner}, dev);
    const void* saved_s = data(tensor(v[1], "saved_scales"), "saved_scales", at::kFloat, {rows, blocks}, dev);
    int64_t stride = 0;
    const void* dp = row_data(dz, "dz", dz.scalar_type(), dz.sizes(), dev, stride);
    const int32_t* end = rows_end(v[3], dev);
    const bool fp8 = truth(v[4]);
    const c10::cuda::CUDAGuard guard(dev);
    at::Tensor d = empty({rows, 2 * inner}, dz.scalar_type(), dev), q, s;
    if (fp8) {
        q = empty({rows, 2 * inner}, at::kFloat8_e4m3fn, dev);
        s = empty({rows, blocks}, at::kFloat, dev);
    }
    check(g_swiglu_back(saved, (const float*)saved_s, dp, stride, code, rows, clamp_int(inner), end, d.data_ptr(), get(q),
                        (float*)get(s), stream(dev)));
    return pack({d, q, s});
}

// (dy, a, a_scales, offsets, type of the output or -1 for dy's, whether it is FP32)
PyObject* weight_gradient(PyObject* const* v)
{
    const at::Tensor& dy = lead_tensor(v[0], "dy");
    const int code = half_code(dy, "dy");
    if (dy.dim() != 2) refuse("dy has %lld dimensions, the call takes [rows][columns]", (long long)dy.dim());
    const at::Device dev = dy.device();
    const int64_t rows = dy.size(0), columns = dy.size(1);
    const at::Tensor& a = tensor(v[1], "a");
    if (a.dim() != 2) refuse("a has %lld dimensions, the call takes [rows][inner]", (long long)a.dim());
    const int64_t inner = a.size(1);
    const int type = small(v[4], "the output's type");
    const bool fp32 = truth(v[5]);
    if (!fp32 && type >= 0 && type != code) refuse("out_dtype is neither dy's type nor 'fp32'");
    const void* yp = data(dy, "dy", dy.scalar_type(), dy.sizes(), dev);
    const void* ap = data(a, "a", at::kFloat8_e4m3fn, {rows, inner}, dev);
    const void* sp = data(tensor(v[2], "a_scales"), "a_scales", at::kFloat, {rows, (inner + 127) / 128}, dev);
    const bool grouped = v[3] != Py_None;
    int64_t groups = 1;
    const void* op = nullptr;
    if (grouped) {
        const at::Tensor& o = tensor(v[3], "offsets");
        if (o.dim() != 1 || o.size(0) < 2) refuse("offsets has shape %s, the call takes [groups + 1]", shape_text(o.sizes()).c_str());
        groups = o.size(0) - 1;
        op = data(o, "offsets", at::kInt, o.sizes(), dev);
    }
    const int64_t shape[3] = {groups, columns, inner};
    const c10::cuda::CUDAGuard guard(dev);
    // a shape that the C ABI refuses gets no storage
    const bool small_enough = columns <= 1 << 20 && inner <= 1 << 20 && groups <= 4096;
    at::Tensor out = empty(!small_enough ? at::IntArrayRef{0} : grouped ? at::IntArrayRef(shape, 3) : at::IntArrayRef(shape + 1, 2),
                           fp32 ? at::kFloat : dy.scalar_type(), dev);
    check(g_gradient(yp, code, ap, (const float*)sp, (const int32_t*)op, rows, clamp_int(groups), clamp_int(columns),
                     clamp_int(inner), fp32, out.data_ptr(), status(dev), stream(dev)));
    return wrap(out);
}

// (x, x_scales, indices, weights, up, up_scales, down, down_scales, first_expert, out type)
PyObject* moe_few_rows(PyObject* const* v)
{
    const at::Tensor& x = lead_tensor(v[0], "x");
    if (x.dim() != 2) refuse("x has %lld dimensions, the call takes [rows][hidden]", (long long)x.dim());
    const bool fp8 = x.scalar_type() == at::kFloat8_e4m3fn;
    const int code = fp8 ? (int)EP_FP8_E4M3 : half_code(x, "x (float8_e4m3fn or)");
    const at::Device dev = x.device();
    const int64_t rows = x.size(0), hidden = x.size(1), hb = (hidden + 127) / 128;
    const void* xp = data(x, "x", x.scalar_type(), x.sizes(), dev);
    if (fp8 != (v[1] != Py_None)) refuse("x_scales goes with float8_e4m3fn rows, and with them alone");
    const void* xs = data_or_null(v[1], "x_scales", at::kFloat, {rows, hb}, dev);
    const at::Tensor& idx = tensor(v[2], "indices");
    if (idx.dim() != 2) refuse("indices has %lld dimensions, the call takes [rows][k]", (long long)idx.dim());
    const int64_t k = idx.size(1);
    const void* ip = data(idx, "indices", at::kInt, {rows, k}, dev);
    const void* wp = data(tensor(v[3], "weights"), "weights", at::kFloat, {rows, k}, dev);
    const at::Tensor& down = tensor(v[6], "down");
    if (down.dim() != 3 || down.size(1) != hidden)
        refuse("down has shape %s, the call takes [experts][%lld][inner]", shape_text(down.sizes()).c_str(), (long long)hidden);
    const int64_t experts = down.size(0), inner = down.size(2), ib = (inner + 127) / 128, ub = (2 * inner + 127) / 128;
    const void* dp = data(down, "down", at::kFloat8_e4m3fn, down.sizes(), dev);
    const void* ds = data(tensor(v[7], "down_scales"), "down_scales", at::kFloat, {experts, hb, ib}, dev);
    const void* up = data(tensor(v[4], "up"), "up", at::kFloat8_e4m3fn, {experts, 2 * inner, hidden}, dev);
    const void* us = data(tensor(v[5], "up_scales"), "up_scales", at::kFloat, {experts, ub, hb}, dev);
    const int first = small(v[8], "first_expert"), type = small(v[9], "the output's type");
    const c10::cuda::CUDAGuard guard(dev);
    const size_t need = g_few_bytes(rows, clamp_int(k), clamp_int(inner));
    at::Tensor out = empty(x.sizes(), type == EP_FP16 ? at::kHalf : at::kBFloat16, dev), work;
    if (need) work = empty({(int64_t)need}, at::kByte, dev);
    check(g_few(xp, (const float*)xs, code, (const int32_t*)ip, (const float*)wp, rows, clamp_int(k), first, clamp_int(experts),
                clamp_int(hidden), clamp_int(inner), up, (const float*)us, dp, (const float*)ds, type, out.data_ptr(),
                get(work), need, stream(dev)));
    return wrap(out);
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

// The C ABI functions that bind() takes, in its order.
struct Bound {
    const char* name;
    void* target;
};
#define EP_BOUND(variable) {#variable, &variable}
const Bound g_bound[] = {EP_BOUND(g_norm), EP_BOUND(g_sort_bytes), EP_BOUND(g_sort), EP_BOUND(g_rows), EP_BOUND(g_return),
                         EP_BOUND(g_back), EP_BOUND(g_matmul), EP_BOUND(g_join), EP_BOUND(g_join_bytes), EP_BOUND(g_join_back),
                         EP_BOUND(g_swiglu), EP_BOUND(g_swiglu_back), EP_BOUND(g_few_bytes),
                         EP_BOUND(g_few), EP_BOUND(g_gradient), EP_BOUND(g_strerror), EP_BOUND(g_last_error)};
constexpr int kBound = sizeof g_bound / sizeof g_bound[0];

// bind(EpError, make_status, addresses of the C ABI functions in the order above)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    void* f[kBound];
    if (n != 2 + kBound) {
        PyErr_Format(PyExc_TypeError, "bind takes EpError, make_status and %d addresses", kBound);
        return nullptr;
    }
    for (int i = 0; i < kBound; ++i) {
        f[i] = PyLong_AsVoidPtr(args[2 + i]);
        if (PyErr_Occurred()) return nullptr;
        if (!f[i]) {
            PyErr_Format(PyExc_ValueError, "bind: the address of %s is 0", g_bound[i].name);
            return nullptr;
        }
    }
    Py_XDECREF(g_error);
    Py_XDECREF(g_make_status);
    g_error = Py_NewRef(args[0]);
    g_make_status = Py_NewRef(args[1]);
    for (int i = 0; i < kBound; ++i) memcpy(g_bound[i].target, &f[i], sizeof f[i]);
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
    {"rms_norm_join", (PyCFunction)(void (*)())entry<join, 9>, METH_FASTCALL, nullptr},
    {"rms_norm_join_backward", (PyCFunction)(void (*)())entry<join_backward, 10>, METH_FASTCALL, nullptr},
    {"swiglu_saved", (PyCFunction)(void (*)())entry<swiglu_saved, 2>, METH_FASTCALL, nullptr},
    {"swiglu_saved_backward", (PyCFunction)(void (*)())entry<swiglu_saved_backward, 5>, METH_FASTCALL, nullptr},
    {"matmul_fp8_weight_gradient", (PyCFunction)(void (*)())entry<weight_gradient, 6>, METH_FASTCALL, nullptr},
    {"moe_few_rows", (PyCFunction)(void (*)())entry<moe_few_rows, 10>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ep_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ep_binding(void) { return PyModule_Create(&g_module); }
