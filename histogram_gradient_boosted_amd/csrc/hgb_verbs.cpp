// The vector verbs on torch tensors: argument checks, outputs and workspaces
// for binding.Context, over the C ABI (include/hgb.h).
//
// A small call's time is the host's: a kernel of two or three microseconds
// waits for its launch (2.5 us), its outputs (0.6 us each) and the checks.
// Through ctypes and Python the same embed took 7.6 us, layer_norm 12.0.
//
// Every function takes the context's handle, its device, its stream's id and
// the verb's arguments by place, and returns the verb's result; or the
// hgb_status of a refused call; or kElsewhere, before it has done anything,
// when the current stream is not the context's (binding.py orders the two).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/GradMode.h>
#include <c10/core/impl/VirtualGuardImpl.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <exception>

#include "hgb.h"

namespace {

constexpr long kElsewhere = -1;
constexpr long kTooLarge = -2;   // sizes for which a workspace function returns -1

using at::Tensor;

// A bad argument: a ValueError in Python.
struct Refused : std::exception {
    char text[256];
    __attribute__((format(printf, 2, 3))) explicit Refused(const char* form, ...)
    {
        va_list ap;
        va_start(ap, form);
        vsnprintf(text, sizeof text, form, ap);
        va_end(ap);
    }
    const char* what() const noexcept override { return text; }
};

struct Call {
    hgb_ctx* ctx;
    int device;
    int64_t stream;
    PyObject* const* args;

    bool elsewhere() const
    {
        const c10::impl::VirtualGuardImpl guard(c10::DeviceType::CUDA);
        return guard.getStream(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device)).id() != stream;
    }
    Tensor make(at::IntArrayRef sizes, at::ScalarType type) const
    {
        return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device)));
    }
    Tensor workspace(int64_t bytes) const { return bytes > 0 ? make({bytes}, at::kByte) : Tensor(); }
};

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

bool given(PyObject* o) { return o != Py_None; }

int64_t whole(PyObject* o, const char* name)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("%s must be an integer", name);
    }
    return v;
}

int32_t whole32(PyObject* o, const char* name)
{
    const int64_t v = whole(o, name);
    if (v != (int32_t)v) throw Refused("%s must fit 32 bits", name);
    return (int32_t)v;
}

float real(PyObject* o, const char* name)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Refused("%s must be a number", name);
    }
    return (float)v;
}

// A yes or no; a tensor's would be a wait for the device.
bool truth(PyObject* o, const char* name)
{
    const int v = THPVariable_Check(o) ? -1 : PyObject_IsTrue(o);
    if (v < 0) {
        PyErr_Clear();
        throw Refused("%s must be a truth value", name);
    }
    return v != 0;
}

const Tensor& tensor(const Call& c, PyObject* o, const char* name)
{
    if (THPVariable_Check(o)) {
        const Tensor& t = THPVariable_Unpack(o);
        // the verbs record nothing for autograd: the result would have no gradient, without a word
        if (t.requires_grad() && c10::GradMode::is_enabled())
            throw Refused("%s requires a gradient, which the verbs do not record: call them under torch.no_grad(), and "
                          "their _backward for gradients", name);
        // what lies in memory is not what such a view holds
        if (t.is_neg()) throw Refused("%s is a negated view: give its resolve_neg()", name);
        if (t.is_cuda() && t.get_device() == c.device) return t;
    }
    throw Refused("%s must be a CUDA tensor on device %d", name, c.device);
}

// The hgb_dtype of a vector's type.
int code(at::ScalarType t, const char* name)
{
    if (t == at::kFloat) return HGB_F32;
    if (t == at::kBFloat16) return HGB_BF16;
    if (t == at::kHalf) return HGB_F16;
    throw Refused("%s must be float32, bfloat16 or float16, got %s", name, at::toString(t));
}

void same(at::ScalarType got, at::ScalarType want, const char* name)
{
    if (got != want) throw Refused("%s must be %s, got %s", name, at::toString(want), at::toString(got));
}

// A [..., dim] vector argument.
struct Rows {
    Tensor t;
    void* p;
    int type;
    int64_t n, dim, stride;
};

Rows rows_of(const Tensor& t, const char* name)
{
    Rows r{t, nullptr, code(t.scalar_type(), name), 0, 0, 0};
    if (t.dim() == 0) throw Refused("%s must have a last dimension", name);
    r.dim = r.stride = t.size(-1);
    if (r.dim < 1) throw Refused("%s has rows of no values", name);
    if (t.dim() == 2) {
        r.n = t.size(0);
        if (r.n > 1) r.stride = t.stride(0);
        if (r.stride < r.dim || (t.stride(1) != 1 && r.dim > 1))
            throw Refused("%s's rows must be contiguous and apart", name);
    } else {
        r.n = t.numel() / r.dim;
        if (!t.is_contiguous()) throw Refused("%s must be contiguous, or two-dimensional with contiguous rows", name);
    }
    r.p = t.data_ptr();
    return r;
}

Rows rows(const Call& c, PyObject* o, const char* name) { return rows_of(tensor(c, o, name), name); }

void shaped(const Rows& r, int64_t n, int64_t dim, const char* name)
{
    if (r.dim != dim) throw Refused("%s has rows of %lld values, needs %lld", name, (long long)r.dim, (long long)dim);
    if (r.n != n) throw Refused("%s holds %lld rows, needs %lld", name, (long long)r.n, (long long)n);
}

// The output: the caller's, checked, or one that allocate() makes once the
// stream is known to be the context's.
struct Out {
    Rows r;
    at::ScalarType type;
    bool made = false;
    Out(const Call& c, PyObject* o, at::ScalarType t, bool typed, int64_t n, int64_t dim) : type(t)
    {
        if (given(o)) {
            r = rows(c, o, "out");
            if (typed) same(r.t.scalar_type(), t, "out");
            shaped(r, n, dim, "out");
        } else {
            made = true;
            r = Rows{Tensor(), nullptr, code(t, "dtype"), n, dim, dim};
        }
    }
    void allocate(const Call& c, at::IntArrayRef sizes)
    {
        if (!made) return;
        r.t = c.make(sizes, type);
        r.p = r.t.data_ptr();
    }
};

at::ScalarType dtype(PyObject* o, at::ScalarType other)
{
    if (!given(o)) return other;
    if (!THPDtype_Check(o)) throw Refused("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// A contiguous tensor of one type.
const Tensor& plain(const Call& c, PyObject* o, const char* name, at::ScalarType type)
{
    const Tensor& t = tensor(c, o, name);
    same(t.scalar_type(), type, name);
    if (!t.is_contiguous()) throw Refused("%s must be contiguous", name);
    return t;
}

// A [dim] parameter, of the rows' type or float32; undefined for None.
Tensor param(const Call& c, PyObject* o, const char* name, const Rows& x)
{
    if (!given(o)) return Tensor();
    const Tensor& t = tensor(c, o, name);
    if (t.scalar_type() != at::kFloat) same(t.scalar_type(), x.t.scalar_type(), name);
    if (t.dim() != 1 || t.size(0) != x.dim) throw Refused("%s must have shape [%lld]", name, (long long)x.dim);
    if (!t.is_contiguous()) throw Refused("%s must be contiguous", name);
    return t;
}

// A routing's position and offsets.
struct Routed {
    const Tensor& position;
    const Tensor& offsets;
    int64_t n;
    int32_t top, experts;
    Routed(const Call& c, PyObject* p, PyObject* o)
        : position(plain(c, p, "route.position", at::kInt)), offsets(plain(c, o, "route.offsets", at::kInt))
    {
        if (position.dim() != 2 || offsets.dim() != 1 || offsets.size(0) < 2)
            throw Refused("route is not what Context.route returns");
        n = position.size(0);
        top = (int32_t)position.size(1);
        experts = (int32_t)offsets.size(0) - 1;
    }
    const int32_t* places() const { return (const int32_t*)position.data_ptr(); }
    const int32_t* ends() const { return (const int32_t*)offsets.data_ptr(); }
    void takes(const Rows& r, const char* name) const
    {
        if (r.n != n) throw Refused("%s: %lld rows for a route of %lld", name, (long long)r.n, (long long)n);
    }
    Tensor weights(const Call& c, PyObject* o) const
    {
        if (!given(o)) return Tensor();
        const Tensor& t = plain(c, o, "weights", at::kFloat);
        if (t.dim() != 2 || t.size(0) != n || t.size(1) != top)
            throw Refused("weights must have shape [%lld, %d]", (long long)n, top);
        return t;
    }
};

PyObject* status(long s) { return PyLong_FromLong(s); }
PyObject* wrap(const Tensor& t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

PyObject* tuple(std::initializer_list<Tensor> ts)
{
    PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    for (const Tensor& t : ts) {
        PyObject* o = wrap(t);
        if (!o) {
            Py_DECREF(r);
            return nullptr;
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// embed(table, tokens, scale, pad, dtype, out)
PyObject* embed(const Call& c)
{
    const Rows table = rows(c, c.args[0], "table");
    if (table.t.dim() != 2) throw Refused("table must be two-dimensional");
    const Tensor& tokens = plain(c, c.args[1], "tokens", at::kInt);
    const float scale = real(c.args[2], "scale");
    const int32_t pad = whole32(c.args[3], "pad");
    Out out(c, c.args[5], dtype(c.args[4], table.t.scalar_type()), given(c.args[4]), tokens.numel(), table.dim);
    if (c.elsewhere()) return status(kElsewhere);
    at::DimVector sizes(tokens.sizes());
    sizes.push_back(table.dim);
    out.allocate(c, sizes);
    const hgb_status s = hgb_embed(c.ctx, table.p, table.type, table.stride, table.n, table.dim, (const int32_t*)tokens.data_ptr(),
                                   tokens.numel(), pad, scale, out.r.p, out.r.type, out.r.stride);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// embed_backward(grad, tokens, vocab, scale, pad, dtype, out)
PyObject* embed_backward(const Call& c)
{
    const Rows grad = rows(c, c.args[0], "grad");
    const Tensor& tokens = plain(c, c.args[1], "tokens", at::kInt);
    if (tokens.numel() != grad.n)
        throw Refused("grad holds %lld rows for %lld tokens", (long long)grad.n, (long long)tokens.numel());
    const int64_t vocab = whole(c.args[2], "vocab");
    const float scale = real(c.args[3], "scale");
    const int32_t pad = whole32(c.args[4], "pad");
    const int64_t bytes = hgb_embed_backward_workspace(grad.n, vocab, grad.dim);
    if (bytes < 0) return status(kTooLarge);
    Out out(c, c.args[6], dtype(c.args[5], grad.t.scalar_type()), given(c.args[5]), vocab, grad.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, {vocab, grad.dim});
    const Tensor ws = c.workspace(bytes);
    const hgb_status s =
        hgb_embed_backward(c.ctx, grad.p, grad.type, grad.stride, grad.n, grad.dim, (const int32_t*)tokens.data_ptr(), pad, scale,
                           vocab, out.r.p, out.r.type, out.r.stride, ptr(ws), bytes);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// layer_norm(x, weight, bias, eps, out)
PyObject* layer_norm(const Call& c)
{
    const Rows x = rows(c, c.args[0], "x");
    const Tensor weight = param(c, c.args[1], "weight", x), bias = param(c, c.args[2], "bias", x);
    if (weight.defined() && bias.defined() && weight.scalar_type() != bias.scalar_type())
        throw Refused("the parameters must have one type");
    const float eps = real(c.args[3], "eps");
    Out out(c, c.args[4], x.t.scalar_type(), true, x.n, x.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, x.t.sizes());
    const at::IntArrayRef lead = x.t.sizes().slice(0, x.t.dim() - 1);
    const Tensor mean = c.make(lead, at::kFloat), rstd = c.make(lead, at::kFloat);
    const Tensor& any = weight.defined() ? weight : bias;
    const hgb_status s =
        hgb_layer_norm(c.ctx, x.p, x.type, x.stride, x.n, x.dim, ptr(weight), ptr(bias),
                       any.defined() ? code(any.scalar_type(), "weight") : HGB_F32, eps, out.r.p, out.r.stride,
                       (float*)mean.data_ptr(), (float*)rstd.data_ptr());
    return s == HGB_OK ? tuple({out.r.t, mean, rstd}) : status(s);
}

// layer_norm_backward(grad, x, mean, rstd, weight, bias, out)
PyObject* layer_norm_backward(const Call& c)
{
    const bool bias = truth(c.args[5], "bias");
    const Rows grad = rows(c, c.args[0], "grad"), x = rows(c, c.args[1], "x");
    same(x.t.scalar_type(), grad.t.scalar_type(), "x");
    shaped(x, grad.n, grad.dim, "x");
    const Tensor& mean = plain(c, c.args[2], "mean", at::kFloat);
    const Tensor& rstd = plain(c, c.args[3], "rstd", at::kFloat);
    if (mean.numel() < x.n || rstd.numel() < x.n)
        throw Refused("mean and rstd must hold %lld values", (long long)x.n);
    const Tensor weight = param(c, c.args[4], "weight", x);
    Out out(c, c.args[6], x.t.scalar_type(), true, x.n, x.dim);
    const int64_t bytes = weight.defined() || bias ? hgb_layer_norm_backward_workspace(x.n, x.dim) : 0;
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, x.t.sizes());
    const at::ScalarType type = weight.defined() ? weight.scalar_type() : at::kFloat;
    const Tensor dw = weight.defined() ? c.make({x.dim}, type) : Tensor(), db = bias ? c.make({x.dim}, type) : Tensor();
    const Tensor ws = c.workspace(bytes);
    const hgb_status s = hgb_layer_norm_backward(
        c.ctx, grad.p, grad.stride, x.p, x.stride, x.type, x.n, x.dim, (const float*)mean.data_ptr(), (const float*)rstd.data_ptr(),
        ptr(weight), code(type, "weight"), out.r.p, out.r.stride, ptr(dw), ptr(db), ptr(ws), bytes);
    return s == HGB_OK ? tuple({out.r.t, dw, db}) : status(s);
}

// route(experts, n_experts)
PyObject* route(const Call& c)
{
    const Tensor& experts = plain(c, c.args[0], "experts", at::kInt);
    if (experts.dim() != 2) throw Refused("experts must be a two-dimensional tensor");
    const int32_t E = whole32(c.args[1], "n_experts");
    const int64_t n = experts.size(0), top = experts.size(1);
    const int64_t bytes = top == (int32_t)top ? hgb_route_workspace(n, (int32_t)top, E) : -1;
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    const Tensor order = c.make({n * top}, at::kInt), position = c.make({n, top}, at::kInt), offsets = c.make({E + 1}, at::kInt);
    const Tensor ws = c.workspace(bytes);
    const hgb_status s = hgb_route(c.ctx, (const int32_t*)experts.data_ptr(), n, (int32_t)top, E, (int32_t*)order.data_ptr(),
                                   (int32_t*)position.data_ptr(), (int32_t*)offsets.data_ptr(), ptr(ws), bytes);
    return s == HGB_OK ? tuple({order, position, offsets}) : status(s);
}

// route_gather(x, position, offsets, out)
PyObject* route_gather(const Call& c)
{
    const Rows x = rows(c, c.args[0], "x");
    const Routed r(c, c.args[1], c.args[2]);
    r.takes(x, "x");
    Out out(c, c.args[3], x.t.scalar_type(), true, r.n * r.top, x.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, {r.n * r.top, x.dim});
    const hgb_status s = hgb_route_gather(c.ctx, x.p, x.type, x.stride, r.n, r.top, x.dim, r.places(), r.ends(), r.experts, out.r.p,
                                          out.r.stride);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// route_gather_backward(grad, position, offsets, out)
PyObject* route_gather_backward(const Call& c)
{
    const Rows grad = rows(c, c.args[0], "grad");
    const Routed r(c, c.args[1], c.args[2]);
    shaped(grad, r.n * r.top, grad.dim, "grad");
    Out out(c, c.args[3], grad.t.scalar_type(), true, r.n, grad.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, {r.n, grad.dim});
    const hgb_status s = hgb_route_gather_backward(c.ctx, grad.p, grad.type, grad.stride, r.n, r.top, grad.dim, r.places(), out.r.p,
                                                   out.r.stride);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// route_combine(y, position, offsets, weights, out)
PyObject* route_combine(const Call& c)
{
    const Rows y = rows(c, c.args[0], "y");
    const Routed r(c, c.args[1], c.args[2]);
    shaped(y, r.n * r.top, y.dim, "y");
    const Tensor w = r.weights(c, c.args[3]);
    Out out(c, c.args[4], y.t.scalar_type(), true, r.n, y.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, {r.n, y.dim});
    const hgb_status s = hgb_route_combine(c.ctx, y.p, y.type, y.stride, r.n, r.top, y.dim, r.places(), (const float*)ptr(w),
                                           out.r.p, out.r.stride);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// route_combine_backward(grad, y, position, offsets, weights, out)
PyObject* route_combine_backward(const Call& c)
{
    const Rows grad = rows(c, c.args[0], "grad"), y = rows(c, c.args[1], "y");
    const Routed r(c, c.args[2], c.args[3]);
    r.takes(grad, "grad");
    same(y.t.scalar_type(), grad.t.scalar_type(), "y");
    shaped(y, r.n * r.top, grad.dim, "y");
    const Tensor w = r.weights(c, c.args[4]);
    Out out(c, c.args[5], grad.t.scalar_type(), true, r.n * r.top, grad.dim);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, {r.n * r.top, grad.dim});
    const Tensor dw = w.defined() ? c.make({r.n, r.top}, at::kFloat) : Tensor();
    const hgb_status s = hgb_route_combine_backward(c.ctx, grad.p, grad.type, grad.stride, y.p, y.stride, r.n, r.top, grad.dim,
                                                    r.places(), r.ends(), r.experts, (const float*)ptr(w), out.r.p, out.r.stride,
                                                    (float*)ptr(dw));
    return s == HGB_OK ? tuple({out.r.t, dw}) : status(s);
}

int32_t score_of(PyObject* o)
{
    const char* name = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
    if (name && !strcmp(name, "softmax")) return HGB_SOFTMAX;
    if (name && !strcmp(name, "sigmoid")) return HGB_SIGMOID;
    PyErr_Clear();
    throw Refused("score must be \"softmax\" or \"sigmoid\"");
}

// gate(logits, top, score, bias, groups, keep, best, renormalise, scale)
PyObject* gate(const Call& c)
{
    const Rows z = rows(c, c.args[0], "logits");
    if (z.t.dim() != 2) throw Refused("logits must be two-dimensional");
    const int32_t top = whole32(c.args[1], "top"), score = score_of(c.args[2]);
    Tensor bias;
    if (given(c.args[3])) {
        bias = plain(c, c.args[3], "bias", at::kFloat);
        if (bias.dim() != 1 || bias.size(0) != z.dim) throw Refused("bias must have shape [%lld]", (long long)z.dim);
    }
    const int32_t groups = whole32(c.args[4], "groups"), keep = whole32(c.args[5], "keep"), best = whole32(c.args[6], "best");
    const bool renormalise = truth(c.args[7], "renormalise");
    const float scale = real(c.args[8], "scale");
    if (z.dim > INT32_MAX) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    const int64_t slots = top > 0 && top <= z.dim ? top : 0;   // others are refused below
    const Tensor experts = c.make({z.n, slots}, at::kInt), share = c.make({z.n, slots}, at::kFloat);
    const hgb_status s = hgb_gate(c.ctx, z.p, z.type, z.stride, z.n, (int32_t)z.dim, score, (const float*)ptr(bias), groups, keep, best,
                                  top, renormalise, scale, (int32_t*)experts.data_ptr(), (float*)share.data_ptr());
    return s == HGB_OK ? tuple({experts, share}) : status(s);
}

// gate_backward(grad, logits, experts, score, renormalise, scale, out)
PyObject* gate_backward(const Call& c)
{
    const Rows z = rows(c, c.args[1], "logits");
    if (z.t.dim() != 2) throw Refused("logits must be two-dimensional");
    const Tensor& grad = plain(c, c.args[0], "grad", at::kFloat);
    const Tensor& experts = plain(c, c.args[2], "experts", at::kInt);
    if (experts.dim() != 2 || experts.size(0) != z.n) throw Refused("experts must have shape [%lld, top]", (long long)z.n);
    if (grad.sizes() != experts.sizes()) throw Refused("grad must have the experts' shape");
    const int32_t score = score_of(c.args[3]);
    const bool renormalise = truth(c.args[4], "renormalise");
    const float scale = real(c.args[5], "scale");
    Out out(c, c.args[6], z.t.scalar_type(), true, z.n, z.dim);
    if (z.dim > INT32_MAX || experts.size(1) > INT32_MAX) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    out.allocate(c, z.t.sizes());
    const hgb_status s = hgb_gate_backward(c.ctx, (const float*)grad.data_ptr(), z.p, z.type, z.stride, z.n, (int32_t)z.dim, score,
                                           (const int32_t*)experts.data_ptr(), (int32_t)experts.size(1), renormalise, scale, out.r.p,
                                           out.r.stride);
    return s == HGB_OK ? wrap(out.r.t) : status(s);
}

// A loss's rows, table and tokens.
struct HeadRows {
    Rows x, table;
    const Tensor& token;
    HeadRows(const Call& c, PyObject* x_, PyObject* table_, PyObject* token_, const char* name, bool slots)
        : x(rows(c, x_, "x")), table(rows(c, table_, "table")), token(plain(c, token_, name, at::kInt))
    {
        if (table.t.dim() != 2) throw Refused("table must be two-dimensional");
        same(table.t.scalar_type(), x.t.scalar_type(), "table");
        if (table.dim != x.dim) throw Refused("table has rows of %lld values, needs %lld", (long long)table.dim, (long long)x.dim);
        const int64_t dims = x.t.dim() - (slots ? 0 : 1);
        if (token.dim() != dims || token.sizes().slice(0, x.t.dim() - 1) != lead())
            throw Refused(slots ? "%s must have x's shape, with the slots last" : "%s must have x's shape, without its last dimension", name);
        if (slots && token.size(-1) > INT32_MAX) throw Refused("%s has too many slots", name);
    }
    at::IntArrayRef lead() const { return x.t.sizes().slice(0, x.t.dim() - 1); }
    const int32_t* tokens() const { return (const int32_t*)token.data_ptr(); }
    // a float for each row
    const Tensor& each(const Call& c, PyObject* o, const char* name) const
    {
        const Tensor& t = plain(c, o, name, at::kFloat);
        if (t.sizes() != lead()) throw Refused("%s must have x's shape, without its last dimension", name);
        return t;
    }
    int64_t bytes() const { return hgb_head_workspace(x.p, x.stride, table.p, table.stride, x.type, x.n, table.n, x.dim); }
    int64_t grad_bytes(int type) const
    {
        return hgb_head_backward_workspace(x.p, x.stride, table.p, table.stride, x.type, type, x.n, table.n, x.dim);
    }
};

// A teacher's logits, one for each token.
struct Teacher {
    const Tensor& t;
    int type;
    Teacher(const Call& c, PyObject* o, const HeadRows& h) : t(tensor(c, o, "teacher")), type(code(t.scalar_type(), "teacher"))
    {
        if (t.scalar_type() != at::kFloat) same(t.scalar_type(), h.x.t.scalar_type(), "teacher");
        if (!t.is_contiguous()) throw Refused("teacher must be contiguous");
        if (t.sizes() != h.token.sizes()) throw Refused("teacher must have the tokens' shape");
    }
};

// cross_entropy(x, table, targets, scale, pad)
PyObject* cross_entropy(const Call& c)
{
    const HeadRows h(c, c.args[0], c.args[1], c.args[2], "targets", false);
    const float scale = real(c.args[3], "scale");
    const int32_t pad = whole32(c.args[4], "pad");
    const int64_t bytes = h.bytes();
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    const Tensor loss = c.make(h.lead(), at::kFloat), lse = c.make(h.lead(), at::kFloat), ws = c.workspace(bytes);
    const hgb_status s = hgb_cross_entropy(c.ctx, h.x.p, h.x.type, h.x.stride, h.x.n, h.x.dim, h.table.p, h.table.stride, h.table.n,
                                           h.tokens(), pad, scale, (float*)loss.data_ptr(), (float*)lse.data_ptr(), ptr(ws), bytes);
    return s == HGB_OK ? tuple({loss, lse}) : status(s);
}

// cross_entropy_backward(grad, x, table, targets, lse, scale, pad, dtype, out)
PyObject* cross_entropy_backward(const Call& c)
{
    const HeadRows h(c, c.args[1], c.args[2], c.args[3], "targets", false);
    const Tensor &grad = h.each(c, c.args[0], "grad"), &lse = h.each(c, c.args[4], "lse");
    const float scale = real(c.args[5], "scale");
    const int32_t pad = whole32(c.args[6], "pad");
    Out dtable(c, Py_None, dtype(c.args[7], h.x.t.scalar_type()), false, h.table.n, h.x.dim);
    Out out(c, c.args[8], h.x.t.scalar_type(), true, h.x.n, h.x.dim);
    const int64_t bytes = h.grad_bytes(dtable.r.type);
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    dtable.allocate(c, {h.table.n, h.x.dim});
    out.allocate(c, h.x.t.sizes());
    const Tensor ws = c.workspace(bytes);
    const hgb_status s = hgb_cross_entropy_backward(
        c.ctx, (const float*)grad.data_ptr(), h.x.p, h.x.type, h.x.stride, h.x.n, h.x.dim, h.table.p, h.table.stride, h.table.n,
        h.tokens(), pad, scale, (const float*)lse.data_ptr(), out.r.p, out.r.stride, dtable.r.p, dtable.r.type, dtable.r.stride, ptr(ws),
        bytes);
    return s == HGB_OK ? tuple({out.r.t, dtable.r.t}) : status(s);
}

// distill(x, table, tokens, teacher, temperature)
PyObject* distill(const Call& c)
{
    const HeadRows h(c, c.args[0], c.args[1], c.args[2], "tokens", true);
    const Teacher teacher(c, c.args[3], h);
    const float heat = real(c.args[4], "temperature");
    const int64_t bytes = h.bytes();
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    const Tensor loss = c.make(h.lead(), at::kFloat), lse = c.make(h.lead(), at::kFloat), picked = c.make(h.token.sizes(), at::kFloat);
    const Tensor ws = c.workspace(bytes);
    const hgb_status s = hgb_distill(c.ctx, h.x.p, h.x.type, h.x.stride, h.x.n, h.x.dim, h.table.p, h.table.stride, h.table.n, h.tokens(),
                                     teacher.t.data_ptr(), teacher.type, (int32_t)h.token.size(-1), heat, (float*)loss.data_ptr(),
                                     (float*)lse.data_ptr(), (float*)picked.data_ptr(), ptr(ws), bytes);
    return s == HGB_OK ? tuple({loss, lse, picked}) : status(s);
}

// distill_backward(grad, x, table, tokens, teacher, lse, picked, temperature, dtype, out)
PyObject* distill_backward(const Call& c)
{
    const HeadRows h(c, c.args[1], c.args[2], c.args[3], "tokens", true);
    const Teacher teacher(c, c.args[4], h);
    const Tensor &grad = h.each(c, c.args[0], "grad"), &lse = h.each(c, c.args[5], "lse");
    const Tensor& picked = plain(c, c.args[6], "picked", at::kFloat);
    if (picked.sizes() != h.token.sizes()) throw Refused("picked must have the tokens' shape");
    const float heat = real(c.args[7], "temperature");
    Out dtable(c, Py_None, dtype(c.args[8], h.x.t.scalar_type()), false, h.table.n, h.x.dim);
    Out out(c, c.args[9], h.x.t.scalar_type(), true, h.x.n, h.x.dim);
    const int64_t bytes = h.grad_bytes(dtable.r.type);
    if (bytes < 0) return status(kTooLarge);
    if (c.elsewhere()) return status(kElsewhere);
    dtable.allocate(c, {h.table.n, h.x.dim});
    out.allocate(c, h.x.t.sizes());
    const Tensor ws = c.workspace(bytes);
    const hgb_status s = hgb_distill_backward(
        c.ctx, (const float*)grad.data_ptr(), h.x.p, h.x.type, h.x.stride, h.x.n, h.x.dim, h.table.p, h.table.stride, h.table.n,
        h.tokens(), teacher.t.data_ptr(), teacher.type, (int32_t)h.token.size(-1), heat, (const float*)lse.data_ptr(),
        (const float*)picked.data_ptr(), out.r.p, out.r.stride, dtable.r.p, dtable.r.type, dtable.r.stride, ptr(ws), bytes);
    return s == HGB_OK ? tuple({out.r.t, dtable.r.t}) : status(s);
}

// The Python function of a verb: (handle, device, stream id, its COUNT arguments).
template <PyObject* (*F)(const Call&), int COUNT>
PyObject* verb(PyObject*, PyObject* const* args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    try {
        if (count != COUNT + 3) throw Refused("%d arguments, needs %d", (int)count, COUNT + 3);
        const Call c{(hgb_ctx*)(uintptr_t)whole(args[0], "the context"), (int)whole(args[1], "device"), whole(args[2], "stream"),
                     args + 3};
        return F(c);
    } catch (const Refused& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(const Call&), int COUNT>
PyMethodDef method(const char* name)
{
    return {name, (PyCFunction)(void (*)(void))verb<F, COUNT>, METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<embed, 6>("embed"),
    method<embed_backward, 7>("embed_backward"),
    method<layer_norm, 5>("layer_norm"),
    method<layer_norm_backward, 7>("layer_norm_backward"),
    method<route, 2>("route"),
    method<route_gather, 4>("route_gather"),
    method<route_gather_backward, 4>("route_gather_backward"),
    method<route_combine, 5>("route_combine"),
    method<route_combine_backward, 6>("route_combine_backward"),
    method<gate, 9>("gate"),
    method<gate_backward, 7>("gate_backward"),
    method<cross_entropy, 5>("cross_entropy"),
    method<cross_entropy_backward, 9>("cross_entropy_backward"),
    method<distill, 5>("distill"),
    method<distill_backward, 10>("distill_backward"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_verbs", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__verbs(void) { return PyModule_Create(&module); }
