// Python calls of the layer operators (layers.py): argument checks, result
// tensors, stream and launch, on torch tensors. A single-token call takes a few
// microseconds on the device, and a Python function that checks nine tensors
// and converts twenty arguments about twenty on the host; so this is compiled.
//
// The functions take positional arguments in the order of layers.py. Refusals
// are TypeError or ValueError raised before anything is launched, a status from
// the library is GdrError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <string>
#include <vector>

#include "gdr.h"

namespace {

using at::Tensor;
typedef const Tensor* Opt;  // null for None

PyObject* gdr_error = nullptr;  // _lib.GdrError

struct Refusal {
    PyObject* type;
    std::string text;
};
[[noreturn]] void bad_value(std::string s) { throw Refusal{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void bad_type(std::string s) { throw Refusal{PyExc_TypeError, std::move(s)}; }

std::string shape_text(at::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        default: return std::string("torch.") + c10::toString(t);
    }
}

// Types a tensor may have.
struct Types {
    at::ScalarType a, b;
    Types(at::ScalarType one) : a(one), b(one) {}
    Types(at::ScalarType one, at::ScalarType two) : a(one), b(two) {}
    bool has(at::ScalarType t) const { return t == a || t == b; }
    std::string text() const { return a == b ? type_text(a) : type_text(a) + " or " + type_text(b); }
};

Opt tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) bad_type(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const Tensor& required(PyObject* o, const char* name) {
    Opt t = tensor(o, name);
    if (!t) bad_type(std::string(name) + " must be a tensor");
    return *t;
}
int code_of(at::ScalarType t) { return t == at::kBFloat16 ? GDR_BF16 : GDR_FP32; }

// An axis's size as the library's int.
int64_t counted(const char* name, int64_t n) {
    if (n > INT_MAX) bad_value(std::string(name) + " has an axis of " + std::to_string(n) + "; the library counts in int");
    return n;
}
// Type code of the tensor that the others are held to.
int first(const char* name, const Tensor& t, int ndim) {
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
        bad_type("unsupported dtype " + type_text(t.scalar_type()) + "; use bfloat16 or float32");
    if (!t.is_cuda()) bad_value(std::string(name) + " is on " + t.device().str() + "; the library takes CUDA tensors");
    if (t.dim() != ndim)
        bad_value(std::string(name) + " has " + std::to_string(t.dim()) + " axes; expected " + std::to_string(ndim));
    for (int64_t n : t.sizes()) counted(name, n);
    return code_of(t.scalar_type());
}
void axes(const char* name, const Tensor& t, int ndim) {
    if (t.dim() != ndim)
        bad_value(std::string(name) + " has " + std::to_string(t.dim()) + " axes; expected " + std::to_string(ndim));
}
// Shape, type and device; the last `tail` axes dense.
void check(const char* name, const Tensor& t, at::IntArrayRef shape, Types types, c10::Device dev, int tail = 1) {
    if (!types.has(t.scalar_type()))
        bad_type(std::string(name) + " has dtype " + type_text(t.scalar_type()) + "; expected " + types.text());
    if (t.device() != dev) bad_value(std::string(name) + " is on " + t.device().str() + "; expected " + dev.str());
    if (t.sizes() != shape)
        bad_value(std::string(name) + " has shape " + shape_text(t.sizes()) + "; expected " + shape_text(shape));
    int64_t want = 1;
    for (int i = 1; i <= tail; ++i) {
        const size_t ax = shape.size() - i;
        if (shape[ax] > 1 && t.stride(ax) != want)
            bad_value(std::string(name) + (tail > 1 ? ": the last " + std::to_string(tail) + " axes must be dense"
                                                    : ": the innermost axis must be dense"));
        want *= shape[ax];
    }
}
void dense(const char* name, Opt t, at::IntArrayRef shape, Types types, c10::Device dev) {
    if (!t) return;
    check(name, *t, shape, types, dev, 0);
    if (!t->is_contiguous()) bad_value(std::string(name) + " must be contiguous");
}

struct Named {
    const char* name;
    Opt t;
};
std::pair<char*, char*> span(const Tensor& t) {
    int64_t n = t.numel() ? 1 : 0;
    if (n)
        for (int64_t i = 0; i < t.dim(); ++i) n += (t.size(i) - 1) * t.stride(i);
    char* p = static_cast<char*>(t.data_ptr());
    return {p, p + n * (int64_t)t.element_size()};
}
// A given result t shares no memory with the others. It may be `same`, the one
// input that the call may overwrite, where that is dense (t is): rows in another
// order over the same memory would be overwritten before they are read.
void apart(const char* name, Opt t, std::initializer_list<Named> others, Named same = {nullptr, nullptr}) {
    if (!t || !t->numel()) return;
    const auto a = span(*t);
    auto refuse = [&](const Named& o, bool whole) {
        if (!o.t || !o.t->numel()) return;
        const auto b = span(*o.t);
        if (whole && b == a && o.t->is_contiguous()) return;
        if (a.first < b.second && b.first < a.second) bad_value(std::string(name) + " overlaps " + o.name);
    };
    for (const Named& o : others) refuse(o, false);
    refuse(same, true);
}

void* ptr(Opt t) { return t ? t->data_ptr() : nullptr; }
float* fptr(Opt t) { return static_cast<float*>(ptr(t)); }
const int* iptr(Opt t) { return static_cast<const int*>(ptr(t)); }
double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        bad_type(std::string(name) + " must be a number");
    }
    return v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v;
}
// The value of one of `options`; `none` for None, where that is allowed (>= 0).
int choice(PyObject* o, const char* name, std::initializer_list<std::pair<const char*, int>> options,
           const char* expected, int none = -1) {
    if (o == Py_None && none >= 0) return none;
    if (PyUnicode_Check(o)) {
        const char* s = PyUnicode_AsUTF8(o);
        if (!s) throw python_error();
        for (const auto& c : options)
            if (!std::strcmp(c.first, s)) return c.second;
    }
    PyObject* r = PyObject_Repr(o);
    const char* text = r ? PyUnicode_AsUTF8(r) : nullptr;
    std::string t = text ? text : "?";
    Py_XDECREF(r);
    PyErr_Clear();
    bad_value(std::string(name) + " " + t + "; expected " + expected);
}

// The device and stream of one call. Tensors that the call makes come from the
// launch stream's pool, so nothing else can be using their memory; with a
// stream other than the current one they are marked as used by that too.
struct Where {
    c10::Device dev;
    c10::cuda::OptionalCUDAGuard device;
    c10::cuda::CUDAStream here, launch;
    bool side = false;

    Where(c10::Device d, PyObject* stream)
        : dev(d), here(c10::cuda::getCurrentCUDAStream(d.index())), launch(here) {
        if (c10::cuda::current_device() != d.index()) device.set_index(d.index());
        if (stream == Py_None) return;
        unsigned long long handle = 0;
        if (PyLong_Check(stream)) {
            handle = PyLong_AsUnsignedLongLong(stream);
            if (PyErr_Occurred()) throw python_error();
        } else {
            PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
            if (!h) throw python_error();
            handle = PyLong_AsUnsignedLongLong(h);
            Py_DECREF(h);
            if (PyErr_Occurred()) throw python_error();
            PyObject* i = PyObject_GetAttrString(stream, "device_index");
            if (i) {
                const long index = PyLong_AsLong(i);
                Py_DECREF(i);
                if (PyErr_Occurred()) throw python_error();
                if (index != d.index())
                    bad_value("stream is on cuda:" + std::to_string(index) + "; expected " + d.str());
            } else {
                PyErr_Clear();
            }
        }
        const auto raw = reinterpret_cast<cudaStream_t>(handle);
        if (raw == here.stream()) return;
        side = true;
        launch = raw ? c10::cuda::getStreamFromExternal(raw, d.index()) : c10::cuda::getDefaultCUDAStream(d.index());
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type, bool result = true) {
        if (!side) return at::detail::empty_cuda(shape, type, dev, c10::nullopt);
        c10::cuda::CUDAStreamGuard guard(launch);
        Tensor t = at::detail::empty_cuda(shape, type, dev, c10::nullopt);
        if (result) t.record_stream(here);
        return t;
    }
    // The caller's workspace, or one of `bytes` from torch, held until the call returns.
    Tensor workspace(Opt given, size_t bytes) {
        if (!given) return empty({(int64_t)(bytes ? bytes : 1)}, at::kByte, false);
        if (given->device() != dev)
            bad_value("workspace is on " + given->device().str() + "; expected " + dev.str());
        if (!given->is_contiguous()) bad_value("workspace must be contiguous");
        return *given;
    }
    void* stream() const { return launch.stream(); }
};
size_t bytes_of(const Tensor& t) { return t.numel() * t.element_size(); }

struct Status {
    const char* fn;
    gdr_status st;
};
void done(const char* fn, gdr_status st) {
    if (st != GDR_OK) throw Status{fn, st};
}

PyObject* wrap(Tensor t) { return t.defined() ? THPVariable_Wrap(std::move(t)) : Py_NewRef(Py_None); }
PyObject* wrap_or(PyObject* given, const Tensor& made) { return given != Py_None ? Py_NewRef(given) : wrap(made); }
PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}
PyObject* dict(std::initializer_list<std::pair<const char*, Tensor>> items) {
    PyObject* d = PyDict_New();
    for (const auto& it : items) {
        PyObject* v = d ? wrap(it.second) : nullptr;
        if (!v || PyDict_SetItemString(d, it.first, v) < 0) {
            Py_XDECREF(v);
            Py_XDECREF(d);
            return nullptr;
        }
        Py_DECREF(v);
    }
    return d;
}

// ---------------------------------------------------------------- convolution

struct ConvArgs {
    const Tensor &x, &weight;
    Opt bias;
    int code, act, W;
    int64_t D;
    Types own, param;
    ConvArgs(PyObject* xo, PyObject* wo, PyObject* bo, PyObject* activation, int ndim)
        : x(required(xo, "x")), weight(required(wo, "weight")), bias(tensor(bo, "bias")), code(first("x", x, ndim)),
          own(x.scalar_type()), param(x.scalar_type(), at::kFloat) {
        const auto dev = x.device();
        D = x.size(ndim - 1);
        axes("weight", weight, 2);
        W = (int)counted("weight", weight.size(1));
        dense("weight", &weight, {D, W}, param, dev);
        dense("bias", bias, {D}, weight.scalar_type(), dev);
        act = choice(activation, "activation", {{"silu", GDR_ACT_SILU}, {"none", GDR_ACT_NONE}}, "'silu' or None",
                     GDR_ACT_NONE);
    }
};

// x, weight, bias, X0, activation, lengths, out, final_state, X_T, stream
PyObject* conv_fwd(PyObject* const* a) {
    const ConvArgs c(a[0], a[1], a[2], a[4], 3);
    const auto dev = c.x.device();
    const int64_t B = c.x.size(0), T = c.x.size(1), D = c.D, W = c.W;
    check("x", c.x, {B, T, D}, c.own, dev);
    const Opt X0 = tensor(a[3], "X0"), lengths = tensor(a[5], "lengths"), out = tensor(a[6], "out"),
              XT = tensor(a[8], "X_T");
    dense("X0", X0, {B, W - 1, D}, c.own, dev);
    dense("X_T", XT, {B, W - 1, D}, c.own, dev);
    dense("out", out, {B, T, D}, c.own, dev);
    dense("lengths", lengths, {B}, at::kInt, dev);
    apart("out", out, {{"x", &c.x}, {"weight", &c.weight}, {"bias", c.bias}, {"lengths", lengths}, {"X0", X0}, {"X_T", XT}});
    apart("X_T", XT, {{"x", &c.x}, {"weight", &c.weight}, {"bias", c.bias}, {"lengths", lengths}}, {"X0", X0});
    const bool final_state = truth(a[7]);
    Where at(dev, a[9]);
    Tensor y, last;
    if (!out) y = at.empty({B, T, D}, c.x.scalar_type());
    if (final_state && !XT) last = at.empty({B, W - 1, D}, c.x.scalar_type());
    const long long st[2] = {c.x.stride(0), c.x.stride(1)};
    done("gdr_conv_fwd",
         gdr_conv_fwd(ptr(&c.x), ptr(&c.weight), ptr(c.bias), ptr(X0), iptr(lengths), ptr(out ? out : &y),
                      !final_state ? nullptr : ptr(XT ? XT : &last), st, B, T, D, W, c.act, c.code,
                      code_of(c.weight.scalar_type()), at.stream()));
    return pair(wrap_or(a[6], y), final_state ? wrap_or(a[8], last) : Py_NewRef(Py_None));
}

// x, weight, bias, X0, dy, dX_T, activation, lengths, workspace, need_dX0, stream
PyObject* conv_bwd(PyObject* const* a) {
    const ConvArgs c(a[0], a[1], a[2], a[6], 3);
    const auto dev = c.x.device();
    const int64_t B = c.x.size(0), T = c.x.size(1), D = c.D, W = c.W;
    check("x", c.x, {B, T, D}, c.own, dev);
    const Tensor& dy = required(a[4], "dy");
    const Opt X0 = tensor(a[3], "X0"), dXT = tensor(a[5], "dX_T"), lengths = tensor(a[7], "lengths"),
              given = tensor(a[8], "workspace");
    check("dy", dy, {B, T, D}, c.param, dev);
    dense("X0", X0, {B, W - 1, D}, c.own, dev);
    dense("dX_T", dXT, {B, W - 1, D}, at::kFloat, dev);
    dense("lengths", lengths, {B}, at::kInt, dev);
    const bool need = truth(a[9]) && X0;
    Where at(dev, a[10]);
    Tensor dx = at.empty({B, T, D}, at::kFloat), dw = at.empty({D, W}, at::kFloat), db, dX0;
    if (c.bias) db = at.empty({D}, at::kFloat);
    if (need) dX0 = at.empty({B, W - 1, D}, at::kFloat);
    const Tensor ws = at.workspace(given, gdr_conv_bwd_workspace_size(B, T, D, W));
    const long long st[4] = {c.x.stride(0), c.x.stride(1), dy.stride(0), dy.stride(1)};
    done("gdr_conv_bwd",
         gdr_conv_bwd(ptr(&c.x), ptr(&c.weight), ptr(c.bias), ptr(X0), iptr(lengths), ptr(&dy), fptr(dXT), fptr(&dx),
                      fptr(&dw), c.bias ? fptr(&db) : nullptr, need ? fptr(&dX0) : nullptr, ptr(&ws), bytes_of(ws), st,
                      B, T, D, W, c.act, c.code, code_of(c.weight.scalar_type()), code_of(dy.scalar_type()),
                      at.stream()));
    return dict({{"dx", dx}, {"dweight", dw}, {"dbias", db}, {"dX0", dX0}});
}

// x, weight, bias, X, activation, out, stream
PyObject* conv_step(PyObject* const* a) {
    const ConvArgs c(a[0], a[1], a[2], a[4], 2);
    const auto dev = c.x.device();
    const int64_t B = c.x.size(0), D = c.D, W = c.W;
    check("x", c.x, {B, D}, c.own, dev);
    const Tensor& X = required(a[3], "X");
    const Opt out = tensor(a[5], "out");
    dense("X", &X, {B, W - 1, D}, c.own, dev);
    dense("out", out, {B, D}, c.own, dev);
    apart("X", &X, {{"x", &c.x}, {"weight", &c.weight}, {"bias", c.bias}});
    apart("out", out, {{"x", &c.x}, {"weight", &c.weight}, {"bias", c.bias}, {"X", &X}});
    Where at(dev, a[6]);
    Tensor y;
    if (!out) y = at.empty({B, D}, c.x.scalar_type());
    const long long st[1] = {c.x.stride(0)};
    done("gdr_conv_step",
         gdr_conv_step(ptr(&c.x), ptr(&c.weight), ptr(c.bias), ptr(&X), ptr(out ? out : &y), st, B, D, W, c.act, c.code,
                       code_of(c.weight.scalar_type()), at.stream()));
    return wrap_or(a[5], y);
}

// ---------------------------------------------------------------- selective scan

// u, delta, A, Bm, Cm, D, z, h first in every call; n: axes before D (1 or 2)
struct ScanTensors {
    const Tensor &u, &delta, &A, &Bm, &Cm;
    Opt D, z, h, bias;
    int code;
    int64_t B, T, Dn, N, G;
    long long st[12];
    ScanTensors(PyObject* const* a, PyObject* bias_o, const char* hname, int n)
        : u(required(a[0], "u")), delta(required(a[1], "delta")), A(required(a[2], "A")), Bm(required(a[3], "Bm")),
          Cm(required(a[4], "Cm")), D(tensor(a[5], "D")), z(tensor(a[6], "z")), h(tensor(a[7], hname)),
          bias(tensor(bias_o, "delta_bias")), code(first("u", u, n + 1)) {
        const auto dev = u.device();
        const Types own(u.scalar_type());
        axes("A", A, 2);
        axes("Bm", Bm, n + 2);
        B = u.size(0);
        T = n == 2 ? u.size(1) : 1;
        Dn = u.size(n);
        N = counted("A", A.size(1));
        G = counted("Bm", Bm.size(n));
        dense("A", &A, {Dn, N}, at::kFloat, dev);
        dense("D", D, {Dn}, at::kFloat, dev);
        dense("delta_bias", bias, {Dn}, at::kFloat, dev);
        dense(hname, h, {B, Dn, N}, at::kFloat, dev);
        const int64_t rows[3] = {B, n == 2 ? T : Dn, Dn}, vecs[4] = {B, n == 2 ? T : G, n == 2 ? G : N, N};
        const at::IntArrayRef row(rows, n + 1), vec(vecs, n + 2);
        check("u", u, row, own, dev);
        check("delta", delta, row, own, dev);
        check("Bm", Bm, vec, own, dev, 2);
        check("Cm", Cm, vec, own, dev, 2);
        if (z) check("z", *z, row, own, dev);
        int k = 0;
        for (const Tensor* t : {&u, &delta, &Bm, &Cm, z})
            for (int i = 0; i < n; ++i) st[k++] = t ? t->stride(i) : 0;
    }
};

// .. h0, delta_bias, delta_softplus, lengths, workspace, out, final_state, h_T, stream
PyObject* scan_fwd(PyObject* const* a) {
    ScanTensors s(a, a[8], "h0", 2);
    const auto dev = s.u.device();
    const Opt lengths = tensor(a[10], "lengths"), out = tensor(a[12], "out"), hT = tensor(a[14], "h_T");
    dense("h_T", hT, {s.B, s.Dn, s.N}, at::kFloat, dev);
    dense("out", out, {s.B, s.T, s.Dn}, s.u.scalar_type(), dev);
    dense("lengths", lengths, {s.B}, at::kInt, dev);
    apart("out", out, {{"u", &s.u}, {"delta", &s.delta}, {"A", &s.A}, {"Bm", &s.Bm}, {"Cm", &s.Cm}, {"D", s.D}, {"z", s.z},
                       {"h0", s.h}, {"delta_bias", s.bias}, {"lengths", lengths}, {"h_T", hT}});
    apart("h_T", hT, {{"u", &s.u}, {"delta", &s.delta}, {"A", &s.A}, {"Bm", &s.Bm}, {"Cm", &s.Cm}, {"D", s.D}, {"z", s.z},
                      {"delta_bias", s.bias}, {"lengths", lengths}}, {"h0", s.h});
    bool split = a[11] != Py_None;
    Opt given = nullptr;
    if (PyUnicode_Check(a[11])) choice(a[11], "workspace", {{"auto", 0}}, "'auto', None or a tensor");
    else given = tensor(a[11], "workspace");
    const bool final_state = truth(a[13]), softplus = truth(a[9]);
    Where at(dev, a[15]);
    Tensor y, last, ws;
    if (!out) y = at.empty({s.B, s.T, s.Dn}, s.u.scalar_type());
    if (final_state && !hT) last = at.empty({s.B, s.Dn, s.N}, at::kFloat);
    const size_t need = split ? gdr_scan_fwd_workspace_size(s.B, s.T, s.Dn, s.N, s.G) : 0;
    if (need) ws = at.workspace(given, need);
    done("gdr_scan_fwd",
         gdr_scan_fwd(ptr(&s.u), ptr(&s.delta), fptr(&s.A), ptr(&s.Bm), ptr(&s.Cm), fptr(s.D), ptr(s.z), fptr(s.bias),
                      fptr(s.h), iptr(lengths), ptr(out ? out : &y), !final_state ? nullptr : fptr(hT ? hT : &last),
                      need ? ptr(&ws) : nullptr, need ? bytes_of(ws) : 0, s.st, s.B, s.T, s.Dn, s.N, s.G, softplus,
                      s.code, at.stream()));
    return pair(wrap_or(a[12], y), final_state ? wrap_or(a[14], last) : Py_NewRef(Py_None));
}

// .. h0, dy, dh_T, delta_bias, delta_softplus, lengths, workspace, need_dh0, stream
PyObject* scan_bwd(PyObject* const* a) {
    ScanTensors s(a, a[10], "h0", 2);
    const auto dev = s.u.device();
    const Tensor& dy = required(a[8], "dy");
    const Opt dhT = tensor(a[9], "dh_T"), lengths = tensor(a[12], "lengths"), given = tensor(a[13], "workspace");
    check("dy", dy, {s.B, s.T, s.Dn}, Types(s.u.scalar_type(), at::kFloat), dev);
    dense("dh_T", dhT, {s.B, s.Dn, s.N}, at::kFloat, dev);
    dense("lengths", lengths, {s.B}, at::kInt, dev);
    s.st[10] = dy.stride(0);
    s.st[11] = dy.stride(1);
    const bool softplus = truth(a[11]), need = truth(a[14]) && s.h;
    Where at(dev, a[15]);
    const auto f32 = at::kFloat;
    Tensor du = at.empty({s.B, s.T, s.Dn}, f32), dd = at.empty({s.B, s.T, s.Dn}, f32), dA = at.empty({s.Dn, s.N}, f32),
           dB = at.empty({s.B, s.T, s.G, s.N}, f32), dC = at.empty({s.B, s.T, s.G, s.N}, f32), dD, dz, db, dh0;
    if (s.D) dD = at.empty({s.Dn}, f32);
    if (s.z) dz = at.empty({s.B, s.T, s.Dn}, f32);
    if (s.bias) db = at.empty({s.Dn}, f32);
    if (need) dh0 = at.empty({s.B, s.Dn, s.N}, f32);
    const Tensor ws = at.workspace(given, gdr_scan_bwd_workspace_size(s.B, s.T, s.Dn, s.N, s.G));
    done("gdr_scan_bwd",
         gdr_scan_bwd(ptr(&s.u), ptr(&s.delta), fptr(&s.A), ptr(&s.Bm), ptr(&s.Cm), fptr(s.D), ptr(s.z), fptr(s.bias),
                      fptr(s.h), iptr(lengths), ptr(&dy), fptr(dhT), fptr(&du), fptr(&dd), fptr(&dA), fptr(&dB),
                      fptr(&dC), s.D ? fptr(&dD) : nullptr, s.z ? fptr(&dz) : nullptr, s.bias ? fptr(&db) : nullptr,
                      need ? fptr(&dh0) : nullptr, ptr(&ws), bytes_of(ws), s.st, s.B, s.T, s.Dn, s.N, s.G, softplus,
                      s.code, code_of(dy.scalar_type()), at.stream()));
    return dict({{"du", du}, {"ddelta", dd}, {"dA", dA}, {"dB", dB}, {"dC", dC}, {"dD", dD}, {"dz", dz},
                 {"ddelta_bias", db}, {"dh0", dh0}});
}

// .. h, delta_bias, delta_softplus, out, stream
PyObject* scan_step(PyObject* const* a) {
    ScanTensors s(a, a[8], "h", 1);
    const auto dev = s.u.device();
    const Tensor& h = required(a[7], "h");
    const Opt out = tensor(a[10], "out");
    dense("out", out, {s.B, s.Dn}, s.u.scalar_type(), dev);
    apart("h", &h, {{"u", &s.u}, {"delta", &s.delta}, {"A", &s.A}, {"Bm", &s.Bm}, {"Cm", &s.Cm}, {"D", s.D}, {"z", s.z},
                    {"delta_bias", s.bias}});
    apart("out", out, {{"u", &s.u}, {"delta", &s.delta}, {"A", &s.A}, {"Bm", &s.Bm}, {"Cm", &s.Cm}, {"D", s.D},
                       {"z", s.z}, {"h", &h}, {"delta_bias", s.bias}});
    const bool softplus = truth(a[9]);
    Where at(dev, a[11]);
    Tensor y;
    if (!out) y = at.empty({s.B, s.Dn}, s.u.scalar_type());
    done("gdr_scan_step",
         gdr_scan_step(ptr(&s.u), ptr(&s.delta), fptr(&s.A), ptr(&s.Bm), ptr(&s.Cm), fptr(s.D), ptr(s.z), fptr(s.bias),
                       fptr(&h), ptr(out ? out : &y), s.st, s.B, s.Dn, s.N, s.G, softplus, s.code, at.stream()));
    return wrap_or(a[10], y);
}

// ---------------------------------------------------------------- norm and rotation

// q, k, q_weight, k_weight, kind, eps, q_scale, positions, inv_freq, rotary, rotary_scale
struct NormTensors {
    const Tensor& q;
    Opt k, qw, kw, pos, freq;
    int code, kind, rotary, pos64 = 0, rot = 0, wcode;
    int64_t B, T, Hq, Hk = 0, d;
    float eps, q_scale, rscale;
    long long st[14] = {};
    explicit NormTensors(PyObject* const* a)
        : q(required(a[0], "q")), k(tensor(a[1], "k")), qw(tensor(a[2], "q_weight")), kw(tensor(a[3], "k_weight")),
          pos(tensor(a[7], "positions")), freq(tensor(a[8], "inv_freq")), code(first("q", q, 4)) {
        const auto dev = q.device();
        const Types own(q.scalar_type());
        B = q.size(0); T = q.size(1); Hq = q.size(2); d = q.size(3);
        check("q", q, {B, T, Hq, d}, own, dev);
        for (int i = 0; i < 3; ++i) st[i] = q.stride(i);
        if (k) {
            axes("k", *k, 4);
            Hk = counted("k", k->size(2));
            check("k", *k, {B, T, Hk, d}, own, dev);
            for (int i = 0; i < 3; ++i) st[3 + i] = k->stride(i);
        }
        Types wt(q.scalar_type(), at::kFloat);
        for (const Named& w : {Named{"q_weight", qw}, Named{"k_weight", kw}})
            if (w.t) {
                dense(w.name, w.t, {d}, wt, dev);
                wt = Types(w.t->scalar_type());
            }
        wcode = code_of(qw || kw ? wt.a : q.scalar_type());
        kind = choice(a[4], "kind", {{"l2", GDR_NORM_L2}, {"rms", GDR_NORM_RMS}}, "'l2' or 'rms'");
        rotary = choice(a[9], "rotary", {{"half", GDR_ROTARY_HALF}, {"interleaved", GDR_ROTARY_INTERLEAVED}},
                        "'half' or 'interleaved'");
        if (freq) {
            rot = (int)std::min<int64_t>(2 * freq->numel(), INT_MAX - 1);  // even; refused where above d
            dense("inv_freq", freq, {freq->numel()}, at::kFloat, dev);
        }
        if (pos) {
            check("positions", *pos, {B, T}, Types(at::kInt, at::kLong), dev, 0);
            pos64 = pos->scalar_type() == at::kLong;
            st[6] = pos->stride(0);
            st[7] = pos->stride(1);
        }
        eps = (float)number(a[5], "eps");
        q_scale = (float)number(a[6], "q_scale");
        rscale = (float)number(a[10], "rotary_scale");
    }
};

// .. q_out, k_out, stream
PyObject* qk_norm_fwd(PyObject* const* a) {
    NormTensors n(a);
    const auto dev = n.q.device();
    const Opt qo = tensor(a[11], "q_out"), ko = tensor(a[12], "k_out");
    dense("q_out", qo, {n.B, n.T, n.Hq, n.d}, n.q.scalar_type(), dev);
    if (ko && !n.k) bad_value("k_out without k");
    dense("k_out", ko, {n.B, n.T, n.Hk, n.d}, n.q.scalar_type(), dev);
    apart("q_out", qo, {{"q_weight", n.qw}, {"k_weight", n.kw}, {"positions", n.pos}, {"inv_freq", n.freq}, {"k", n.k},
                        {"k_out", ko}}, {"q", &n.q});
    apart("k_out", ko, {{"q_weight", n.qw}, {"k_weight", n.kw}, {"positions", n.pos}, {"inv_freq", n.freq}, {"q", &n.q}},
          {"k", n.k});
    Where at(dev, a[13]);
    Tensor yq, yk;
    if (!qo) yq = at.empty({n.B, n.T, n.Hq, n.d}, n.q.scalar_type());
    if (n.k && !ko) yk = at.empty({n.B, n.T, n.Hk, n.d}, n.q.scalar_type());
    done("gdr_qk_norm_fwd",
         gdr_qk_norm_fwd(ptr(&n.q), ptr(n.k), ptr(n.qw), ptr(n.kw), ptr(n.pos), fptr(n.freq), ptr(qo ? qo : &yq),
                         !n.k ? nullptr : ptr(ko ? ko : &yk), n.st, n.B, n.T, n.Hq, n.Hk, n.d, n.rot, n.kind, n.rotary,
                         n.eps, n.q_scale, n.rscale, n.pos64, n.code, n.wcode, at.stream()));
    return pair(wrap_or(a[11], yq), wrap_or(a[12], yk));
}

// .. dq, dk, workspace, stream
PyObject* qk_norm_bwd(PyObject* const* a) {
    NormTensors n(a);
    const auto dev = n.q.device();
    const Tensor& gq = required(a[11], "dq");
    const Opt gk = tensor(a[12], "dk"), given = tensor(a[13], "workspace");
    check("dq", gq, {n.B, n.T, n.Hq, n.d}, Types(n.q.scalar_type(), at::kFloat), dev);
    if (!gk != !n.k) bad_value("dk is given exactly when k is");
    if (gk) check("dk", *gk, {n.B, n.T, n.Hk, n.d}, gq.scalar_type(), dev);
    for (int i = 0; i < 3; ++i) {
        n.st[8 + i] = gq.stride(i);
        n.st[11 + i] = gk ? gk->stride(i) : 0;
    }
    Where at(dev, a[14]);
    Tensor dq = at.empty({n.B, n.T, n.Hq, n.d}, at::kFloat), dk, dqw, dkw, ws;
    if (n.k) dk = at.empty({n.B, n.T, n.Hk, n.d}, at::kFloat);
    if (n.qw) dqw = at.empty({n.d}, at::kFloat);
    if (n.kw) dkw = at.empty({n.d}, at::kFloat);
    const bool weights = n.qw || n.kw;
    if (weights) ws = at.workspace(given, gdr_qk_norm_bwd_workspace_size((int)n.d));
    done("gdr_qk_norm_bwd",
         gdr_qk_norm_bwd(ptr(&n.q), ptr(n.k), ptr(n.qw), ptr(n.kw), ptr(n.pos), fptr(n.freq), ptr(&gq), ptr(gk),
                         fptr(&dq), n.k ? fptr(&dk) : nullptr, n.qw ? fptr(&dqw) : nullptr,
                         n.kw ? fptr(&dkw) : nullptr, weights ? ptr(&ws) : nullptr, weights ? bytes_of(ws) : 0, n.st,
                         n.B, n.T, n.Hq, n.Hk, n.d, n.rot, n.kind, n.rotary, n.eps, n.q_scale, n.rscale, n.pos64,
                         n.code, n.wcode, code_of(gq.scalar_type()), at.stream()));
    return dict({{"dq", dq}, {"dk", dk}, {"dq_weight", dqw}, {"dk_weight", dkw}});
}

// ---------------------------------------------------------------- the module

// name, tensor, shape, tail: the check of one tensor (its own type and device), returns its strides
PyObject* check_tensor(PyObject* const* a) {
    const Tensor& t = required(a[1], "tensor");
    std::vector<int64_t> shape;
    for (Py_ssize_t i = 0; i < PyTuple_Size(a[2]); ++i) shape.push_back(PyLong_AsLongLong(PyTuple_GetItem(a[2], i)));
    if (PyErr_Occurred()) throw python_error();
    check(PyUnicode_AsUTF8(a[0]), t, shape, Types(at::kBFloat16), t.device(), (int)PyLong_AsLong(a[3]));
    PyObject* r = PyTuple_New(t.dim());
    for (int64_t i = 0; i < t.dim(); ++i) PyTuple_SetItem(r, i, PyLong_FromLongLong(t.stride(i)));
    return r;
}
// name, tensor, other name, other tensor, may be the same
PyObject* check_apart(PyObject* const* a) {
    const Opt t = tensor(a[1], "tensor"), o = tensor(a[3], "tensor");
    const Named other = {PyUnicode_AsUTF8(a[2]), o};
    if (truth(a[4])) apart(PyUnicode_AsUTF8(a[0]), t, {}, other);
    else apart(PyUnicode_AsUTF8(a[0]), t, {other});
    Py_RETURN_NONE;
}
PyObject* set_error(PyObject* const* a) {
    Py_XDECREF(gdr_error);
    gdr_error = Py_NewRef(a[0]);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int ARGC>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != ARGC) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGC, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal& r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    } catch (const Status& s) {
        PyObject* e = gdr_error ? PyObject_CallFunction(gdr_error, "si", s.fn, (int)s.st) : nullptr;
        if (e) PyErr_SetObject(gdr_error, e);
        else if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s returned status %d", s.fn, (int)s.st);
        Py_XDECREF(e);
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

#define GDR_METHOD(F, ARGC) {#F, (PyCFunction)(void (*)(void))entry<F, ARGC>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    GDR_METHOD(conv_fwd, 10), GDR_METHOD(conv_bwd, 11), GDR_METHOD(conv_step, 7), GDR_METHOD(scan_fwd, 16),
    GDR_METHOD(scan_bwd, 16), GDR_METHOD(scan_step, 12), GDR_METHOD(qk_norm_fwd, 14), GDR_METHOD(qk_norm_bwd, 15),
    GDR_METHOD(check_tensor, 4), GDR_METHOD(check_apart, 5), GDR_METHOD(set_error, 1), {nullptr, nullptr, 0, nullptr}};
#undef GDR_METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&module); }
