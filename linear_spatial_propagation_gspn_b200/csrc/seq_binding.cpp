// seq_binding.cpp -- the common case of the token-sequence calls without the interpreter's work.
//
// A call for a few tokens is launched faster than Python checks its arguments, so the calls of seq.py
// come here first. Each function takes its arguments in a fixed order and either makes the whole call
// (checks, allocation of what is returned, launch on the current stream) or returns None: for whatever
// is not plain CUDA tensors of the right shapes and types on the current device, and for a call that
// the library refuses. seq.py then goes through its own checks, which say what is wrong. No torch type
// crosses the C ABI: the library's entry points are called by address, as ctypes calls them.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "gspn_seq.h"

namespace {

using at::ScalarType;
using at::Tensor;

// Entry points, in the order of `names` in init().
struct {
    decltype(&gspn_conv_workspace_size) conv_ws;
    decltype(&gspn_conv_forward) conv_forward;
    decltype(&gspn_conv_backward) conv_backward;
    decltype(&gspn_conv_step) conv_step;
    decltype(&gspn_ssm_workspace_size) ssm_ws;
    decltype(&gspn_ssm_hsave_size) ssm_hsave;
    decltype(&gspn_ssm_forward) ssm_forward;
    decltype(&gspn_ssm_backward) ssm_backward;
    decltype(&gspn_ssm_step) ssm_step;
    decltype(&gspn_norm_workspace_size) norm_ws;
    decltype(&gspn_norm_forward) norm_forward;
    decltype(&gspn_norm_backward) norm_backward;
} lib;

#define DECLINE Py_RETURN_NONE
#define NEED(c) \
    if (!(c)) DECLINE

// A call that got as far as the device must not be made again by the Python path: a step would move its
// states twice. Its error is raised here.
PyObject* raised(const char* what, int status) {
    PyObject* package = PyImport_ImportModule("linear_spatial_propagation_gspn_b200");
    PyObject* type = package ? PyObject_GetAttrString(package, "GspnError") : nullptr;
    PyObject* error = type ? PyObject_CallFunction(type, "is", status, what) : nullptr;
    if (error) PyErr_SetObject(type, error);
    Py_XDECREF(error);
    Py_XDECREF(type);
    Py_XDECREF(package);
    return nullptr;
}
#define RUN(name, ...)                                             \
    {                                                              \
        const int status = lib.name(__VA_ARGS__);                  \
        if (status == GSPN_ERR_CUDA) return raised("gspn_" #name, status); \
        NEED(status == GSPN_OK);                                   \
    }

typedef const Tensor* Opt;

// A plain tensor (or Parameter), or None.
bool get(PyObject* o, Opt& t) {
    if (o == Py_None) {
        t = nullptr;
        return true;
    }
    if (!THPVariable_CheckExact(o)) return false;
    t = &THPVariable_Unpack(o);
    return true;
}
bool all(PyObject* const* a, std::initializer_list<Opt*> to) {
    for (Opt* t : to)
        if (!get(*a++, *t)) return false;
    return true;
}

bool yes(PyObject* o) { return o == Py_True; }

// The call's device and storage type.
struct Ctx {
    int dev;
    ScalarType ty;
    bool start(Opt x) {
        if (!x || !x->is_cuda()) return false;
        dev = x->get_device();
        ty = x->scalar_type();
        return (ty == ScalarType::Float || ty == ScalarType::BFloat16) && dev == c10::cuda::current_device();
    }
    int code() const { return ty == ScalarType::Float ? GSPN_F32 : GSPN_BF16; }
    void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
    bool on(const Tensor& t, ScalarType type, at::IntArrayRef shape) const {
        return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.sizes() == shape;
    }
    bool is(Opt t, ScalarType type, at::IntArrayRef shape) const { return t && on(*t, type, shape) && t->is_contiguous(); }
    bool opt(Opt t, ScalarType type, at::IntArrayRef shape) const { return !t || is(t, type, shape); }
    bool f32(Opt t, at::IntArrayRef shape) const { return is(t, ScalarType::Float, shape); }
    bool opt_f32(Opt t, at::IntArrayRef shape) const { return opt(t, ScalarType::Float, shape); }
    // Strides of the leading `lead` axes (row, token); the axes behind them stand side by side.
    bool tokens(Opt t, at::IntArrayRef shape, int lead, long long& row, long long& tok) const {
        if (!t || !on(*t, ty, shape)) return false;
        int64_t inner = 1;
        for (int i = (int)shape.size() - 1; i >= lead; --i) {
            if (shape[i] != 1 && t->stride(i) != inner) return false;
            inner *= shape[i];
        }
        row = shape[0] > 1 ? t->stride(0) : 0;
        tok = lead > 1 && shape[1] > 1 ? t->stride(1) : 0;
        return true;
    }
    Tensor empty(at::IntArrayRef shape, ScalarType type) const {
        return Tensor(at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, (c10::DeviceIndex)dev), std::nullopt));
    }
};

void* ptr(Opt t) { return t ? t->data_ptr() : nullptr; }
template <typename T> T* as(Opt t) { return t ? (T*)t->data_ptr() : nullptr; }
bool fits_int(at::IntArrayRef s) {
    for (int64_t v : s)
        if (v > 0x7fffffff) return false;
    return true;
}
// Packed sequences: S for the descriptor, and how many sequences there are.
bool packed(const Ctx& c, Opt cu, const Tensor& x, int& S, int64_t& n) {
    S = 0;
    n = x.size(0);
    if (!cu) return true;
    if (cu->dim() != 1 || cu->size(0) < 2 || x.size(0) != 1 || !c.is(cu, ScalarType::Int, cu->sizes())) return false;
    n = cu->size(0) - 1;
    S = (int)n;
    return true;
}
// Tells autograd that the call wrote to tensors of the caller's through their pointers.
void wrote(std::initializer_list<Opt> ts) {
    for (Opt t : ts)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
PyObject* wrap(Tensor t) { return THPVariable_Wrap(std::move(t)); }

// A tensor to write to: the caller's, or a new one. `o` owns a new one.
struct Out {
    Tensor made;
    Opt t = nullptr;
    bool take(const Ctx& c, Opt given, bool wanted, ScalarType type, at::IntArrayRef shape) {
        if (given) {
            t = given;
            return c.is(given, type, shape);
        }
        if (wanted) {
            made = c.empty(shape, type);
            t = &made;
        }
        return true;
    }
    PyObject* object(PyObject* given) const {
        if (!t) Py_RETURN_NONE;
        if (!made.defined()) {
            Py_INCREF(given);
            return given;
        }
        return wrap(made);
    }
};
PyObject* tuple(std::initializer_list<PyObject*> items) {
    PyObject* r = PyTuple_New((Py_ssize_t)items.size());
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

// ------------------------------------------------------------------------------- convolution
bool conv_desc(const Ctx& c, Opt x, Opt w, Opt bias, bool silu, Opt cu, gspn_conv_desc& d, int64_t& n) {
    if (x->dim() != 3 || !w || w->dim() != 2 || !fits_int(x->sizes())) return false;
    const int64_t C = x->size(2), K = w->size(1);
    if (!c.f32(w, {C, K}) || !c.opt_f32(bias, {C})) return false;
    d = gspn_conv_desc{(int)x->size(0), (int)x->size(1), (int)C, (int)K, 0, c.code(), silu, 0, 0};
    return packed(c, cu, *x, d.S, n) && c.tokens(x, x->sizes(), 2, d.x_row, d.x_tok);
}

// x, w, bias, cu, state0, y, state, silu
PyObject* conv_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, w, bias, cu, state0, y, state;
    NEED(all(a, {&x, &w, &bias, &cu, &state0, &y, &state}));
    Ctx c;
    NEED(c.start(x));
    gspn_conv_desc d;
    int64_t n;
    NEED(conv_desc(c, x, w, bias, yes(a[7]), cu, d, n));
    NEED(c.opt(state0, c.ty, {n, d.K - 1, d.C}) && c.opt(state, c.ty, {n, d.K - 1, d.C}));
    Out o;
    NEED(o.take(c, y, true, c.ty, x->sizes()));
    RUN(conv_forward, &d, ptr(x), as<float>(w), as<float>(bias), as<int>(cu), ptr(state0), ptr(o.t), ptr(state),
                          c.stream());
    wrote({y, state});
    return o.object(a[5]);
}

// x, w, bias, cu, state0, dy, dstate, silu
PyObject* conv_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, w, bias, cu, state0, dy, dstate;
    NEED(all(a, {&x, &w, &bias, &cu, &state0, &dy, &dstate}));
    Ctx c;
    NEED(c.start(x));
    gspn_conv_desc d;
    int64_t n;
    NEED(conv_desc(c, x, w, bias, yes(a[7]), cu, d, n));
    const int64_t ss[3] = {n, d.K - 1, d.C};
    NEED(c.is(dy, c.ty, x->sizes()) && c.opt(state0, c.ty, ss) && c.opt(dstate, c.ty, ss));
    const size_t bytes = lib.conv_ws(&d, 1);
    NEED(bytes > 0);
    const Tensor ws = c.empty({(int64_t)bytes}, ScalarType::Byte);
    Out dx, dw, db, ds;
    NEED(dx.take(c, nullptr, true, c.ty, x->sizes()) && dw.take(c, nullptr, true, ScalarType::Float, w->sizes()) &&
         db.take(c, nullptr, bias, ScalarType::Float, {d.C}) && ds.take(c, nullptr, state0, c.ty, ss));
    RUN(conv_backward, &d, ptr(x), as<float>(w), as<float>(bias), as<int>(cu), ptr(state0), ptr(dy), ptr(dstate),
                           ptr(dx.t), as<float>(dw.t), as<float>(db.t), ptr(ds.t), ws.data_ptr(), bytes,
                           c.stream());
    return tuple({dx.object(nullptr), dw.object(nullptr), db.object(nullptr), ds.object(nullptr)});
}

bool slots_ok(const Ctx& c, Opt idx, Opt state, int64_t rows) {
    return idx ? c.is(idx, ScalarType::Int, {rows}) : state->size(0) >= rows;
}

// x, w, bias, state, idx, y, silu
PyObject* conv_step(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, w, bias, state, idx, y;
    NEED(all(a, {&x, &w, &bias, &state, &idx, &y}));
    Ctx c;
    NEED(c.start(x) && x->dim() == 2 && w && w->dim() == 2 && state && state->dim() == 3 && fits_int(state->sizes()) &&
         fits_int(x->sizes()));
    const int64_t B = x->size(0), C = x->size(1), K = w->size(1);
    NEED(c.f32(w, {C, K}) && c.opt_f32(bias, {C}) && c.is(state, c.ty, {state->size(0), K - 1, C}) && slots_ok(c, idx, state, B));
    gspn_conv_desc d{(int)B, 1, (int)C, (int)K, 0, c.code(), yes(a[6]), 0, 0};
    NEED(c.tokens(x, x->sizes(), 1, d.x_row, d.x_tok));
    Out o;
    NEED(o.take(c, y, true, c.ty, x->sizes()));
    RUN(conv_step, &d, ptr(x), as<float>(w), as<float>(bias), as<int>(idx), (int)state->size(0), ptr(state), ptr(o.t),
                       c.stream());
    wrote({state, y});
    return o.object(a[5]);
}

// ------------------------------------------------------------------------------ selective scan
bool ssm_desc(const Ctx& c, Opt x, Opt dt, Opt A, Opt B, Opt C, Opt D, Opt z, Opt bias, bool softplus, Opt cu,
              gspn_ssm_desc& d, int64_t& n) {
    if (x->dim() != 3 || !B || B->dim() != 4 || !fits_int(x->sizes()) || !fits_int(B->sizes())) return false;
    const int64_t Ch = x->size(2), G = B->size(2), N = B->size(3);
    if (G < 1 || Ch % G != 0 || !c.f32(A, {Ch, N}) || !c.opt_f32(D, {Ch}) || !c.opt_f32(bias, {Ch})) return false;
    d = gspn_ssm_desc{};
    d.B = (int)x->size(0);
    d.L = (int)x->size(1);
    d.C = (int)Ch;
    d.G = (int)G;
    d.N = (int)N;
    d.dtype = c.code();
    d.softplus = softplus;
    const int64_t bc[4] = {d.B, d.L, G, N};
    return packed(c, cu, *x, d.S, n) && c.tokens(x, x->sizes(), 2, d.x_row, d.x_tok) &&
           c.tokens(dt, x->sizes(), 2, d.dt_row, d.dt_tok) && (!z || c.tokens(z, x->sizes(), 2, d.z_row, d.z_tok)) &&
           c.tokens(B, bc, 2, d.b_row, d.b_tok) && c.tokens(C, bc, 2, d.c_row, d.c_tok);
}

// x, dt, A, B, C, D, z, dt_bias, cu, h0, y, h, softplus, save: y, or (y, hsave)
PyObject* ssm_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, dt, A, B, C, D, z, bias, cu, h0, y, h;
    NEED(all(a, {&x, &dt, &A, &B, &C, &D, &z, &bias, &cu, &h0, &y, &h}));
    Ctx c;
    NEED(c.start(x) && PyBool_Check(a[12]));
    gspn_ssm_desc d;
    int64_t n;
    NEED(ssm_desc(c, x, dt, A, B, C, D, z, bias, yes(a[12]), cu, d, n));
    NEED(c.opt_f32(h0, {n, d.C, d.N}) && c.opt_f32(h, {n, d.C, d.N}));
    Out o;
    NEED(o.take(c, y, true, c.ty, x->sizes()));
    const bool save = yes(a[13]);
    Tensor hsave, ws;
    if (save) {
        const size_t bytes = lib.ssm_hsave(&d);
        NEED(bytes > 0);
        hsave = c.empty({(int64_t)bytes / 4}, ScalarType::Float);
    }
    const size_t bytes = lib.ssm_ws(&d, 0);
    NEED(bytes > 0);
    if (bytes > 256) ws = c.empty({(int64_t)bytes}, ScalarType::Byte);
    RUN(ssm_forward, &d, ptr(x), ptr(dt), as<float>(A), ptr(B), ptr(C), as<float>(D), ptr(z), as<float>(bias), as<int>(cu),
                         as<float>(h0), ptr(o.t), as<float>(h), save ? (float*)hsave.data_ptr() : nullptr,
                         bytes > 256 ? ws.data_ptr() : nullptr, bytes, c.stream());
    wrote({y, h});
    if (!save) return o.object(a[10]);
    return tuple({o.object(a[10]), wrap(hsave)});
}

// x, dt, A, B, C, dy, hsave, D, z, dt_bias, cu, h0, dh, softplus
PyObject* ssm_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, dt, A, B, C, dy, hsave, D, z, bias, cu, h0, dh;
    NEED(all(a, {&x, &dt, &A, &B, &C, &dy, &hsave, &D, &z, &bias, &cu, &h0, &dh}));
    Ctx c;
    NEED(c.start(x));
    gspn_ssm_desc d;
    int64_t n;
    NEED(ssm_desc(c, x, dt, A, B, C, D, z, bias, yes(a[13]), cu, d, n));
    const int64_t ss[3] = {n, d.C, d.N};
    NEED(c.is(dy, c.ty, x->sizes()) && c.opt_f32(h0, ss) && c.opt_f32(dh, ss) &&
         c.f32(hsave, {(int64_t)lib.ssm_hsave(&d) / 4}));
    const size_t bytes = lib.ssm_ws(&d, 1);
    NEED(bytes > 0);
    const Tensor ws = c.empty({(int64_t)bytes}, ScalarType::Byte);
    const ScalarType f = ScalarType::Float;
    Out dx, ddt, dA, dB, dC, dD, dz, dbias, dh0;
    NEED(dx.take(c, nullptr, true, c.ty, x->sizes()) && ddt.take(c, nullptr, true, c.ty, x->sizes()) &&
         dA.take(c, nullptr, true, f, A->sizes()) && dB.take(c, nullptr, true, c.ty, B->sizes()) &&
         dC.take(c, nullptr, true, c.ty, B->sizes()) && dD.take(c, nullptr, D, f, {d.C}) &&
         dz.take(c, nullptr, z, c.ty, x->sizes()) && dbias.take(c, nullptr, bias, f, {d.C}) && dh0.take(c, nullptr, h0, f, ss));
    RUN(ssm_backward, &d, ptr(x), ptr(dt), as<float>(A), ptr(B), ptr(C), as<float>(D), ptr(z), as<float>(bias), as<int>(cu),
                          as<float>(hsave), ptr(dy), as<float>(dh), ptr(dx.t), ptr(ddt.t), as<float>(dA.t), ptr(dB.t), ptr(dC.t),
                          as<float>(dD.t), ptr(dz.t), as<float>(dbias.t), as<float>(dh0.t), ws.data_ptr(), bytes,
                          c.stream());
    return tuple({dx.object(nullptr), ddt.object(nullptr), dA.object(nullptr), dB.object(nullptr), dC.object(nullptr),
                  dD.object(nullptr), dz.object(nullptr), dbias.object(nullptr), dh0.object(nullptr)});
}

// x, dt, A, B, C, h, D, z, dt_bias, idx, y, softplus
PyObject* ssm_step(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt x, dt, A, B, C, h, D, z, bias, idx, y;
    NEED(all(a, {&x, &dt, &A, &B, &C, &h, &D, &z, &bias, &idx, &y}));
    Ctx c;
    NEED(c.start(x) && x->dim() == 2 && B && B->dim() == 3 && h && h->dim() == 3 && fits_int(h->sizes()) && fits_int(x->sizes()) &&
         fits_int(B->sizes()));
    const int64_t R = x->size(0), Ch = x->size(1), G = B->size(1), N = B->size(2);
    NEED(G >= 1 && Ch % G == 0 && c.f32(A, {Ch, N}) && c.opt_f32(D, {Ch}) && c.opt_f32(bias, {Ch}) &&
         c.f32(h, {h->size(0), Ch, N}) && slots_ok(c, idx, h, R));
    gspn_ssm_desc d{};
    d.B = (int)R;
    d.L = 1;
    d.C = (int)Ch;
    d.G = (int)G;
    d.N = (int)N;
    d.dtype = c.code();
    d.softplus = yes(a[11]);
    long long none;
    NEED(c.tokens(x, x->sizes(), 1, d.x_row, none) && c.tokens(dt, x->sizes(), 1, d.dt_row, none) &&
         (!z || c.tokens(z, x->sizes(), 1, d.z_row, none)) && c.tokens(B, {R, G, N}, 1, d.b_row, none) &&
         c.tokens(C, {R, G, N}, 1, d.c_row, none));
    Out o;
    NEED(o.take(c, y, true, c.ty, x->sizes()));
    RUN(ssm_step, &d, ptr(x), ptr(dt), as<float>(A), ptr(B), ptr(C), as<float>(D), ptr(z), as<float>(bias), as<int>(idx),
                      (int)h->size(0), as<float>(h), ptr(o.t), c.stream());
    wrote({h, y});
    return o.object(a[10]);
}

// ------------------------------------------------------------------------- norms around a block
// Stride between the rows of a contiguous (..., C) tensor, or of a 2-d one.
bool rows_of(const Ctx& c, Opt t, ScalarType type, at::IntArrayRef shape, long long& row) {
    row = 0;
    if (!t) return true;
    if (!c.on(*t, type, shape)) return false;
    const int64_t C = shape.back();
    if (t->is_contiguous()) {
        row = C;
        return true;
    }
    if (shape.size() != 2 || (C != 1 && t->stride(1) != 1)) return false;
    row = shape[0] > 1 ? t->stride(0) : C;
    return true;
}
bool norm_desc(const Ctx& c, Opt y, Opt gate, Opt wp, Opt bp, Opt scale, Opt r, Opt w, Opt b, ScalarType res, PyObject* eps,
               bool center, gspn_norm_desc& d) {
    if (y->dim() < 1 || !fits_int(y->sizes())) return false;
    const int64_t C = y->sizes().back();
    for (Opt t : {wp, bp, scale, w, b})
        if (!c.opt_f32(t, {C})) return false;
    if ((bp && !wp) || (b && !w) || C < 1) return false;
    const int64_t rows = y->numel() / C;
    if (rows > 0x7fffffff || (res != ScalarType::Float && res != c.ty)) return false;
    const double e = PyFloat_AsDouble(eps);
    if (e == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        return false;
    }
    d = gspn_norm_desc{(int)rows, (int)C, c.code(), res == ScalarType::Float ? GSPN_F32 : GSPN_BF16, center, (float)e, 0, 0, 0};
    return rows_of(c, y, c.ty, y->sizes(), d.y_row) && rows_of(c, gate, c.ty, y->sizes(), d.gate_row) &&
           rows_of(c, r, res, y->sizes(), d.r_row);
}

// y, r, gate, w_post, b_post, scale, w_pre, b_pre, r_out, o, eps, center
PyObject* norm_forward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt y, r, gate, wp, bp, scale, w, b, r_out, o;
    NEED(all(a, {&y, &r, &gate, &wp, &bp, &scale, &w, &b, &r_out, &o}));
    Ctx c;
    NEED(c.start(y));
    const ScalarType res = r ? r->scalar_type() : c.ty;
    gspn_norm_desc d;
    NEED(norm_desc(c, y, gate, wp, bp, scale, r, w, b, res, a[10], yes(a[11]), d));
    Out s, q;
    NEED(s.take(c, r_out, true, res, y->sizes()) && q.take(c, w ? o : nullptr, w, c.ty, y->sizes()));
    RUN(norm_forward, &d, ptr(y), ptr(gate), as<float>(wp), as<float>(bp), as<float>(scale), ptr(r), as<float>(w), as<float>(b),
                          ptr(s.t), ptr(q.t), c.stream());
    wrote({r_out, w ? o : nullptr});
    return tuple({s.object(a[8]), q.object(a[9])});
}

// y, r_out, dr, do, gate, w_post, b_post, scale, w_pre, b_pre, eps, center
PyObject* norm_backward(PyObject*, PyObject* const* a, Py_ssize_t) {
    Opt y, r, dr, go, gate, wp, bp, scale, w, b;
    NEED(all(a, {&y, &r, &dr, &go, &gate, &wp, &bp, &scale, &w, &b}));
    Ctx c;
    NEED(c.start(y) && (w != nullptr) == (go != nullptr) && (r || dr) && (r || !w));
    const ScalarType res = r ? r->scalar_type() : dr->scalar_type();
    gspn_norm_desc d;
    NEED(norm_desc(c, y, gate, wp, bp, scale, r, w, b, res, a[10], yes(a[11]), d));
    NEED(c.opt(dr, res, y->sizes()) && c.opt(go, c.ty, y->sizes()));
    const size_t bytes = lib.norm_ws(&d, 1);
    NEED(bytes > 0);
    const Tensor ws = c.empty({(int64_t)bytes}, ScalarType::Byte);
    const ScalarType f = ScalarType::Float;
    const int64_t cs[1] = {d.C};
    Out dy, dri, dg, dwp, dbp, ds, dw, db;
    NEED(dy.take(c, nullptr, true, c.ty, y->sizes()) && dri.take(c, nullptr, true, res, y->sizes()) &&
         dg.take(c, nullptr, gate, c.ty, y->sizes()) && dwp.take(c, nullptr, wp, f, cs) && dbp.take(c, nullptr, bp, f, cs) &&
         ds.take(c, nullptr, scale, f, cs) && dw.take(c, nullptr, w, f, cs) && db.take(c, nullptr, b, f, cs));
    RUN(norm_backward, &d, ptr(y), ptr(gate), as<float>(wp), as<float>(bp), as<float>(scale), ptr(r), as<float>(w), ptr(dr),
                           ptr(go), ptr(dy.t), ptr(dri.t), ptr(dg.t), as<float>(dwp.t), as<float>(dbp.t), as<float>(ds.t),
                           as<float>(dw.t), as<float>(db.t), ws.data_ptr(), bytes, c.stream());
    return tuple({dy.object(nullptr), dri.object(nullptr), dg.object(nullptr), dwp.object(nullptr), dbp.object(nullptr),
                  ds.object(nullptr), dw.object(nullptr), db.object(nullptr)});
}

// A C++ exception (an allocation that fails, say) must not leave through the interpreter's C frames: the
// call is declined, and the Python path raises what it meets.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t), int ARGS>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    if (n != ARGS) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    if (!PyBool_Check(a[ARGS - 1])) DECLINE;                      // other truths may fail to be one
    try {
        return F(self, a, n);
    } catch (...) {
        Py_RETURN_NONE;
    }
}

PyObject* init(PyObject*, PyObject* addresses) {
    static const char* const names[] = {
        "gspn_conv_workspace_size", "gspn_conv_forward", "gspn_conv_backward", "gspn_conv_step",
        "gspn_ssm_workspace_size", "gspn_ssm_hsave_size", "gspn_ssm_forward", "gspn_ssm_backward", "gspn_ssm_step",
        "gspn_norm_workspace_size", "gspn_norm_forward", "gspn_norm_backward"};
    void** to = (void**)&lib;
    static_assert(sizeof(lib) == sizeof(names) / sizeof(names[0]) * sizeof(void*), "one name for each entry point");
    for (const char* n : names) {
        PyObject* v = PyDict_GetItemString(addresses, n);
        *to = v ? PyLong_AsVoidPtr(v) : nullptr;
        if (!*to++) {
            PyErr_Format(PyExc_ValueError, "no address for %s", n);
            return nullptr;
        }
    }
    Py_RETURN_NONE;
}

#define FN(name, args) {#name, (PyCFunction)(void*)guarded<name, args>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(conv_forward, 8), FN(conv_backward, 8), FN(conv_step, 7), FN(ssm_forward, 14), FN(ssm_backward, 14),
                         FN(ssm_step, 12), FN(norm_forward, 12), FN(norm_backward, 12), {"init", init, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_seq_fast", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__seq_fast() { return PyModule_Create(&module); }
