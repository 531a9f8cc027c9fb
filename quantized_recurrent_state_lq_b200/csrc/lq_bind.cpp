// lq_bind.cpp -- native half of lq.py's calls for the recurrent layer: checks of
// the tensors (device, type, shape, evenly spaced rows), allocation of what was
// not given, and the call of the C ABI on torch's current stream.  A decode
// step's operators take the GPU a few microseconds each, so an eager caller
// waits for the host: checked here a call takes about 5 us, in Python with a
// foreign call of 12 to 17 arguments 13 to 17.
//
// Arguments are positional, in the order of lq.py's functions without stream.
// A call returns its tensors, or the library's error code as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <string>

#include "lq_state.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;
using Shape = c10::SmallVector<int64_t, 6>;

// liblq.so's entry points, set once by load().
struct Api {
    decltype(&lq_conv_prefill) conv_prefill;
    decltype(&lq_conv_step) conv_step;
    decltype(&lq_ssm_workspace_bytes) ssm_workspace_bytes;
    decltype(&lq_ssm_prefill) ssm_prefill;
    decltype(&lq_ssm_step) ssm_step;
    decltype(&lq_norm_in) norm_in;
    decltype(&lq_norm_out) norm_out;
} api;

struct Refusal {};   // the Python error is set

[[noreturn]] void refuse(PyObject *type, const char *format, ...) {
    va_list v;
    va_start(v, format);
    PyErr_FormatV(type, format, v);
    va_end(v);
    throw Refusal{};
}

std::string str(IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}

const char *type_name(ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kDouble: return "torch.float64";
        case at::kInt: return "torch.int32";
        case at::kLong: return "torch.int64";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

int type_code(ScalarType t) {
    if (t == at::kFloat) return LQ_F32;
    if (t == at::kBFloat16) return LQ_BF16;
    if (t == at::kHalf) return LQ_F16;
    refuse(PyExc_TypeError, "activations must be float32, bfloat16 or float16, got %s", type_name(t));
}

int act_code(PyObject *o) {
    if (o == Py_None) return LQ_ACT_NONE;
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return LQ_ACT_SILU;
        if (PyUnicode_CompareWithASCIIString(o, "sigmoid") == 0) return LQ_ACT_SIGMOID;
    }
    refuse(PyExc_ValueError, "unknown activation %R", o);
}

bool truth(PyObject *o) {
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Refusal{};
    return t != 0;
}

double number(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refusal{};
    return v;
}

int32_t i32(int64_t v) {
    if (v > INT32_MAX) refuse(PyExc_ValueError, "size %lld is too large", (long long)v);
    return (int32_t)v;
}

// The first argument of a call, whose device is the call's.
const Tensor &first(PyObject *o, const char *call) {
    if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(PyExc_TypeError, "%s takes CUDA tensors", call);
    return THPVariable_Unpack(o);
}

// The call's device, made current while it differs.
struct Device {
    int id;
    c10::cuda::OptionalCUDAGuard guard;

    explicit Device(const Tensor &x) : id(x.get_device()) {
        if (id != c10::cuda::current_device()) guard.set_index((c10::DeviceIndex)id);
    }
    void *stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)id).stream(); }
};

const Tensor &tensor(PyObject *o, const char *name, int dev) {
    if (!THPVariable_Check(o) || THPVariable_Unpack(o).get_device() != dev)
        refuse(PyExc_TypeError, "%s must be a CUDA tensor on device %d", name, dev);
    return THPVariable_Unpack(o);
}

void check(const Tensor &t, const char *name, IntArrayRef shape, ScalarType type) {
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, str(t.sizes()).c_str(), str(shape).c_str());
}

// A tensor of token rows: its last n_tail dimensions are one contiguous row of
// `width` elements, the others evenly spaced rows.
struct Rows {
    void *p = nullptr;
    int64_t ld = 0;
};
Rows rows(const Tensor &t, const char *name, IntArrayRef shape, int n_tail, int64_t width, ScalarType type) {
    check(t, name, shape, type);
    if (t.is_contiguous()) return {t.data_ptr(), width};
    const IntArrayRef st = t.strides();
    const int n = (int)st.size();
    int64_t w = 1;
    for (int i = n - 1; i >= n - n_tail; --i)
        if (shape[i] != 1) {
            if (st[i] != w) refuse(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
            w *= shape[i];
        }
    int64_t ld = width, count = 1;
    for (int i = n - n_tail - 1; i >= 0; --i)
        if (shape[i] != 1) {
            if (count == 1) ld = st[i];
            else if (st[i] != count * ld) refuse(PyExc_ValueError, "%s: rows must be evenly spaced", name);
            count *= shape[i];
        }
    return {t.data_ptr(), ld};
}
Rows rows(PyObject *o, const char *name, IntArrayRef shape, int n_tail, int64_t width, ScalarType type, int dev) {
    return rows(tensor(o, name, dev), name, shape, n_tail, width, type);
}
Rows rows_or_none(PyObject *o, const char *name, IntArrayRef shape, int n_tail, int64_t width, ScalarType type, int dev) {
    return o == Py_None ? Rows{} : rows(o, name, shape, n_tail, width, type, dev);
}

// A contiguous tensor (flat: or None).
template <typename T = float>
T *given(PyObject *o, const char *name, IntArrayRef shape, int dev, ScalarType type = at::kFloat) {
    const Tensor &t = tensor(o, name, dev);
    check(t, name, shape, type);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    return static_cast<T *>(t.data_ptr());
}
template <typename T = float>
T *flat(PyObject *o, const char *name, IntArrayRef shape, int dev, ScalarType type = at::kFloat) {
    return o == Py_None ? nullptr : given<T>(o, name, shape, dev, type);
}

// An output: the given tensor or a new one of the first argument's device.
struct Out {
    PyObject *o;

    Out(PyObject *given, const Tensor &like, IntArrayRef shape, ScalarType type)
        : o(given == Py_None ? THPVariable_Wrap(at::empty(shape, like.options().dtype(type).requires_grad(false)))
                             : Py_NewRef(given)) {
        if (!o) throw Refusal{};
    }
    Out(const Out &) = delete;
    ~Out() { Py_XDECREF(o); }
    PyObject *release() {
        PyObject *r = o;
        o = nullptr;
        return r;
    }
};

PyObject *result(int rc, Out &y) { return rc == LQ_OK ? y.release() : PyLong_FromLong(rc); }
PyObject *result(int rc, Out &y, Out &s) { return rc == LQ_OK ? PyTuple_Pack(2, y.o, s.o) : PyLong_FromLong(rc); }

// Sequences, rows and offsets of a packed or time-major prompt batch.
struct Prompt {
    int32_t B, rows;
    const int32_t *cu;
};
Prompt prompt(const Tensor &x, PyObject *cu, int n_tail, int dev) {
    const int64_t lead = x.dim() - n_tail;
    if (cu == Py_None) {
        if (lead != 2)
            refuse(PyExc_ValueError, "a time-major prompt is [T, B, ...], got %s; a packed one needs cu",
                   str(x.sizes()).c_str());
        return {i32(x.size(1)), i32(x.size(0) * x.size(1)), nullptr};
    }
    if (lead != 1) refuse(PyExc_ValueError, "a packed prompt is [rows, ...], got %s", str(x.sizes()).c_str());
    const Tensor &c = tensor(cu, "cu", dev);
    if (c.dim() != 1 || c.size(0) < 2) refuse(PyExc_ValueError, "cu must hold B+1 offsets");
    return {i32(c.size(0) - 1), i32(x.size(0)), flat<int32_t>(cu, "cu", c.sizes(), dev, at::kInt)};
}

// Taps [C, K].
void taps(PyObject *o, int dev, int64_t &ch, int64_t &K) {
    const Tensor &w = tensor(o, "w", dev);
    if (w.dim() != 2) refuse(PyExc_ValueError, "w is [C, K], got %s", str(w.sizes()).c_str());
    ch = w.size(0);
    K = w.size(1);
}

// Groups and key rows of Bm [..., G, dk].
void groups(PyObject *o, int dev, int64_t &G, int64_t &dk) {
    const Tensor &b = tensor(o, "Bm", dev);
    if (b.dim() < 2) refuse(PyExc_ValueError, "Bm is [..., G, dk], got %s", str(b.sizes()).c_str());
    G = b.size(-2);
    dk = b.size(-1);
}

Shape shape_of(IntArrayRef lead, std::initializer_list<int64_t> tail) {
    Shape s(lead.begin(), lead.end());
    s.append(tail.begin(), tail.end());
    return s;
}

// x, w, bias, act, state0, state_out, y, cu
PyObject *conv_prefill(PyObject *const *a) {
    const Tensor &x = first(a[0], "lq_conv_prefill");
    const Device dev(x);
    const ScalarType t = x.scalar_type();
    const int code = type_code(t);
    const Prompt pr = prompt(x, a[7], 1, dev.id);
    int64_t ch, K;
    taps(a[1], dev.id, ch, K);
    const Shape sx = shape_of(x.sizes().slice(0, x.dim() - 1), {ch}), sw{pr.B, K - 1, ch};
    const Rows px = rows(x, "x", sx, 1, ch, t);
    const float *w = flat(a[1], "w", {ch, K}, dev.id), *bias = flat(a[2], "bias", {ch}, dev.id);
    const lq_conv_config cfg{code, pr.B, i32(ch), i32(K), act_code(a[3])};
    const void *s0 = flat<void>(a[4], "state0", sw, dev.id, t);
    if (K < 1) refuse(PyExc_ValueError, "w has no taps");
    Out y(a[6], x, sx, t), so(a[5], x, sw, t);
    const Rows py = rows(y.o, "y", sx, 1, ch, t, dev.id);
    void *s1 = flat<void>(so.o, "state_out", sw, dev.id, t);
    return result(api.conv_prefill(&cfg, pr.rows, pr.cu, px.p, px.ld, w, bias, s0, s1, py.p, py.ld, dev.stream()), y, so);
}

// state, x, w, bias, act, y
PyObject *conv_step(PyObject *const *a) {
    const Tensor &s = first(a[0], "lq_conv_step");
    const Device dev(s);
    const Tensor &x = tensor(a[1], "x", dev.id);
    const ScalarType t = x.scalar_type();
    const int code = type_code(t);
    int64_t ch, K;
    taps(a[2], dev.id, ch, K);
    if (x.dim() != 2) refuse(PyExc_ValueError, "x is [B, C], got %s", str(x.sizes()).c_str());
    const int64_t B = x.size(0);
    const Rows px = rows(x, "x", {B, ch}, 1, ch, t);
    const float *w = flat(a[2], "w", {ch, K}, dev.id), *bias = flat(a[3], "bias", {ch}, dev.id);
    const lq_conv_config cfg{code, i32(B), i32(ch), i32(K), act_code(a[4])};
    void *ps = flat<void>(a[0], "state", {B, K - 1, ch}, dev.id, t);
    Out y(a[5], x, {B, ch}, t);
    const Rows py = rows(y.o, "y", {B, ch}, 1, ch, t, dev.id);
    return result(api.conv_step(&cfg, ps, px.p, px.ld, w, bias, py.p, py.ld, dev.stream()), y);
}

// x, dt, A, Bm, Cm, D, dt_bias, softplus, S0, S_out, y, cu, workspace
PyObject *ssm_prefill(PyObject *const *a) {
    const Tensor &x = first(a[0], "lq_ssm_prefill");
    const Device dev(x);
    const ScalarType t = x.scalar_type();
    const int code = type_code(t);
    const Prompt pr = prompt(x, a[11], 2, dev.id);
    int64_t G, dk;
    groups(a[3], dev.id, G, dk);
    const IntArrayRef lead = x.sizes().slice(0, x.dim() - 2);
    const int64_t H = x.size(-2), dv = x.size(-1);
    const Shape sx = shape_of(lead, {H, dv}), sb = shape_of(lead, {G, dk}), sd = shape_of(lead, {H});
    const Shape st{pr.B, H, dk, dv};
    const Rows px = rows(x, "x", sx, 2, H * dv, t), pd = rows(a[1], "dt", sd, 1, H, t, dev.id);
    const Rows pb = rows(a[3], "Bm", sb, 2, G * dk, t, dev.id), pc = rows(a[4], "Cm", sb, 2, G * dk, t, dev.id);
    const float *A = given(a[2], "A", {H}, dev.id), *D = flat(a[5], "D", {H}, dev.id);
    const float *bias = flat(a[6], "dt_bias", {H}, dev.id), *S0 = flat(a[8], "S0", st, dev.id);
    const lq_ssm_config cfg{code, pr.B, i32(H), i32(G), i32(dk), i32(dv), truth(a[7]) ? 1 : 0};
    Out y(a[10], x, sx, t), So(a[9], x, st, at::kFloat);
    const Rows py = rows(y.o, "y", sx, 2, H * dv, t, dev.id);
    float *S1 = flat(So.o, "S_out", st, dev.id);
    size_t n_ws = api.ssm_workspace_bytes(&cfg, pr.rows);
    void *ws = nullptr;
    Tensor own;
    if (a[12] != Py_None) {
        const Tensor &w = tensor(a[12], "workspace", dev.id);
        n_ws = (size_t)w.numel();
        ws = flat<void>(a[12], "workspace", {w.numel()}, dev.id, at::kByte);
    } else if (n_ws) {
        own = at::empty({(int64_t)n_ws}, x.options().dtype(at::kByte).requires_grad(false));
        ws = own.data_ptr();
    }
    return result(api.ssm_prefill(&cfg, pr.rows, pr.cu, px.p, px.ld, pd.p, pd.ld, A, pb.p, pb.ld, pc.p, pc.ld, D, bias,
                                  S0, S1, py.p, py.ld, ws, n_ws, dev.stream()),
                  y, So);
}

// S, x, dt, A, Bm, Cm, D, dt_bias, softplus, y
PyObject *ssm_step(PyObject *const *a) {
    const Tensor &s = first(a[0], "lq_ssm_step");
    const Device dev(s);
    const Tensor &x = tensor(a[1], "x", dev.id);
    const ScalarType t = x.scalar_type();
    const int code = type_code(t);
    if (x.dim() != 3) refuse(PyExc_ValueError, "x is [B, H, dv], got %s", str(x.sizes()).c_str());
    const int64_t B = x.size(0), H = x.size(1), dv = x.size(2);
    int64_t G, dk;
    groups(a[4], dev.id, G, dk);
    const Rows px = rows(x, "x", {B, H, dv}, 2, H * dv, t), pd = rows(a[2], "dt", {B, H}, 1, H, t, dev.id);
    const Rows pb = rows(a[4], "Bm", {B, G, dk}, 2, G * dk, t, dev.id);
    const Rows pc = rows(a[5], "Cm", {B, G, dk}, 2, G * dk, t, dev.id);
    const float *A = given(a[3], "A", {H}, dev.id), *D = flat(a[6], "D", {H}, dev.id);
    const float *bias = flat(a[7], "dt_bias", {H}, dev.id);
    float *S = flat(a[0], "S", {B, H, dk, dv}, dev.id);
    const lq_ssm_config cfg{code, i32(B), i32(H), i32(G), i32(dk), i32(dv), truth(a[8]) ? 1 : 0};
    Out y(a[9], x, {B, H, dv}, t);
    const Rows py = rows(y.o, "y", {B, H, dv}, 2, H * dv, t, dev.id);
    return result(api.ssm_step(&cfg, S, px.p, px.ld, pd.p, pd.ld, A, pb.p, pb.ld, pc.p, pc.ld, D, bias, py.p, py.ld,
                               dev.stream()),
                  y);
}

// The residual scale: a number, or a float32 tensor.
const float *scale_of(PyObject *o, IntArrayRef shape, int dev, float &factor) {
    if (THPVariable_Check(o)) {
        factor = 1.0f;
        return flat(o, "scale", shape, dev);
    }
    factor = (float)number(o);
    return nullptr;
}

// x, w, res, scale, eps, h, y
PyObject *norm_in(PyObject *const *a) {
    const Tensor &x = first(a[0], "lq_norm_in");
    const Device dev(x);
    const ScalarType t = x.scalar_type();
    const int code = type_code(t);
    if (x.dim() < 1) refuse(PyExc_ValueError, "x is [..., D], got ()");
    const IntArrayRef sx = x.sizes();
    const int64_t D = x.size(-1);
    const Rows px = rows(x, "x", sx, 1, D, t), pr = rows_or_none(a[2], "res", sx, 1, D, t, dev.id);
    float factor;
    const float *w = given(a[1], "w", {D}, dev.id), *ps = scale_of(a[3], {D}, dev.id, factor);
    const lq_norm_config cfg{code, code, i32(x.numel() / std::max<int64_t>(D, 1)), 1, i32(D), 0, 0, 0,
                             (float)number(a[4]), factor};
    Out h(a[5], x, sx, t), y(a[6], x, sx, t);
    const Rows ph = rows(h.o, "h", sx, 1, D, t, dev.id), py = rows(y.o, "y", sx, 1, D, t, dev.id);
    return result(api.norm_in(&cfg, px.p, px.ld, w, pr.p, pr.ld, ps, ph.p, ph.ld, py.p, py.ld, dev.stream()), y, h);
}

// x, w, z, act, gate_first, res, scale, eps, y
PyObject *norm_out(PyObject *const *a) {
    const Tensor &x = first(a[0], "lq_norm_out");
    const Device dev(x);
    if (x.dim() < 2) refuse(PyExc_ValueError, "x is [..., G, D], got %s", str(x.sizes()).c_str());
    ScalarType t = x.scalar_type();
    for (const int i : {8, 2, 5})   // the type of a given y, z or res, else x's
        if (a[i] != Py_None) {
            t = tensor(a[i], i == 8 ? "y" : i == 2 ? "z" : "res", dev.id).scalar_type();
            break;
        }
    const int xcode = type_code(x.scalar_type()), code = type_code(t);
    const IntArrayRef sx = x.sizes();
    const int64_t G = x.size(-2), D = x.size(-1), n = G * D;
    const Rows px = rows(x, "x", sx, 2, n, x.scalar_type()), pz = rows_or_none(a[2], "z", sx, 2, n, t, dev.id);
    const Rows pr = rows_or_none(a[5], "res", sx, 2, n, t, dev.id);
    const bool wg = tensor(a[1], "w", dev.id).dim() == 2;
    const float *w = wg ? flat(a[1], "w", {G, D}, dev.id) : flat(a[1], "w", {D}, dev.id);
    float factor;
    const float *ps = scale_of(a[6], {G, D}, dev.id, factor);
    const lq_norm_config cfg{code, xcode, i32(x.numel() / std::max<int64_t>(n, 1)), i32(G), i32(D), wg ? 1 : 0,
                             act_code(a[3]), truth(a[4]) ? 1 : 0, (float)number(a[7]), factor};
    Out y(a[8], x, sx, t);
    const Rows py = rows(y.o, "y", sx, 2, n, t, dev.id);
    return result(api.norm_out(&cfg, px.p, px.ld, w, pz.p, pz.ld, pr.p, pr.ld, ps, py.p, py.ld, dev.stream()), y);
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The addresses of the C ABI's functions, in the order of Api.
PyObject *load(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void *p[sizeof(Api) / sizeof(void *)];
    if (n != (Py_ssize_t)(sizeof(p) / sizeof(p[0]))) {
        PyErr_SetString(PyExc_TypeError, "takes one address for each entry point");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        p[i] = PyLong_AsVoidPtr(args[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
            return nullptr;
        }
    }
    static_assert(sizeof(p) == sizeof(Api), "one pointer each");
    memcpy(&api, p, sizeof(api));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"load", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&load)), METH_FASTCALL, nullptr},
    method<conv_prefill, 8>("conv_prefill"),
    method<conv_step, 6>("conv_step"),
    method<ssm_prefill, 13>("ssm_prefill"),
    method<ssm_step, 10>("ssm_step"),
    method<norm_in, 7>("norm_in"),
    method<norm_out, 9>("norm_out"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
