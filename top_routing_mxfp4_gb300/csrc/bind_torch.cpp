// Binding of the short calls (norms, MXFP4 linear, grouped products) on torch
// tensors: the same marshalling as the ctypes functions of lmoe.py (checks of
// types, shapes and devices, outputs allocated in the call's stream, then the C
// entry point of the same name), in C++.  These calls run for a few
// microseconds; through ctypes a call with two outputs cost 12 us of host time,
// here about 4.
//
// The module is not linked to the library: lmoe.py hands it the addresses of the
// entry points of the library it loaded (bind).
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <stdexcept>
#include <string>

#include "lmoe.h"

namespace {

struct Entries {
    decltype(&lmoe_rms_norm) rms_norm;
    decltype(&lmoe_residual_norm) residual_norm;
    decltype(&lmoe_linear_mxfp4) linear_mxfp4;
    decltype(&lmoe_linear_mxfp4_workspace_size) linear_mxfp4_workspace_size;
    decltype(&lmoe_grouped_linear_bf16) grouped_linear;
    decltype(&lmoe_grouped_swiglu_bf16) grouped_swiglu;
    decltype(&lmoe_grouped_workspace_size) grouped_workspace_size;
} E = {};
PyObject *g_error = nullptr;  // lmoe.LmoeError
// The workspace of the latest call that made its own, kept so that the errors
// the call found on the GPU can be asked for (lmoe.last_call_status).
PyObject *g_own_ws = nullptr;

struct Bad : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PyError {};  // a Python exception is already set

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) throw Bad(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

[[noreturn]] void mismatch(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, const char *name, int dev)
{
    std::ostringstream s;
    s << name << ": expected contiguous " << type << ' ' << shape << " on cuda:" << dev << ", got " << t.scalar_type()
      << ' ' << t.sizes() << " on " << t.device() << ", strides " << t.strides();
    throw Bad(s.str());
}

// Checks one tensor; returns its address.
void *need(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, const char *name, int dev)
{
    if (t.scalar_type() != type || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        mismatch(t, type, shape, name, dev);
    return t.data_ptr();
}
void *need_or_null(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int dev)
{
    return o == Py_None ? nullptr : need(tensor(o, name), type, shape, name, dev);
}

int cuda_index(const at::Tensor &t, const char *name)
{
    if (!t.is_cuda()) throw Bad(std::string(name) + ": expected a CUDA tensor");
    return int(t.get_device());
}

int float_fmt(const at::Tensor &t, const char *name)
{
    if (t.scalar_type() == at::kBFloat16) return LMOE_BF16;
    if (t.scalar_type() == at::kFloat) return LMOE_F32;
    throw Bad(std::string(name) + ": expected bfloat16 or float32");
}

void rank_is(const at::Tensor &t, int64_t n, const char *name)
{
    if (t.dim() != n) throw Bad(std::string(name) + ": expected " + std::to_string(n) + " dimensions");
}

// The call's device and stream made current (allocations go to that stream).
struct On {
    c10::cuda::CUDAGuard device;
    c10::cuda::OptionalCUDAStreamGuard other;
    cudaStream_t stream;
    On(int dev, PyObject *s) : device(c10::DeviceIndex(dev))
    {
        if (s == Py_None) {
            stream = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
            return;
        }
        PyObject *h = PyObject_GetAttrString(s, "cuda_stream"), *i = PyObject_GetAttrString(s, "device_index");
        if (!h || !i) {
            Py_XDECREF(h);
            Py_XDECREF(i);
            throw PyError();
        }
        stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
        const long at = PyLong_AsLong(i);
        Py_DECREF(h);
        Py_DECREF(i);
        if (PyErr_Occurred()) throw PyError();
        if (at != dev)
            throw Bad("stream on cuda:" + std::to_string(at) + ", tensors on cuda:" + std::to_string(dev));
        other.reset_stream(c10::cuda::getStreamFromExternal(stream, c10::DeviceIndex(dev)));
    }
};

// An output: the caller's, checked, or a new one.
struct Out {
    PyObject *obj;  // a new reference
    void *ptr;
    Out(PyObject *given, const at::Tensor &like, at::IntArrayRef shape, at::ScalarType type, const char *name, int dev)
    {
        if (given != Py_None) {
            ptr = need(tensor(given, name), type, shape, name, dev);
            Py_INCREF(given);
            obj = given;
        } else {
            at::Tensor t = at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
            ptr = t.data_ptr();
            obj = THPVariable_Wrap(std::move(t));
        }
    }
    Out(const Out &) = delete;
    ~Out() { Py_XDECREF(obj); }
    PyObject *release()
    {
        PyObject *o = obj;
        obj = nullptr;
        return o;
    }
};

// A workspace: the caller's, or a zeroed one for this call.
struct Ws {
    at::Tensor own;
    void *ptr;
    size_t bytes;
    Ws(PyObject *given, size_t want, const at::Tensor &like, int dev)
    {
        const at::Tensor *t = &own;
        if (given != Py_None) {
            t = &tensor(given, "ws");
            need(*t, at::kByte, t->sizes(), "ws", dev);
        } else {
            own = at::zeros({int64_t(want < 256 ? 256 : want)}, like.options().dtype(at::kByte));
            PyObject *o = THPVariable_Wrap(own);
            if (!o) throw PyError();
            Py_XSETREF(g_own_ws, o);
        }
        ptr = t->data_ptr();
        bytes = size_t(t->numel());
    }
};

void check(lmoe_status code, const char *what)
{
    if (code == LMOE_OK) return;
    if (PyObject *e = PyObject_CallFunction(g_error, "is", int(code), what)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw PyError();
}

double as_double(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyError();
    return v;
}
int64_t as_int(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyError();
    return v;
}

template <PyObject *(*F)(PyObject *const *)>
PyObject *entry(PyObject *, PyObject *const *a, Py_ssize_t)
{
    try {
        if (!E.rms_norm) throw Bad("not bound to a library");
        return F(a);
    } catch (const PyError &) {
    } catch (const Bad &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (x, w, eps, out, stream)
PyObject *rms_norm(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x");
    rank_is(x, 2, "x");
    const int dev = cuda_index(x, "x"), fmt = float_fmt(x, "x");
    const int64_t T = x.size(0), H = x.size(1);
    const void *xp = need(x, x.scalar_type(), {T, H}, "x", dev);
    const void *wp = need(tensor(a[1], "w"), at::kFloat, {H}, "w", dev);
    const double eps = as_double(a[2]);
    On on(dev, a[4]);
    Out out(a[3], x, {T, H}, at::kBFloat16, "out", dev);
    if (H > INT32_MAX) throw Bad("x: too wide");
    check(E.rms_norm(xp, fmt, static_cast<const float *>(wp), float(eps), T, int32_t(H),
                     static_cast<uint16_t *>(out.ptr), on.stream),
          "lmoe_rms_norm");
    return out.release();
}

// The kind of a gate on [T][H] and its address.
int gate_kind(PyObject *o, int64_t T, int64_t H, int dev, const void *&ptr)
{
    ptr = nullptr;
    if (o == Py_None) return LMOE_GATE_NONE;
    const at::Tensor &g = tensor(o, "gate");
    if (g.scalar_type() == at::kBFloat16) {
        ptr = need(g, at::kBFloat16, {T, H}, "gate", dev);
        return LMOE_GATE_FULL;
    }
    if (g.dim() == 2 && g.size(0) == T && g.size(1) == 1) {
        ptr = need(g, at::kFloat, {T, 1}, "gate", dev);
        return LMOE_GATE_TOKEN;
    }
    ptr = g.dim() == 2 ? need(g, at::kFloat, {1, H}, "gate", dev) : need(g, at::kFloat, {H}, "gate", dev);
    return LMOE_GATE_CHANNEL;
}

// (y, res, post_w, gate, scale, next_w, eps, res_out, next_out, stream) -> (res_out, next_out or None)
PyObject *residual_norm(PyObject *const *a)
{
    const at::Tensor &y = tensor(a[0], "y"), &res = tensor(a[1], "res");
    rank_is(y, 2, "y");
    const int dev = cuda_index(y, "y"), fmt = float_fmt(res, "res");
    const int64_t T = y.size(0), H = y.size(1);
    if (H > INT32_MAX) throw Bad("y: too wide");
    const void *yp = need(y, at::kBFloat16, {T, H}, "y", dev), *rp = need(res, res.scalar_type(), {T, H}, "res", dev);
    const void *pw = need_or_null(a[2], at::kFloat, {H}, "post_w", dev), *gp;
    const int kind = gate_kind(a[3], T, H, dev, gp);
    const double scale = as_double(a[4]), eps = as_double(a[6]);
    const void *nw = need_or_null(a[5], at::kFloat, {H}, "next_w", dev);
    if (!nw && a[8] != Py_None) throw Bad("next_out without next_w");
    On on(dev, a[9]);
    Out ro(a[7], res, {T, H}, res.scalar_type(), "res_out", dev);
    auto call = [&](void *next) {
        check(E.residual_norm(static_cast<const uint16_t *>(yp), rp, fmt, static_cast<const float *>(pw), gp, kind,
                              float(scale), float(eps), static_cast<const float *>(nw), T, int32_t(H), ro.ptr,
                              static_cast<uint16_t *>(next), on.stream),
              "lmoe_residual_norm");
    };
    PyObject *next = Py_None;
    if (nw) {
        Out no(a[8], y, {T, H}, at::kBFloat16, "next_out", dev);
        call(no.ptr);
        next = no.release();
    } else {
        call(nullptr);
        Py_INCREF(Py_None);
    }
    PyObject *two = PyTuple_New(2);
    if (!two) {
        Py_DECREF(next);
        throw PyError();
    }
    PyTuple_SET_ITEM(two, 0, ro.release());
    PyTuple_SET_ITEM(two, 1, next);
    return two;
}

// (x, q, s, N, out, ws, stream)
PyObject *linear_mxfp4(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x");
    rank_is(x, 2, "x");
    const int dev = cuda_index(x, "x");
    const int64_t rows = x.size(0), K = x.size(1), N = as_int(a[3]);
    if (K <= 0 || K % 32 || N <= 0 || K > INT32_MAX || N > INT32_MAX)
        throw Bad("weights [" + std::to_string(N) + ", " + std::to_string(K) + "]: K must be a multiple of 32");
    const int64_t KC = (K + 127) / 128;
    const void *xp = need(x, at::kBFloat16, {rows, K}, "x", dev);
    const void *qp = need(tensor(a[1], "q"), at::kByte, {N * KC * 64}, "q", dev);
    const void *sp = need(tensor(a[2], "s"), at::kByte, {(N + 127) / 128 * KC * 512}, "s", dev);
    On on(dev, a[6]);
    Out out(a[4], x, {rows, N}, at::kBFloat16, "out", dev);
    Ws ws(a[5], a[5] == Py_None ? E.linear_mxfp4_workspace_size(rows, int32_t(K), int32_t(N)) : 0, x, dev);
    check(E.linear_mxfp4(static_cast<const uint16_t *>(xp), static_cast<const uint8_t *>(qp),
                         static_cast<const uint8_t *>(sp), rows, int32_t(K), int32_t(N),
                         static_cast<uint16_t *>(out.ptr), ws.ptr, ws.bytes, on.stream),
          "lmoe_linear_mxfp4");
    return out.release();
}

// (x, W, Wu or None, offsets, perm, k, gather, row_w, out, ws, stream)
PyObject *grouped(PyObject *const *a)
{
    const at::Tensor &x = tensor(a[0], "x"), &W = tensor(a[1], "W");
    rank_is(x, 2, "x");
    rank_is(W, 3, "W");
    const int dev = cuda_index(x, "x");
    const int64_t n_exp = W.size(0), N = W.size(1), K = W.size(2), rows = x.size(0);
    if (n_exp > INT32_MAX || N > INT32_MAX || K > INT32_MAX) throw Bad("W: too large");
    const void *xp = need(x, at::kBFloat16, {rows, K}, "x", dev);
    const void *wp = need(W, at::kBFloat16, {n_exp, N, K}, "W", dev);
    const void *up = need_or_null(a[2], at::kBFloat16, {n_exp, N, K}, "Wu", dev);
    const bool perm = a[4] != Py_None;
    const int64_t P = perm ? tensor(a[4], "perm").numel() : rows, k = as_int(a[5]);
    if (k < 1 || k > INT32_MAX) throw Bad("k: expected at least 1");
    lmoe_groups g;
    g.offsets = static_cast<const int32_t *>(need(tensor(a[3], "offsets"), at::kInt, {n_exp + 1}, "offsets", dev));
    g.perm = static_cast<const int32_t *>(need_or_null(a[4], at::kInt, {P}, "perm", dev));
    g.P = P;
    g.E = int32_t(n_exp);
    g.k = int32_t(k);
    const int gather = a[6] == Py_None ? int(perm) : PyObject_IsTrue(a[6]);
    if (gather < 0) throw PyError();
    const void *rw = nullptr;
    if (a[7] != Py_None) {
        const at::Tensor &r = tensor(a[7], "row_w");
        if (r.numel() != P)
            throw Bad("row_w: " + std::to_string(P) + " values expected, got " + std::to_string(r.numel()));
        rw = need(r, at::kFloat, r.sizes(), "row_w", dev);
    }
    // without `out`: bf16, or fp32 of weighted rows
    const int fmt = a[8] != Py_None ? float_fmt(tensor(a[8], "out"), "out") : rw ? LMOE_F32 : LMOE_BF16;
    if (up && fmt != LMOE_BF16) throw Bad("out: expected bfloat16");
    On on(dev, a[10]);
    Out out(a[8], x, {P, N}, fmt == LMOE_F32 ? at::kFloat : at::kBFloat16, "out", dev);
    Ws ws(a[9], E.grouped_workspace_size(), x, dev);
    if (up)
        check(E.grouped_swiglu(static_cast<const uint16_t *>(xp), rows, static_cast<const uint16_t *>(wp),
                               static_cast<const uint16_t *>(up), &g, gather, int32_t(K), int32_t(N),
                               static_cast<uint16_t *>(out.ptr), ws.ptr, ws.bytes, on.stream),
              "lmoe_grouped_swiglu_bf16");
    else
        check(E.grouped_linear(static_cast<const uint16_t *>(xp), rows, static_cast<const uint16_t *>(wp), &g, gather,
                               static_cast<const float *>(rw), int32_t(K), int32_t(N), fmt, out.ptr, ws.ptr, ws.bytes,
                               on.stream),
              "lmoe_grouped_linear_bf16");
    return out.release();
}

// bind(error class, addresses of the seven entry points in the order of Entries)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "bind: the error class and seven addresses");
        return nullptr;
    }
    void *p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i + 1]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: a null address");
            return nullptr;
        }
    }
    Py_INCREF(a[0]);
    Py_XDECREF(g_error);
    g_error = a[0];
    E.rms_norm = reinterpret_cast<decltype(E.rms_norm)>(p[0]);
    E.residual_norm = reinterpret_cast<decltype(E.residual_norm)>(p[1]);
    E.linear_mxfp4 = reinterpret_cast<decltype(E.linear_mxfp4)>(p[2]);
    E.linear_mxfp4_workspace_size = reinterpret_cast<decltype(E.linear_mxfp4_workspace_size)>(p[3]);
    E.grouped_linear = reinterpret_cast<decltype(E.grouped_linear)>(p[4]);
    E.grouped_swiglu = reinterpret_cast<decltype(E.grouped_swiglu)>(p[5]);
    E.grouped_workspace_size = reinterpret_cast<decltype(E.grouped_workspace_size)>(p[6]);
    Py_RETURN_NONE;
}

// own_ws() -> the workspace of the latest call that made its own, or None
PyObject *own_ws(PyObject *, PyObject *)
{
    PyObject *o = g_own_ws ? g_own_ws : Py_None;
    Py_INCREF(o);
    return o;
}

// keep_ws(workspace): as if the latest call had made it
PyObject *keep_ws(PyObject *, PyObject *ws)
{
    Py_INCREF(ws);
    Py_XSETREF(g_own_ws, ws);
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), int N>
PyObject *counted(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    return entry<F>(self, a, n);
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {
    {"bind", FAST(bind), METH_FASTCALL, nullptr},
    {"rms_norm", FAST((counted<rms_norm, 5>)), METH_FASTCALL, nullptr},
    {"residual_norm", FAST((counted<residual_norm, 10>)), METH_FASTCALL, nullptr},
    {"linear_mxfp4", FAST((counted<linear_mxfp4, 7>)), METH_FASTCALL, nullptr},
    {"grouped", FAST((counted<grouped, 11>)), METH_FASTCALL, nullptr},
    {"own_ws", own_ws, METH_NOARGS, nullptr},
    {"keep_ws", keep_ws, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lmoe_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// BUILT_FOR: the torch and Python of the build (build.py), whose layouts are
// compiled in; lmoe.py compares it with what runs.
extern "C" PyObject *PyInit__lmoe_torch(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "BUILT_FOR", LMOE_BUILT_FOR) != 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
