// fastcall.cpp -- the common call of the decode head's bindings in one
// step: tensors checked, device and stream looked up and the library's C
// function called from here instead of from Python (a call's overhead from 6 to 12 us to
// 3 us; the kernels of one token take 2 to 4).
//
// Every function returns the library's status, or -1 where a call is not the
// common one (a tensor of another kind, shape, layout or device, a device that
// is not the current one): binding.py then takes its own path, which serves
// what can be served and says what is wrong with the rest.  No computation
// happens here, and nothing is kept from one call for the next.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/luce_moe.h"

namespace {

using at::ScalarType;

decltype(&luce_quantize_i8) f_quantize;
decltype(&luce_rmsnorm_i8) f_rmsnorm;
decltype(&luce_add_rmsnorm_i8) f_add_rmsnorm;
decltype(&luce_linear_i8) f_linear;
decltype(&luce_logits_process) f_logits;
decltype(&luce_linear_w4) f_linear_w4;
decltype(&luce_sample) f_sample;

// The arguments of one call: `ok` turns false at the first that is not the common kind.
struct Args {
    bool ok = true;
    int dev = -1;

    const at::Tensor *tensor(PyObject *o, int dims)
    {
        if (!ok || !THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda() || t.dim() != dims || t.layout() != at::kStrided) {
            ok = false;
            return nullptr;
        }
        if (dev < 0)
            dev = t.get_device();
        ok = t.get_device() == dev;
        return &t;
    }
    // a contiguous tensor of a type and shape (b < 0: one axis)
    void *data(PyObject *o, ScalarType type, int64_t a, int64_t b = -1)
    {
        const at::Tensor *t = tensor(o, b < 0 ? 1 : 2);
        if (!ok || t->scalar_type() != type || t->size(0) != a || (b >= 0 && t->size(1) != b) || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void *data_or_none(PyObject *o, ScalarType type, int64_t a, int64_t b = -1)
    {
        return o == Py_None ? nullptr : data(o, type, a, b);
    }
    // a matrix with contiguous rows; its row stride
    void *rows(const at::Tensor *t, int64_t &ld)
    {
        if (!ok)
            return nullptr;
        ld = t->size(0) > 1 ? t->stride(0) : t->size(1);
        ok = t->size(1) == 1 || t->stride(1) == 1;
        return t->data_ptr();
    }
    luce_dtype dtype(const at::Tensor *t)
    {
        switch (ok ? t->scalar_type() : ScalarType::Undefined) {
        case ScalarType::Float:
            return LUCE_F32;
        case ScalarType::BFloat16:
            return LUCE_BF16;
        case ScalarType::Half:
            return LUCE_F16;
        default:
            ok = false;
            return LUCE_F32;
        }
    }
    int64_t size(const at::Tensor *t, int i) { return ok ? t->size(i) : 0; }
    int small(int64_t n) // an int argument of the library
    {
        ok = ok && n <= INT32_MAX;
        return (int)n;
    }
    void *stream()
    {
        ok = ok && c10::cuda::current_device() == dev;
        return ok ? (void *)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream() : nullptr;
    }
};

// A call's status for Python; whatever goes wrong on the way leaves the call to binding.py.
// (No catch of everything: a thread that the interpreter ends at its exit unwinds through here.)
template <class F> PyObject *result(F &&call)
{
    int status = -1;
    try {
        status = call();
    } catch (const std::exception &) {
        PyErr_Clear();
        status = -1;
    }
    return PyLong_FromLong(status);
}

// The library's function, without the interpreter's lock (as ctypes calls it): a
// launch may wait for a full queue, or for a host function that needs Python.
// The caller holds references to the tensors meanwhile.
template <class F, class... A> int unlocked(F f, A... args)
{
    int status = -1;
    PyThreadState *state = PyEval_SaveThread();
    try {
        status = (int)f(args...);
    } catch (const std::exception &) {
    }
    PyEval_RestoreThread(state);
    return status;
}

bool number(PyObject *o, float &v)
{
    if (!PyFloat_Check(o))
        return false;
    v = (float)PyFloat_AS_DOUBLE(o);
    return true;
}

PyObject *quantize_i8(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        if (n != 3 || !f_quantize)
            return -1;
        Args a;
        const at::Tensor *x = a.tensor(p[0], 2);
        const int64_t T = a.size(x, 0), H = a.size(x, 1);
        const luce_dtype dt = a.dtype(x);
        a.ok = a.ok && x->is_contiguous();
        void *q = a.data(p[1], ScalarType::Char, T, H), *s = a.data(p[2], ScalarType::Float, T);
        const int t = a.small(T), h = a.small(H);
        void *stream = a.stream();
        return a.ok ? unlocked(f_quantize, x->data_ptr(), dt, t, h, (int8_t *)q, (float *)s, stream) : -1;
    });
}

PyObject *rmsnorm_i8(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        float eps = 0;
        if (n != 5 || !f_rmsnorm || !number(p[2], eps))
            return -1;
        Args a;
        const at::Tensor *x = a.tensor(p[0], 2);
        const int64_t T = a.size(x, 0), H = a.size(x, 1);
        const luce_dtype dt = a.dtype(x);
        a.ok = a.ok && x->is_contiguous();
        void *g = a.data(p[1], ScalarType::Float, H), *q = a.data(p[3], ScalarType::Char, T, H),
             *s = a.data(p[4], ScalarType::Float, T);
        const int t = a.small(T), h = a.small(H);
        void *stream = a.stream();
        return a.ok ? unlocked(f_rmsnorm, x->data_ptr(), dt, (const float *)g, eps, t, h, (int8_t *)q, (float *)s, stream)
                    : -1;
    });
}

PyObject *add_rmsnorm_i8(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        float eps = 0;
        if (n != 7 || !f_add_rmsnorm || !number(p[4], eps))
            return -1;
        Args a;
        const at::Tensor *x = a.tensor(p[0], 2);
        const int64_t T = a.size(x, 0), H = a.size(x, 1);
        const luce_dtype dt = a.dtype(x);
        a.ok = a.ok && x->is_contiguous();
        const ScalarType st = a.ok ? x->scalar_type() : ScalarType::Float;
        void *r = a.data(p[1], st, T, H), *sum = a.data_or_none(p[2], st, T, H),
             *g = a.data(p[3], ScalarType::Float, H), *q = a.data(p[5], ScalarType::Char, T, H),
             *s = a.data(p[6], ScalarType::Float, T);
        const int t = a.small(T), h = a.small(H);
        void *stream = a.stream();
        return a.ok ? unlocked(f_add_rmsnorm, x->data_ptr(), r, sum, dt, (const float *)g, eps, t, h, (int8_t *)q,
                                         (float *)s, stream)
                    : -1;
    });
}

PyObject *linear_i8(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        if (n != 6 || !f_linear)
            return -1;
        Args a;
        const at::Tensor *x = a.tensor(p[0], 2), *w = a.tensor(p[2], 2), *o = a.tensor(p[5], 2);
        const int64_t T = a.size(x, 0), K = a.size(x, 1), N = a.size(w, 0);
        int64_t ldo = 0;
        a.ok = a.ok && o->size(0) == T && o->size(1) == N;
        const luce_dtype dt = a.dtype(o);
        void *out = a.rows(o, ldo), *xq = a.data(p[0], ScalarType::Char, T, K), *xs = a.data(p[1], ScalarType::Float, T),
             *wq = a.data(p[2], ScalarType::Char, N, K), *ws = a.data(p[3], ScalarType::Float, N),
             *b = a.data_or_none(p[4], ScalarType::Float, N);
        const int t = a.small(T), nn = a.small(N), k = a.small(K);
        void *stream = a.stream();
        return a.ok ? unlocked(f_linear, (const int8_t *)xq, (const float *)xs, (const int8_t *)wq, (const float *)ws,
                                    (const float *)b, t, nn, k, out, dt, ldo, stream)
                    : -1;
    });
}

// logits, out, hist, hist_len, prompt_len, repetition, frequency, presence, bias_ids, bias_vals, mask, mask_rows
PyObject *logits_process(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        if (n != 12 || !f_logits)
            return -1;
        Args a;
        const at::Tensor *l = a.tensor(p[0], 2), *o = a.tensor(p[1], 2);
        const int64_t R = a.size(l, 0), V = a.size(l, 1);
        int64_t ldl = 0, ldo = 0, ldh = 0, nb = 0, nm = 0, ldm = 0;
        a.ok = a.ok && o->size(0) == R && o->size(1) == V && o->scalar_type() == ScalarType::Float;
        const luce_dtype dt = a.dtype(l);
        void *lp = a.rows(l, ldl), *op = a.rows(o, ldo), *hp = nullptr, *hl = nullptr, *bi = nullptr, *bv = nullptr,
             *mp = nullptr;
        if (p[2] != Py_None) {
            ldh = a.size(a.tensor(p[2], 2), 1);
            a.ok = a.ok && ldh > 0; // (an empty history: binding.py)
            hp = a.data(p[2], ScalarType::Int, R, ldh);
            hl = a.data(p[3], ScalarType::Int, R);
        } else {
            a.ok = a.ok && p[3] == Py_None && p[4] == Py_None;
        }
        if (p[8] != Py_None) {
            nb = a.size(a.tensor(p[8], 2), 1);
            bi = a.data(p[8], ScalarType::Int, R, nb);
            bv = a.data(p[9], ScalarType::Float, R, nb);
        } else {
            a.ok = a.ok && p[9] == Py_None;
        }
        if (p[10] != Py_None) {
            const at::Tensor *m = a.tensor(p[10], 2);
            nm = a.size(m, 0);
            ldm = a.size(m, 1);
            a.ok = a.ok && nm > 0 && ldm > 0; // (no masks, or masks without words: binding.py)
            mp = a.data(p[10], a.ok && m->scalar_type() == ScalarType::UInt32 ? ScalarType::UInt32 : ScalarType::Int, nm, ldm);
        } else {
            a.ok = a.ok && p[11] == Py_None;
        }
        void *pl = a.data_or_none(p[4], ScalarType::Int, R), *rep = a.data_or_none(p[5], ScalarType::Float, R),
             *fr = a.data_or_none(p[6], ScalarType::Float, R), *pr = a.data_or_none(p[7], ScalarType::Float, R),
             *mr = a.data_or_none(p[11], ScalarType::Int, R);
        const int r = a.small(R), b = a.small(nb), m = a.small(nm);
        void *stream = a.stream();
        return a.ok ? unlocked(f_logits, lp, dt, r, V, ldl, (const int32_t *)hp, ldh, (const int32_t *)hl, (const int32_t *)pl,
                                    (const float *)rep, (const float *)fr, (const float *)pr, (const int32_t *)bi,
                                    (const float *)bv, b, (const uint32_t *)mp, m, ldm, (const int32_t *)mr, (float *)op,
                                    ldo, stream)
                    : -1;
    });
}

// x, x_scale, wq, scale, zeros, group, bias, out
PyObject *linear_w4(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        if (n != 8 || !f_linear_w4 || !PyLong_Check(p[5]))
            return -1;
        const long group = PyLong_AsLong(p[5]);
        if (group != 32 && group != 64 && group != 128) {
            PyErr_Clear(); // (of a number beyond a long)
            return -1;
        }
        Args a;
        const at::Tensor *x = a.tensor(p[0], 2), *w = a.tensor(p[2], 2), *s = a.tensor(p[3], 2), *o = a.tensor(p[7], 2);
        const int64_t T = a.size(x, 0), K = a.size(x, 1), N = a.size(w, 0), G = (K + group - 1) / group;
        int64_t ldx = 0, ldo = 0;
        a.ok = a.ok && o->size(0) == T && o->size(1) == N;
        const bool i8 = a.ok && x->scalar_type() == ScalarType::Char;
        const luce_dtype xt = i8 ? LUCE_I8 : a.dtype(x), st = a.dtype(s), ot = a.dtype(o);
        a.ok = a.ok && st != LUCE_F32 && i8 == (p[1] != Py_None);
        void *xp = a.rows(x, ldx), *out = a.rows(o, ldo), *xs = a.data_or_none(p[1], ScalarType::Float, T),
             *wq = a.data(p[2], ScalarType::Byte, N, (K + 127) / 128 * 64),
             *ws = a.data(p[3], st == LUCE_F16 ? ScalarType::Half : ScalarType::BFloat16, N, G),
             *z = a.data_or_none(p[4], ScalarType::Byte, N, G), *b = a.data_or_none(p[6], ScalarType::Float, N);
        const int t = a.small(T), nn = a.small(N), k = a.small(K);
        void *stream = a.stream();
        return a.ok ? unlocked(f_linear_w4, (const void *)xp, xt, ldx, (const float *)xs, (const uint8_t *)wq, (const void *)ws, st,
                               (const uint8_t *)z, (int)group, (const float *)b, t, nn, k, out, ot, ldo, stream)
                    : -1;
    });
}

// logits, u, idx, prob, temperature, top_k, top_p, min_p
PyObject *sample(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    return result([&] {
        if (n != 8 || !f_sample)
            return -1;
        Args a;
        const at::Tensor *l = a.tensor(p[0], 2);
        const int64_t R = a.size(l, 0), V = a.size(l, 1);
        int64_t ld = 0;
        const luce_dtype dt = a.dtype(l);
        void *lp = a.rows(l, ld), *u = a.data(p[1], ScalarType::Float, R), *idx = a.data(p[2], ScalarType::Int, R),
             *prob = a.data_or_none(p[3], ScalarType::Float, R), *t = a.data_or_none(p[4], ScalarType::Float, R),
             *k = a.data_or_none(p[5], ScalarType::Int, R), *tp = a.data_or_none(p[6], ScalarType::Float, R),
             *mp = a.data_or_none(p[7], ScalarType::Float, R);
        const int r = a.small(R);
        void *stream = a.stream();
        return a.ok ? unlocked(f_sample, (const void *)lp, dt, r, V, ld, (const float *)u, (const float *)t, (const int32_t *)k,
                               (const float *)tp, (const float *)mp, (int32_t *)idx, (float *)prob, stream)
                    : -1;
    });
}

// bind(addresses): the library's functions, in the order of the pointers above; bind_more: the last two
PyObject *bind(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "bind takes five addresses");
        return nullptr;
    }
    void *at[5];
    for (int i = 0; i < 5; i++) {
        at[i] = PyLong_AsVoidPtr(p[i]);
        if (!at[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "bind takes addresses that are not null");
            return nullptr;
        }
    }
    f_quantize = reinterpret_cast<decltype(f_quantize)>(at[0]);
    f_rmsnorm = reinterpret_cast<decltype(f_rmsnorm)>(at[1]);
    f_add_rmsnorm = reinterpret_cast<decltype(f_add_rmsnorm)>(at[2]);
    f_linear = reinterpret_cast<decltype(f_linear)>(at[3]);
    f_logits = reinterpret_cast<decltype(f_logits)>(at[4]);
    Py_RETURN_NONE;
}

PyObject *bind_more(PyObject *, PyObject *const *p, Py_ssize_t n)
{
    if (n != 2) {
        PyErr_SetString(PyExc_TypeError, "bind_more takes two addresses");
        return nullptr;
    }
    void *at[2];
    for (int i = 0; i < 2; i++) {
        at[i] = PyLong_AsVoidPtr(p[i]);
        if (!at[i]) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "bind_more takes addresses that are not null");
            return nullptr;
        }
    }
    f_linear_w4 = reinterpret_cast<decltype(f_linear_w4)>(at[0]);
    f_sample = reinterpret_cast<decltype(f_sample)>(at[1]);
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),      METHOD(quantize_i8),    METHOD(rmsnorm_i8), METHOD(add_rmsnorm_i8),
                         METHOD(linear_i8), METHOD(logits_process), METHOD(bind_more),  METHOD(linear_w4),
                         METHOD(sample),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "luce_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

} // namespace

PyMODINIT_FUNC PyInit_luce_call(void) { return PyModule_Create(&module); }
