// fg_bind.cpp - the calls of a serving step from Python without Python's price: each takes the binding's arguments,
// checks what the binding checks and calls the entry point.  Arguments that do not pass (or are not tensors at all)
// are left to the binding, which says what is wrong: the result is then None, else the entry point's status.
//
// These calls take 2 to 15 us on the GPU; marshalling one in Python takes 3.5 us on a GB300's host besides the 2.2 us of its
// launch, here 0.4.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "fg.h"

namespace {

using at::ScalarType;
using at::Tensor;

const Tensor* tensor(PyObject* o, ScalarType type) {
    if (!THPVariable_Check(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    return t.is_cuda() && t.scalar_type() == type ? &t : nullptr;
}
const Tensor* whole(PyObject* o, ScalarType type) {
    const Tensor* t = tensor(o, type);
    return t && t->is_contiguous() ? t : nullptr;
}
template <class T>
T* at_of(const Tensor* t) { return static_cast<T*>(t->data_ptr()); }

// [T, heads, D] BF16 whose heads are contiguous; ld: elements between tokens.
struct Rows {
    const Tensor* t;
    int64_t n, heads, d, ld;
};
bool rows(PyObject* o, Rows& r) {
    r.t = tensor(o, ScalarType::BFloat16);
    if (!r.t || r.t->dim() != 3) return false;
    r.n = r.t->size(0);
    r.heads = r.t->size(1);
    r.d = r.t->size(2);
    r.ld = r.heads * r.d;
    if (r.t->is_contiguous()) return true;
    if (!((r.t->stride(2) == 1 || r.d == 1) && (r.t->stride(1) == r.d || r.heads == 1))) return false;
    if (r.n > 1) r.ld = r.t->stride(0);
    return true;
}
bool same(const Rows& a, const Rows& b) { return a.n == b.n && a.heads == b.heads && a.d == b.d; }

struct Cache {
    const Tensor* a[4];           // codes and scales of keys, of values
    int64_t pages, heads, size, d;
};
bool cache(PyObject* const* o, Cache& c) {
    for (int i = 0; i < 4; ++i)
        if (!(c.a[i] = whole(o[i], ScalarType::Byte))) return false;
    if (c.a[0]->dim() != 4) return false;
    c.pages = c.a[0]->size(0);
    c.heads = c.a[0]->size(1);
    c.size = c.a[0]->size(2);
    c.d = 2 * c.a[0]->size(3);
    const int64_t n = c.a[0]->numel();
    return c.d % 32 == 0 && c.a[2]->numel() == n && c.a[1]->numel() * 16 == n && c.a[3]->numel() * 16 == n;
}

bool fits(int64_t x) { return x == static_cast<int>(x); }
template <class... A>
bool fits(int64_t x, A... rest) { return fits(x) && fits(rest...); }
bool integer(PyObject* o, int& x) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &over);
    x = static_cast<int>(v);
    return !over && v == x;
}
bool number(PyObject* o, double& x) {
    if (!PyFloat_CheckExact(o)) return false;
    x = PyFloat_AS_DOUBLE(o);
    return true;
}
// The interpreter's other threads go on while a call is made (a full launch queue makes it wait).
struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F>
PyObject* status(F call) {
    int st;
    {
        Unlocked unlocked;
        st = call();
    }
    return PyLong_FromLong(st);
}
fg_stream_t stream() { return reinterpret_cast<fg_stream_t>(c10::cuda::getCurrentCUDAStream().stream()); }

// Arguments as the binding's functions have them, without the stream (the current one); workspaces by their need.
PyObject* tables(PyObject* const* o) {
    const Tensor* a[10];
    for (int i = 0; i < 10; ++i)
        if (!(a[i] = whole(o[i], ScalarType::Int))) return nullptr;
    int page, pages;
    if (!integer(o[10], page) || !integer(o[11], pages) || a[4]->dim() != 2) return nullptr;
    const int64_t s = a[4]->size(0), width = a[4]->size(1), t = a[7]->numel(), n = a[2]->numel();
    if (a[0]->numel() != s || a[1]->numel() != s || a[6]->numel() != s || a[5]->numel() != s + 1 || a[8]->numel() != t ||
        a[3]->numel() != 1 || a[9]->numel() != 1 || !fits(s, t, width, n))
        return nullptr;
    using I = int32_t;
    return status([&] { return fg_build_block_tables(
        static_cast<int>(s), static_cast<int>(t), page, pages, static_cast<int>(width), static_cast<int>(n), at_of<I>(a[0]),
        at_of<I>(a[1]), at_of<I>(a[2]), at_of<I>(a[3]), at_of<I>(a[4]), at_of<I>(a[5]), at_of<I>(a[6]), at_of<I>(a[7]),
        at_of<I>(a[8]), at_of<I>(a[9]), stream()); });
}

PyObject* rope(PyObject* const* o) {
    Rows q, k, qo, ko;
    if (!rows(o[0], q) || !rows(o[1], k) || !rows(o[4], qo) || !rows(o[5], ko)) return nullptr;
    const Tensor *pos = whole(o[2], ScalarType::Int), *cs = whole(o[3], ScalarType::Float), *w[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i)
        if (o[6 + i] != Py_None && (!(w[i] = whole(o[6 + i], ScalarType::BFloat16)) || w[i]->numel() != q.d)) return nullptr;
    double eps;
    if (!pos || !cs || cs->dim() != 2 || !number(o[8], eps) || !PyBool_Check(o[9])) return nullptr;
    if (k.n != q.n || k.d != q.d || !same(q, qo) || !same(k, ko) || pos->numel() != q.n ||
        !fits(q.n, q.heads, k.heads, q.d, cs->size(0), cs->size(1)))
        return nullptr;
    const int turn = o[9] == Py_True;
    return status([&] { return fg_qk_norm_rope(
        static_cast<int>(q.n), static_cast<int>(q.heads), static_cast<int>(k.heads), static_cast<int>(q.d),
        static_cast<int>(cs->size(1)), static_cast<int>(cs->size(0)), q.t->data_ptr(), q.ld, k.t->data_ptr(), k.ld,
        w[0] ? w[0]->data_ptr() : nullptr, w[1] ? w[1]->data_ptr() : nullptr, static_cast<float>(eps), at_of<int32_t>(pos),
        at_of<float>(cs), turn, qo.t->data_ptr(), qo.ld, ko.t->data_ptr(), ko.ld, stream()); });
}

PyObject* move(PyObject* const* o, bool append) {             // k, v, slots, cache
    Rows k, v;
    Cache c;
    const Tensor* slots = whole(o[2], ScalarType::Int);
    if (!rows(o[0], k) || !rows(o[1], v) || !slots || !cache(o + 3, c)) return nullptr;
    if (!same(k, v) || k.n != slots->numel() || k.heads != c.heads || k.d != c.d || !fits(k.n, c.heads, c.d, c.size, c.pages))
        return nullptr;
    const int t = static_cast<int>(k.n), heads = static_cast<int>(c.heads), d = static_cast<int>(c.d), size = static_cast<int>(c.size),
              pages = static_cast<int>(c.pages);
    using U = uint8_t;
    U *kc = at_of<U>(c.a[0]), *ks = at_of<U>(c.a[1]), *vc = at_of<U>(c.a[2]), *vs = at_of<U>(c.a[3]);
    return status([&] {
        return append ? fg_kv_append_mxfp4(t, heads, d, size, pages, k.t->data_ptr(), k.ld, v.t->data_ptr(), v.ld, at_of<int32_t>(slots),
                                    kc, ks, vc, vs, stream())
               : fg_kv_gather_mxfp4(t, heads, d, size, pages, at_of<int32_t>(slots), kc, ks, vc, vs, k.t->data_ptr(), k.ld,
                                    v.t->data_ptr(), v.ld, stream());
    });
}

PyObject* attention(PyObject* const* o) {
    Cache c;
    const Tensor *q = whole(o[0], ScalarType::BFloat16), *table = whole(o[5], ScalarType::Int), *start = whole(o[6], ScalarType::Int),
                 *lens = whole(o[7], ScalarType::Int), *out = whole(o[8], ScalarType::BFloat16);
    if (!q || !table || !start || !lens || !out || !cache(o + 1, c) || !THPVariable_Check(o[9])) return nullptr;
    const Tensor& ws = THPVariable_Unpack(o[9]);
    int window;
    double scale = 0.0;
    if (q->dim() != 3 || out->sizes() != q->sizes() || table->dim() != 2 || !integer(o[11], window) ||
        (o[10] != Py_None && !number(o[10], scale)))
        return nullptr;
    const int64_t t = q->size(0), hq = q->size(1), s = table->size(0), width = table->size(1);
    if (q->size(2) != c.d || start->numel() != s + 1 || lens->numel() != s || !fits(t, s, hq, width, c.pages, c.heads, c.size, c.d) ||
        !ws.is_cuda() || !ws.is_contiguous())
        return nullptr;
    if (o[10] == Py_None) scale = 1.0 / std::sqrt(static_cast<double>(c.d));
    const int T = static_cast<int>(t), S = static_cast<int>(s), Hq = static_cast<int>(hq), Hkv = static_cast<int>(c.heads),
              D = static_cast<int>(c.d);
    if (static_cast<long long>(ws.nbytes()) < fg_paged_attention_workspace(T, S, Hq, Hkv, D)) return nullptr;
    using I = int32_t;
    using U = uint8_t;
    return status([&] { return fg_paged_attention_mxfp4(
        T, S, Hq, Hkv, D, static_cast<int>(c.size), static_cast<int>(c.pages), static_cast<int>(width), q->data_ptr(), at_of<U>(c.a[0]),
        at_of<U>(c.a[1]), at_of<U>(c.a[2]), at_of<U>(c.a[3]), at_of<I>(table), at_of<I>(start), at_of<I>(lens),
        static_cast<float>(scale), window, out->data_ptr(), ws.data_ptr(), stream()); });
}

template <Py_ssize_t kArgs, class F>
PyObject* guarded(PyObject* const* o, Py_ssize_t n, F f) {
    try {
        if (n == kArgs)
            if (PyObject* r = f(o)) return r;
    } catch (...) {                                            // a tensor without storage and the like
    }
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NONE;
}
PyObject* py_tables(PyObject*, PyObject* const* o, Py_ssize_t n) { return guarded<12>(o, n, tables); }
PyObject* py_rope(PyObject*, PyObject* const* o, Py_ssize_t n) { return guarded<10>(o, n, rope); }
PyObject* py_append(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded<7>(o, n, [](PyObject* const* x) { return move(x, true); });
}
PyObject* py_gather(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded<7>(o, n, [](PyObject* const* x) { return move(x, false); });
}
PyObject* py_attention(PyObject*, PyObject* const* o, Py_ssize_t n) { return guarded<12>(o, n, attention); }

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<py_tables>("tables"), method<py_rope>("rope"), method<py_append>("append"),
                           method<py_gather>("gather"), method<py_attention>("attention"), {nullptr, nullptr, 0, nullptr}};
// The docstring says which torch and which Python the module is built for: it holds their inlined code, so it is not
// loaded beside others (the build script's bind_fits looks for it in the file).
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "fg_bind", FG_BIND_ABI, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_fg_bind() { return PyModule_Create(&g_module); }
