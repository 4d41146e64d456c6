// Marshalling of the calls that a decoding step makes, where the host is the longer part of a call: a Python extension that
// reads the tensors' types, shapes, strides and pointers and calls the C entry point. Host time of a call on the GPU machine,
// against attribute by attribute through Python and ctypes: the cache's write 3.1 us against 11.5, attention over the cache
// 4.7 against 14.7, the norm 4.4 against 9.5; a launch alone is 2 to 3 of it.
//
// It takes what a right call passes and nothing else: each function returns the entry point's status, or None where anything
// is out of the ordinary (another type or device, an unusual stride, an empty tensor, a number beyond 32 bits). The Python binding then
// goes through its own checks, which say what is wrong or make the call.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>

#include "mptp.h"

namespace {

// One call's arguments; `ok` stays true while they are ordinary.
struct Args {
    PyObject* const* a;
    bool ok = true;
    int device = -1;  // the current one, asked for with the first tensor

    bool here(const at::Tensor& t) {
        if (device < 0) device = c10::cuda::current_device();
        return t.get_device() == device;
    }
    const at::Tensor* tensor(int i, at::ScalarType type) {
        if (!ok || !THPVariable_Check(a[i])) return fail();
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (t.scalar_type() != type || !t.is_cuda() || t.layout() != at::kStrided || t.numel() == 0 || !here(t))
            return fail();
        return &t;
    }
    // Contiguous, of this shape.
    void* pointer(int i, at::ScalarType type, at::IntArrayRef shape) {
        const at::Tensor* t = tensor(i, type);
        if (!t || t->sizes() != shape || !t->is_contiguous()) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    // [T, heads, d] with contiguous rows: pointer and pitch.
    void* rows(int i, int64_t T, int64_t heads, int64_t d, long long* ld) {
        const at::Tensor* t = tensor(i, at::kBFloat16);
        if (!t || t->dim() != 3 || t->size(0) != T || t->size(1) != heads || t->size(2) != d || t->stride(2) != 1 ||
            t->stride(1) != d || (T > 1 && t->stride(0) < heads * d)) {
            ok = false;
            return nullptr;
        }
        *ld = T > 1 ? t->stride(0) : heads * d;
        return t->data_ptr();
    }
    int integer(int i) {
        if (!ok || !PyLong_CheckExact(a[i])) return ok = false, 0;
        int over = 0;
        const long v = PyLong_AsLongAndOverflow(a[i], &over);
        if (over != 0 || v < INT_MIN || v > INT_MAX) return ok = false, 0;
        return static_cast<int>(v);
    }
    double number(int i) {
        if (!ok || !PyFloat_CheckExact(a[i])) return ok = false, 0.0;
        return PyFloat_AS_DOUBLE(a[i]);
    }
    void* workspace(int i, size_t* bytes) {
        if (!ok || !THPVariable_Check(a[i])) return ok = false, nullptr;
        const at::Tensor& t = THPVariable_Unpack(a[i]);
        if (!t.is_cuda() || t.layout() != at::kStrided || t.numel() == 0 || !here(t) || !t.is_contiguous())
            return ok = false, nullptr;
        *bytes = t.nbytes();
        return t.data_ptr();
    }
    uint32_t* status(int i) {
        return a[i] == Py_None ? nullptr : static_cast<uint32_t*>(pointer(i, at::kInt, {1}));
    }
    // None: the current one of the current device; else its handle.
    void* stream(int i) {
        if (a[i] == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
        if (!PyLong_CheckExact(a[i])) return ok = false, nullptr;
        void* s = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            ok = false;
        }
        return s;
    }

  private:
    const at::Tensor* fail() {
        ok = false;
        return nullptr;
    }
};

template <typename F>
PyObject* call(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "%zd arguments wanted, got %zd", want, n);
        return nullptr;
    }
    try {
        Args args{a};
        const int code = f(args);
        if (args.ok) return PyLong_FromLong(code);
    } catch (...) {  // a tensor that does not answer like an ordinary one
        PyErr_Clear();   // nor does what its answers in Python raised stay set
    }
    Py_RETURN_NONE;
}

// The entry point's status, the interpreter free meanwhile: a launch waits where the device's queue is full.
template <typename F>
int unlocked(F f) {
    PyThreadState* state = PyEval_SaveThread();
    const int code = static_cast<int>(f());
    PyEval_RestoreThread(state);
    return code;
}

// A rotation's sections: a tuple of at most four ints.
int sections(Args& g, int i, int* out) {
    if (!g.ok || !PyTuple_CheckExact(g.a[i]) || PyTuple_GET_SIZE(g.a[i]) > 4 || PyTuple_GET_SIZE(g.a[i]) < 1)
        return g.ok = false, 0;
    const int n = static_cast<int>(PyTuple_GET_SIZE(g.a[i]));
    for (int k = 0; k < n; ++k) {
        PyObject* item = PyTuple_GET_ITEM(g.a[i], k);
        Args one{&item};
        out[k] = one.integer(0);
        if (!one.ok) return g.ok = false, 0;
    }
    return n;
}

// (x, y, wq, wk, pos, q_heads, sections, base, eps, flags, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 11, [](Args& g) {
        int sec[4];
        const int axes = sections(g, 6, sec), q_heads = g.integer(5), flags = g.integer(9);
        const at::Tensor* x = g.tensor(0, at::kBFloat16);
        if (!g.ok || x->dim() != 3 || x->size(0) > INT_MAX || x->size(1) > INT_MAX || x->size(2) > INT_MAX)
            return g.ok = false, 0;
        const int64_t T = x->size(0), heads = x->size(1), d = x->size(2);
        long long ldx = 0, ldy = 0;
        auto* px = static_cast<const mp_bf16*>(g.rows(0, T, heads, d, &ldx));
        auto* py = static_cast<mp_bf16*>(g.rows(1, T, heads, d, &ldy));
        auto* wq = static_cast<const mp_bf16*>(g.pointer(2, at::kBFloat16, {d}));
        auto* wk = static_cast<const mp_bf16*>(g.pointer(3, at::kBFloat16, {d}));
        auto* pos = static_cast<const int32_t*>(g.pointer(4, at::kInt, {axes, T}));
        const double base = g.number(7), eps = g.number(8);
        void* s = g.stream(10);
        if (!g.ok) return 0;
        return unlocked([&] {
            return mp_qk_norm_rope(px, py, wq, wk, pos, T, heads, q_heads, d, ldx, ldy, axes, sec, base,
                                   static_cast<float>(eps), flags, s);
        });
    });
}

// (x, dy, dx, wq, wk, dwq, dwk, pos, workspace, q_heads, sections, base, eps, flags, stream)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 15, [](Args& g) {
        int sec[4];
        const int axes = sections(g, 10, sec), q_heads = g.integer(9), flags = g.integer(13);
        const at::Tensor* x = g.tensor(0, at::kBFloat16);
        if (!g.ok || x->dim() != 3 || x->size(0) > INT_MAX || x->size(1) > INT_MAX || x->size(2) > INT_MAX)
            return g.ok = false, 0;
        const int64_t T = x->size(0), heads = x->size(1), d = x->size(2);
        long long ldx = 0, ldg = 0, ldd = 0;
        auto* px = static_cast<const mp_bf16*>(g.rows(0, T, heads, d, &ldx));
        auto* pg = static_cast<const mp_bf16*>(g.rows(1, T, heads, d, &ldg));
        auto* pd = static_cast<mp_bf16*>(g.rows(2, T, heads, d, &ldd));
        auto* wq = static_cast<const mp_bf16*>(g.pointer(3, at::kBFloat16, {d}));
        auto* wk = static_cast<const mp_bf16*>(g.pointer(4, at::kBFloat16, {d}));
        auto* dwq = static_cast<float*>(g.pointer(5, at::kFloat, {d}));
        auto* dwk = static_cast<float*>(g.pointer(6, at::kFloat, {d}));
        auto* pos = static_cast<const int32_t*>(g.pointer(7, at::kInt, {axes, T}));
        size_t bytes = 0;
        void* ws = g.workspace(8, &bytes);
        const double base = g.number(11), eps = g.number(12);
        void* s = g.stream(14);
        if (!g.ok) return 0;
        return unlocked([&] {
            return mp_qk_norm_rope_bwd(px, pg, pd, wq, wk, dwq, dwk, pos, ws, bytes, T, heads, q_heads, d, ldx, ldg, ldd,
                                       axes, sec, base, static_cast<float>(eps), flags, s);
        });
    });
}

// The pool's tensors kc, vc, ks, vs, page_table from argument i on.
struct Pool {
    uint8_t* codes[2];
    float* scales[2];
    const int32_t* table;
    long long ld_codes[2], ld_scales[2];
    int pages, max_pages, page, kv, d, nseq;
};
bool pool(Args& g, int i, int table, Pool& p) {
    const at::Tensor* kc = g.tensor(i, at::kFloat8_e4m3fn);
    const at::Tensor* pt = g.tensor(table, at::kInt);
    if (!g.ok || kc->dim() != 4 || pt->dim() != 2 || !pt->is_contiguous() || kc->size(0) < 2) return g.ok = false;
    for (int k = 0; k < 4; ++k)
        if (kc->size(k) > INT_MAX) return g.ok = false;
    if (pt->size(0) > INT_MAX || pt->size(1) > INT_MAX) return g.ok = false;
    p.pages = kc->size(0), p.kv = kc->size(1), p.page = kc->size(2), p.d = kc->size(3);
    p.nseq = pt->size(0), p.max_pages = pt->size(1), p.table = static_cast<const int32_t*>(pt->data_ptr());
    for (int k = 0; k < 2; ++k) {
        const at::Tensor* c = g.tensor(i + k, at::kFloat8_e4m3fn);
        const at::Tensor* s = g.tensor(i + 2 + k, at::kFloat);
        if (!g.ok || c->sizes() != kc->sizes() || c->stride(3) != 1 || c->stride(2) != p.d ||
            c->stride(1) != static_cast<int64_t>(p.page) * p.d || s->dim() != 2 || s->size(0) != p.pages ||
            s->size(1) != p.kv || s->stride(1) != 1)
            return g.ok = false;
        p.codes[k] = static_cast<uint8_t*>(c->data_ptr());
        p.scales[k] = static_cast<float*>(s->data_ptr());
        p.ld_codes[k] = c->stride(0);
        p.ld_scales[k] = s->stride(0);
    }
    return true;
}

// (K, V, kc, vc, ks, vs, page_table, cu, start, max_n, d_status, stream); READ: K and V are written.
template <bool READ>
PyObject* kv_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 12, [](Args& g) {
        Pool p;
        if (!pool(g, 2, 6, p)) return 0;
        const at::Tensor* k = g.tensor(0, at::kBFloat16);
        if (!g.ok || k->dim() != 3 || k->size(0) > INT_MAX) return g.ok = false, 0;
        const int64_t T = k->size(0);
        long long ldk = 0, ldv = 0;
        auto* K = static_cast<mp_bf16*>(g.rows(0, T, p.kv, p.d, &ldk));
        auto* V = static_cast<mp_bf16*>(g.rows(1, T, p.kv, p.d, &ldv));
        auto* cu = static_cast<const int32_t*>(g.pointer(7, at::kInt, {p.nseq + 1ll}));
        auto* start = READ && g.a[8] == Py_None ? nullptr : static_cast<const int32_t*>(g.pointer(8, at::kInt, {p.nseq}));
        const int max_n = g.integer(9);
        uint32_t* status = g.status(10);
        void* s = g.stream(11);
        if (!g.ok) return 0;
        return unlocked([&] {
            if (READ)
                return mp_kv_cache_read(p.codes[0], p.codes[1], p.scales[0], p.scales[1], K, V, p.table, cu, start, p.nseq, T,
                                        max_n, p.kv, p.d, p.page, p.pages, p.max_pages, ldk, ldv, p.ld_codes[0],
                                        p.ld_codes[1], p.ld_scales[0], p.ld_scales[1], status, s);
            return mp_kv_cache_write(K, V, p.codes[0], p.codes[1], p.scales[0], p.scales[1], p.table, cu, start, p.nseq, T,
                                     max_n, p.kv, p.d, p.page, p.pages, p.max_pages, ldk, ldv, p.ld_codes[0], p.ld_codes[1],
                                     p.ld_scales[0], p.ld_scales[1], status, s);
        });
    });
}

// (Q, kc, vc, ks, vs, O, LSE, page_table, cu_q, lens, workspace, max_q, causal, scale, d_status, stream)
PyObject* attn_cache_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(a, n, 16, [](Args& g) {
        Pool p;
        if (!pool(g, 1, 7, p)) return 0;
        const at::Tensor* q = g.tensor(0, at::kBFloat16);
        if (!g.ok || q->dim() != 3 || q->size(0) > INT_MAX || q->size(1) > INT_MAX) return g.ok = false, 0;
        const int64_t T = q->size(0), heads = q->size(1);
        long long ldq = 0, ldo = 0;
        auto* Q = static_cast<const mp_bf16*>(g.rows(0, T, heads, p.d, &ldq));
        auto* O = static_cast<mp_bf16*>(g.rows(5, T, heads, p.d, &ldo));
        auto* lse = static_cast<float*>(g.pointer(6, at::kFloat, {heads, T}));
        auto* cu = static_cast<const int32_t*>(g.pointer(8, at::kInt, {p.nseq + 1ll}));
        auto* lens = static_cast<const int32_t*>(g.pointer(9, at::kInt, {p.nseq}));
        size_t bytes = 0;
        void* ws = g.workspace(10, &bytes);
        const int max_q = g.integer(11), causal = g.integer(12);
        const double scale = g.a[13] == Py_None ? 1.0 / std::sqrt(static_cast<double>(p.d)) : g.number(13);
        uint32_t* status = g.status(14);
        void* s = g.stream(15);
        if (!g.ok) return 0;
        return unlocked([&] {
            return mp_attn_cache_fwd(Q, p.codes[0], p.codes[1], p.scales[0], p.scales[1], O, lse, p.table, cu, lens, ws, bytes,
                                     p.nseq, T, max_q, heads, p.kv, p.d, p.page, p.pages, p.max_pages, ldq, ldo,
                                     p.ld_codes[0], p.ld_codes[1], p.ld_scales[0], p.ld_scales[1], causal,
                                     static_cast<float>(scale), status, s);
        });
    });
}

#define METHOD(name, f)                                                                 \
    {                                                                                   \
        name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, \
            "status, or None where an argument is out of the ordinary"                  \
    }
PyMethodDef methods[] = {METHOD("qk_norm_rope", qk_norm_rope),
                         METHOD("qk_norm_rope_bwd", qk_norm_rope_bwd),
                         METHOD("kv_cache_write", kv_cache<false>),
                         METHOD("kv_cache_read", kv_cache<true>),
                         METHOD("attn_cache_fwd", attn_cache_fwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mptp_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mptp_bind() { return PyModule_Create(&module); }
