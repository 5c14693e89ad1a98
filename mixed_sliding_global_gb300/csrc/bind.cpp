// bind.cpp -- the Python calls of the 4-bit cache and of sampling: arguments checked and marshalled
// natively. A decode step makes several of these calls per layer, and marshalled in the interpreter
// each took longer than its kernels: an attention call 12.1 us of host time, an append 10.4 (the
// Grace cores); here 3.3 and 3.0, most of it the launch.
//
// binding.py holds the functions' signatures and documentation and passes every argument by
// position. Nothing is kept from one call to the next. Returns the C call's status; a check that
// fails raises before any launch.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "gemma_attn.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const char* text) {
    PyErr_SetString(type, text);
    throw Raised{};
}

struct Ref {  // an owned reference
    PyObject* o = nullptr;
    Ref() = default;
    explicit Ref(PyObject* p) : o(p) {
        if (!o) throw Raised{};
    }
    Ref(const Ref&) = delete;
    Ref& operator=(Ref&& r) {
        std::swap(o, r.o);
        return *this;
    }
    ~Ref() { Py_XDECREF(o); }
};

int to_int(PyObject* o) {
    const long v = PyLong_AsLong(o);  // (through __index__)
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT_MIN || v > INT_MAX) raise(PyExc_OverflowError, "argument does not fit 32 bits");
    return (int)v;
}
float to_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
}
bool to_bool(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}
// A tensor, or nullptr for None.
const at::Tensor* optional(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, "expected a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o) {
    const at::Tensor* t = optional(o);
    if (!t) raise(PyExc_TypeError, "expected a tensor");
    return *t;
}
int dtype_code(const at::Tensor& t) {
    if (t.scalar_type() == at::kBFloat16) return GEMMA_BF16;
    if (t.scalar_type() == at::kFloat) return GEMMA_FP32;
    raise(PyExc_TypeError, "unsupported dtype: bf16 or fp32 expected");
}
// Index of a tensor's device, which must be the current one: launches go there.
int current(const at::Tensor& t) {
    if (!t.is_cuda()) raise(PyExc_ValueError, "expected a CUDA tensor");
    const int dev = t.get_device();
    if (dev != c10::cuda::current_device())
        raise(PyExc_ValueError, "tensors of another device than the current one");
    return dev;
}
// Address of a contiguous tensor on device dev.
void* on(int dev, const at::Tensor* t) {
    if (!t) return nullptr;
    if (!t->is_cuda() || t->get_device() != dev)
        raise(PyExc_ValueError, "expected tensors of one CUDA device");
    if (!t->is_contiguous()) raise(PyExc_ValueError, "expected a contiguous tensor");
    return t->data_ptr();
}
void* on(int dev, const at::Tensor& t) { return on(dev, &t); }
size_t bytes(const at::Tensor* t) { return t ? t->nbytes() : 0; }
// torch's current stream, or the raw handle given
void* stream_of(PyObject* o, int dev) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Raised{};
    return p;
}
uint32_t* error_word(int dev, PyObject* o) {
    const at::Tensor* t = optional(o);
    if (t && t->nbytes() < 4) raise(PyExc_ValueError, "device_error must hold 32 bits");
    return static_cast<uint32_t*>(on(dev, t));
}

// The layer whose cache `layer` reads, or -1 for a layer or a map that the C calls refuse.
int owner_of(PyObject* map, int layer) {
    const Py_ssize_t n = PySequence_Size(map);
    if (n < 0) throw Raised{};
    auto owner = [&](Py_ssize_t i) {
        Ref r(PySequence_GetItem(map, i));
        return to_int(r.o);
    };
    const int o = layer >= 0 && layer < n ? owner(layer) : -1;
    return o < 0 || o > layer || owner(o) != o ? -1 : o;
}

// The owner layer's 4-bit cache as a model of that one layer, and where its rows lie.
struct Cache {
    void *kc, *ks, *vc, *vs;
    const int32_t zero = 0;
    const int32_t* table = nullptr;
    int max_pages = 0, page = 0, n_pages = 0, cap = 0, dev = 0;
    Ref held[4];

    // a: k_codes, k_scales, v_codes, v_scales; o: the owner layer
    Cache(PyObject* const* a, int o, bool k_eq_v, int64_t d, int64_t n_kv, int64_t batch, PyObject* table_,
          const at::Tensor& of) {
        const at::Tensor* t[4] = {nullptr, nullptr, nullptr, nullptr};
        for (int i = 0; i < (k_eq_v ? 2 : 4); ++i) {
            if (a[i] != Py_None) {
                held[i] = Ref(PySequence_GetItem(a[i], o));
                t[i] = optional(held[i].o);
            }
            if (!t[i])
                raise(PyExc_ValueError,
                      i < 2 ? "the owner layer has no cache" : "the layer needs a V cache");
        }
        const auto shape = t[0]->sizes();
        if (shape.size() != 4 || shape[1] != n_kv || shape[3] * 2 != d)
            raise(PyExc_ValueError, "codes must be [batch][n_kv][capacity][head_dim / 2]");
        for (int i = 0; i < 4; ++i) {
            if (!t[i]) continue;
            if (t[i]->scalar_type() != (i & 1 ? at::kBFloat16 : at::kByte))
                raise(PyExc_TypeError, "4-bit caches hold uint8 codes and bf16 scales");
            const auto s = t[i]->sizes();
            if (s.size() != 4 || s[0] != shape[0] || s[1] != n_kv || s[2] != shape[2] ||
                s[3] != (i & 1 ? d / 64 : d / 2))
                raise(PyExc_ValueError,
                      i & 1 ? "scales must be [batch][n_kv][capacity][head_dim / 64]"
                            : "codes of K and V must have one shape");
        }
        if (shape[2] > INT_MAX || shape[0] > INT_MAX)
            raise(PyExc_ValueError, "cache sizes must fit 32 bits");
        const at::Tensor* bt = optional(table_);
        if (!bt) {
            if (shape[0] != batch)
                raise(PyExc_ValueError, "the cache must have one entry per sequence");
        } else if (bt->scalar_type() != at::kInt || bt->dim() != 2 || bt->size(0) != batch ||
                   bt->size(1) > INT_MAX) {
            raise(PyExc_ValueError, "block_table must be int32 [batch][max_pages]");
        }
        dev = current(of);
        kc = on(dev, t[0]);
        ks = on(dev, t[1]);
        vc = on(dev, t[2]);
        vs = on(dev, t[3]);
        if (bt) {
            table = static_cast<const int32_t*>(on(dev, bt));
            max_pages = (int)bt->size(1);
            page = (int)shape[2];
            n_pages = (int)shape[0];
        } else {
            cap = (int)shape[2];
        }
    }
};

int checked(int64_t v) {
    if (v < INT_MIN || v > INT_MAX) raise(PyExc_ValueError, "tensor sizes must fit 32 bits");
    return (int)v;
}
void is_int32(const at::Tensor& t, int64_t n, const char* text) {
    if (t.scalar_type() != at::kInt || t.numel() != n) raise(PyExc_ValueError, text);
}

template <class F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
    try {
        if (given != wanted) raise(PyExc_TypeError, "wrong number of arguments");
        return PyLong_FromLong(f());
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
        return nullptr;
    }
}

// k_codes, k_scales, v_codes, v_scales, owner_map, layer, k_rows, v_rows, pos, k_eq_v, kind,
// block_table, device_error, stream
int rows(PyObject* const* a, bool append) {
    const int layer = to_int(a[5]), owner = owner_of(a[4], layer);
    if (owner < 0) return GEMMA_ERR_INVALID_ARG;
    if (append && owner != layer) return GEMMA_OK;  // a shared layer writes no cache
    const at::Tensor& k = tensor(a[6]);
    if (k.dim() != 4) raise(PyExc_ValueError, "rows must be [batch][n][n_kv][head_dim]");
    const at::Tensor& pos = tensor(a[8]);
    is_int32(pos, k.size(0), "positions must be int32 [batch]");
    const bool k_eq_v = to_bool(a[9]);
    const at::Tensor* v = k_eq_v ? nullptr : optional(a[7]);
    if (!k_eq_v && (!v || v->sizes() != k.sizes() || v->scalar_type() != k.scalar_type()))
        raise(PyExc_ValueError, "K and V rows must have one shape and type");
    Cache c(a, owner, k_eq_v, k.size(3), k.size(2), k.size(0), a[11], k);
    const int B = checked(k.size(0)), n = checked(k.size(1)), n_kv = checked(k.size(2)),
              d = checked(k.size(3)), kind = to_int(a[10]);
    const auto dt = (gemma_dtype)dtype_code(k);
    void *kp = on(c.dev, k), *vp = on(c.dev, v);
    const auto* pp = static_cast<const int32_t*>(on(c.dev, pos));
    uint32_t* err = error_word(c.dev, a[12]);
    void* st = stream_of(a[13], c.dev);
    int status;
    Py_BEGIN_ALLOW_THREADS
    if (append)
        status = gemma_kv_append_q4(&c.kc, &c.ks, &c.vc, &c.vs, &c.zero, 1, 0, kp, vp, pp, c.table,
                                    c.max_pages, c.page, c.n_pages, B, n, (gemma_layer_kind)kind,
                                    n_kv, d, c.cap, k_eq_v, dt, err, st);
    else
        status = gemma_kv_read_q4(&c.kc, &c.ks, &c.vc, &c.vs, &c.zero, 1, 0, kp, vp, pp, c.table,
                                  c.max_pages, c.page, c.n_pages, B, n, (gemma_layer_kind)kind,
                                  n_kv, d, c.cap, k_eq_v, dt, err, st);
    Py_END_ALLOW_THREADS
    return status;
}
PyObject* append_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] { return rows(a, true); });
}
PyObject* read_q4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&] { return rows(a, false); });
}

// k_codes, k_scales, v_codes, v_scales, owner_map, layer, out, q, seq_lens, max_seq_len, kind,
// window, n_kv, k_eq_v, scale, softcap, block_table, workspace, device_error, stream
PyObject* attn_q4(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 20, [&]() -> int {
        const int owner = owner_of(a[4], to_int(a[5]));
        if (owner < 0) return GEMMA_ERR_INVALID_ARG;
        const at::Tensor &out = tensor(a[6]), &q = tensor(a[7]), &lens = tensor(a[8]);
        if (q.dim() != 4 || out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
            raise(PyExc_ValueError, "q and out must be [batch][n_new][n_q][head_dim] of one type");
        is_int32(lens, q.size(0), "seq_lens must be int32 [batch]");
        const int msl = to_int(a[9]), kind = to_int(a[10]), window = to_int(a[11]),
                  n_kv = to_int(a[12]);
        const bool k_eq_v = to_bool(a[13]);
        const float scale = to_float(a[14]), softcap = to_float(a[15]);
        Cache c(a, owner, k_eq_v, q.size(3), n_kv, q.size(0), a[16], q);
        const at::Tensor* ws = optional(a[17]);
        const int B = checked(q.size(0)), n = checked(q.size(1)), n_q = checked(q.size(2)),
                  d = checked(q.size(3));
        const auto dt = (gemma_dtype)dtype_code(q);
        void *op = on(c.dev, out), *qp = on(c.dev, q), *wp = on(c.dev, ws);
        const auto* lp = static_cast<const int32_t*>(on(c.dev, lens));
        uint32_t* err = error_word(c.dev, a[18]);
        void* st = stream_of(a[19], c.dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_attn_q4(op, qp, &c.kc, &c.ks, &c.vc, &c.vs, &c.zero, 1, 0, lp, c.table,
                               c.max_pages, c.page, c.n_pages, msl, n, B, (gemma_layer_kind)kind,
                               window, n_q, n_kv, d, k_eq_v, c.cap, scale, softcap, dt, wp,
                               bytes(ws), err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// logits, token_out, uniform, temperature, top_k, top_p, min_p, softcap, workspace, device_error,
// stream
PyObject* logit_sample(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&] {
        const at::Tensor& x = tensor(a[0]);
        if (x.dim() != 2) raise(PyExc_ValueError, "logits must be [B][V]");
        // token_out, uniform, temperature, top_k, top_p, min_p
        const at::Tensor* t[6];
        for (int i = 0; i < 6; ++i) {
            t[i] = i < 2 ? &tensor(a[1 + i]) : optional(a[1 + i]);
            const bool ints = i == 0 || i == 3;
            if (t[i] && (t[i]->scalar_type() != (ints ? at::kInt : at::kFloat) ||
                         t[i]->numel() != x.size(0)))
                raise(PyExc_TypeError, ints ? "token_out and top_k must be int32 [batch]"
                                            : "uniform, temperature, top_p and min_p must be fp32 "
                                              "[batch]");
        }
        const float softcap = to_float(a[7]);
        const int dev = current(x);
        const at::Tensor* ws = optional(a[8]);
        const int B = checked(x.size(0)), V = checked(x.size(1));
        const auto dt = (gemma_dtype)dtype_code(x);
        void *xp = on(dev, x), *wp = on(dev, ws), *p[6];
        for (int i = 0; i < 6; ++i) p[i] = on(dev, t[i]);
        uint32_t* err = error_word(dev, a[9]);
        void* st = stream_of(a[10], dev);
        auto f = [](void* v) { return static_cast<const float*>(v); };
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_logit_sample(xp, B, V, dt, softcap, f(p[2]),
                                    static_cast<const int32_t*>(p[3]), f(p[4]), f(p[5]), f(p[1]),
                                    static_cast<int32_t*>(p[0]), wp, bytes(ws), err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {
    {"kv_append_q4", fast(append_q4), METH_FASTCALL, nullptr},
    {"kv_read_q4", fast(read_q4), METH_FASTCALL, nullptr},
    {"attn_q4", fast(attn_q4), METH_FASTCALL, nullptr},
    {"logit_sample", fast(logit_sample), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
