// bind.cpp -- the Python calls of the 4-bit cache, of sampling, of drafted trees and of pages:
// arguments checked and marshalled natively. A decode step makes several of these calls per layer, and
// marshalled in the interpreter each took longer than its kernels: an attention call 12.1 us of host
// time, an append 10.4 (the Grace cores); here 3.3 and 3.0, most of it the launch.
//
// binding.py holds the functions' signatures and documentation and passes every argument by
// position. Nothing is kept from one call to the next. Returns the C call's status; a check that
// fails raises before any launch.
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <vector>

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

// ---------------------------------------------------------------------------------------------
// drafted trees and pages
// ---------------------------------------------------------------------------------------------
const int32_t* ints(int dev, const at::Tensor* t, int64_t n, const char* text) {
    if (t) is_int32(*t, n, text);
    return static_cast<const int32_t*>(on(dev, t));
}
int32_t* ints_out(int dev, const at::Tensor* t, int64_t n, const char* text) {
    return const_cast<int32_t*>(ints(dev, t, n, text));
}
// A block table of `batch` sequences (batch < 0: of any number).
void is_table(const at::Tensor& t, int64_t batch) {
    if (t.scalar_type() != at::kInt || t.dim() != 2 || (batch >= 0 && t.size(0) != batch))
        raise(PyExc_ValueError, "block_table must be int32 [batch][max_pages]");
}

// k_cache, v_cache, owner_map, layer, out, q, seq_lens, parents, max_seq_len, kind, window, n_kv,
// k_eq_v, scale, softcap, n_real, block_table, workspace, device_error, stream
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 20, [&]() -> int {
        const int owner = owner_of(a[2], to_int(a[3]));
        if (owner < 0) return GEMMA_ERR_INVALID_ARG;
        const at::Tensor &out = tensor(a[4]), &q = tensor(a[5]), &lens = tensor(a[6]),
                         &parents = tensor(a[7]);
        if (q.dim() != 4 || out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
            raise(PyExc_ValueError, "q and out must be [batch][n_nodes][n_q][head_dim] of one type");
        const int B = checked(q.size(0)), n = checked(q.size(1)), n_q = checked(q.size(2)),
                  d = checked(q.size(3));
        const int msl = to_int(a[8]), kind = to_int(a[9]), window = to_int(a[10]),
                  n_kv = to_int(a[11]);
        const bool k_eq_v = to_bool(a[12]);
        const float scale = to_float(a[13]), softcap = to_float(a[14]);
        const auto dt = (gemma_dtype)dtype_code(q);
        const int dev = current(q);
        const at::Tensor *bt = optional(a[16]), *ws = optional(a[17]);
        Ref held[2];
        const at::Tensor* c[2] = {nullptr, nullptr};
        for (int i = 0; i < (k_eq_v ? 1 : 2); ++i) {
            if (a[i] != Py_None) {
                held[i] = Ref(PySequence_GetItem(a[i], owner));
                c[i] = optional(held[i].o);
            }
            if (!c[i])
                raise(PyExc_ValueError,
                      i ? "the layer needs a V cache" : "the owner layer has no cache");
            const auto s = c[i]->sizes();
            if (s.size() != 4 || s[1] != n_kv || s[3] != d || (i && s != c[0]->sizes()) ||
                (!bt && s[0] != B))
                raise(PyExc_ValueError, "caches must be [batch][n_kv][capacity][head_dim]");
            if (c[i]->scalar_type() != q.scalar_type())
                raise(PyExc_TypeError, "caches and q must have one type");
        }
        if (bt) is_table(*bt, B);
        const int rows = checked(c[0]->size(0)), slots = checked(c[0]->size(2)),
                  max_pages = bt ? checked(bt->size(1)) : 0;
        const void *kp = on(dev, c[0]), *vp = on(dev, c[1]);
        const int32_t zero = 0;
        const auto* lp = ints(dev, &lens, B, "seq_lens must be int32 [batch]");
        const auto* pp = ints(dev, &parents, (int64_t)B * n, "parents must be int32 [batch][n_nodes]");
        const auto* rp = ints(dev, optional(a[15]), B, "n_real must be int32 [batch]");
        const auto* tp = static_cast<const int32_t*>(on(dev, bt));
        void *op = on(dev, out), *qp = on(dev, q), *wp = on(dev, ws);
        uint32_t* err = error_word(dev, a[18]);
        void* st = stream_of(a[19], dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_attn_tree(op, qp, &kp, &vp, &zero, 1, 0, lp, pp, rp, tp, max_pages,
                                 bt ? slots : 0, bt ? rows : 0, msl, n, B, (gemma_layer_kind)kind,
                                 window, n_q, n_kv, d, k_eq_v, bt ? 0 : slots, scale, softcap, dt,
                                 wp, bytes(ws), err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// tokens, parents, next, path_out, n_keep_out, token_out, n_real, seq_lens, lens_out,
// device_error, stream
PyObject* tree_accept(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 11, [&] {
        const at::Tensor& tokens = tensor(a[0]);
        if (tokens.dim() != 2) raise(PyExc_ValueError, "tokens must be [batch][n_nodes]");
        const int B = checked(tokens.size(0)), n = checked(tokens.size(1)), dev = current(tokens);
        const int64_t all = tokens.numel();
        const char *nodes = "tokens, parents, next and path_out must be int32 [batch][n_nodes]",
                   *seqs = "n_keep_out, token_out, n_real, seq_lens and lens_out must be int32 [batch]";
        const auto *tk = ints(dev, &tokens, all, nodes), *pa = ints(dev, &tensor(a[1]), all, nodes),
                   *nx = ints(dev, &tensor(a[2]), all, nodes);
        auto* path = ints_out(dev, &tensor(a[3]), all, nodes);
        auto *keep = ints_out(dev, &tensor(a[4]), B, seqs), *tok = ints_out(dev, &tensor(a[5]), B, seqs);
        const auto *real = ints(dev, optional(a[6]), B, seqs), *lens = ints(dev, optional(a[7]), B, seqs);
        auto* lens_out = ints_out(dev, optional(a[8]), B, seqs);
        uint32_t* err = error_word(dev, a[9]);
        void* st = stream_of(a[10], dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_tree_accept(tk, pa, nx, real, lens, B, n, path, keep, tok, lens_out, err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// Caches or pools of one call: their addresses, KV heads and bytes per row.
struct Rows {
    std::vector<void*> p;
    std::vector<int32_t> n_kv, row_bytes;
    int64_t outer = 0, slots = 0;  // sequences or pages; slots of a head
    int dev = -1;

    explicit Rows(PyObject* list) {
        const Py_ssize_t n = PySequence_Size(list);
        if (n < 0) throw Raised{};
        for (Py_ssize_t i = 0; i < n; ++i) {
            Ref r(PySequence_GetItem(list, i));
            const at::Tensor& t = tensor(r.o);
            if (t.dim() < 4 || t.numel() == 0)
                raise(PyExc_ValueError, "caches must be [batch][n_kv][capacity][row]");
            if (i == 0) {
                dev = current(t);
                outer = t.size(0);
                slots = t.size(2);
            } else if (t.size(0) != outer || t.size(2) != slots) {
                raise(PyExc_ValueError, "the caches of a call must have the same sizes");
            }
            p.push_back(on(dev, t));
            n_kv.push_back(checked(t.size(1)));
            row_bytes.push_back(checked((int64_t)(t.nbytes() / (outer * t.size(1) * slots))));
        }
    }
};

// caches, write_pos, path, n_keep, kind, block_table, device_error, stream
PyObject* kv_keep(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> int {
        const at::Tensor &pos = tensor(a[1]), &path = tensor(a[2]), &keep = tensor(a[3]);
        const int kind = to_int(a[4]);
        Rows c(a[0]);
        if (c.p.empty()) return GEMMA_OK;
        for (size_t i = 1; i < c.p.size(); ++i)
            if (c.n_kv[i] != c.n_kv[0] || c.row_bytes[i] != c.row_bytes[0])
                raise(PyExc_ValueError, "the caches of a call must have the same sizes");
        if (path.dim() != 2) raise(PyExc_ValueError, "path must be int32 [batch][n_nodes]");
        const int B = checked(path.size(0)), n = checked(path.size(1));
        const at::Tensor* bt = optional(a[5]);
        if (bt) is_table(*bt, B);
        else if (c.outer != B)
            raise(PyExc_ValueError, "the cache must have one entry per sequence");
        const int max_pages = bt ? checked(bt->size(1)) : 0, outer = checked(c.outer),
                  slots = checked(c.slots);
        const auto *wp = ints(c.dev, &pos, B, "write_pos must be int32 [batch]"),
                   *pp = ints(c.dev, &path, path.numel(), "path must be int32 [batch][n_nodes]"),
                   *kp = ints(c.dev, &keep, B, "n_keep must be int32 [batch]");
        const auto* tp = static_cast<const int32_t*>(on(c.dev, bt));
        uint32_t* err = error_word(c.dev, a[6]);
        void* st = stream_of(a[7], c.dev);
        const int n_caches = checked((int64_t)c.p.size());
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_kv_keep(c.p.data(), n_caches, wp, pp, kp, tp, max_pages, bt ? slots : 0,
                               bt ? outer : 0, B, n, (gemma_layer_kind)kind, c.n_kv[0],
                               bt ? 0 : slots, c.row_bytes[0], err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// A block table and its pages' reference counts.
struct Table {
    int32_t *table, *refs;
    int batch, max_pages, n_pages, dev;
    Table(PyObject* table_, PyObject* refs_) {
        const at::Tensor &t = tensor(table_), &r = tensor(refs_);
        is_table(t, -1);
        dev = current(t);
        batch = checked(t.size(0));
        max_pages = checked(t.size(1));
        n_pages = checked(r.numel());
        table = static_cast<int32_t*>(on(dev, t));
        refs = ints_out(dev, &r, n_pages, "page_refs must be int32 [n_pages]");
    }
};

// block_table, page_refs, page_size, keep_from, keep_to, device_error, stream
PyObject* pages_free(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 7, [&] {
        const Table t(a[0], a[1]);
        const int page = to_int(a[2]);
        const auto *from = ints(t.dev, optional(a[3]), t.batch, "keep_from must be int32 [batch]"),
                   *to = ints(t.dev, optional(a[4]), t.batch, "keep_to must be int32 [batch]");
        uint32_t* err = error_word(t.dev, a[5]);
        void* st = stream_of(a[6], t.dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_pages_free(t.table, t.max_pages, page, t.n_pages, t.refs, from, to, t.batch,
                                  err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// block_table, page_refs, seq_lens, src, dst, page_size, device_error, stream
PyObject* pages_fork(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&] {
        const Table t(a[0], a[1]);
        const at::Tensor &src = tensor(a[3]), &dst = tensor(a[4]);
        const int n = checked(src.numel()), page = to_int(a[5]);
        auto* lens = ints_out(t.dev, &tensor(a[2]), t.batch, "seq_lens must be int32 [batch]");
        const auto *sp = ints(t.dev, &src, n, "src and dst must be int32 [n]"),
                   *dp = ints(t.dev, &dst, n, "src and dst must be int32 [n]");
        uint32_t* err = error_word(t.dev, a[6]);
        void* st = stream_of(a[7], t.dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_pages_fork(t.table, t.max_pages, page, t.n_pages, t.refs, lens, sp, dp, n,
                                  t.batch, err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// The pools of a call, on the device of its table and with its pages.
int page_size_of(const Rows& c, const Table& t) {
    if (c.p.empty()) raise(PyExc_ValueError, "expected the pools of the block table");
    if (c.dev != t.dev || c.outer != t.n_pages)
        raise(PyExc_ValueError, "pools must be [n_pages][n_kv][page_size][row], one count per page");
    return checked(c.slots);
}

// pools, block_table, page_refs, seq_lens, n_add, workspace, device_error, stream
PyObject* pages_reserve(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&] {
        const Table t(a[1], a[2]);
        Rows c(a[0]);
        const int page = page_size_of(c, t), n = checked((int64_t)c.p.size());
        const auto *lens = ints(t.dev, &tensor(a[3]), t.batch, "seq_lens must be int32 [batch]"),
                   *add = ints(t.dev, &tensor(a[4]), t.batch, "n_add must be int32 [batch]");
        const at::Tensor* ws = optional(a[5]);
        void* wp = on(t.dev, ws);
        uint32_t* err = error_word(t.dev, a[6]);
        void* st = stream_of(a[7], t.dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_pages_reserve(c.p.data(), c.n_kv.data(), c.row_bytes.data(), n, t.table,
                                     t.max_pages, page, t.n_pages, t.refs, lens, add, t.batch, wp,
                                     bytes(ws), err, st);
        Py_END_ALLOW_THREADS
        return status;
    });
}

// pools, block_table, page_refs, n_used, workspace, device_error, stream
PyObject* pages_compact(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded(nargs, 7, [&] {
        const Table t(a[1], a[2]);
        Rows c(a[0]);
        const int page = page_size_of(c, t), n = checked((int64_t)c.p.size());
        auto* used = ints_out(t.dev, optional(a[3]), 1, "n_used must be one int32");
        const at::Tensor* ws = optional(a[4]);
        void* wp = on(t.dev, ws);
        uint32_t* err = error_word(t.dev, a[5]);
        void* st = stream_of(a[6], t.dev);
        int status;
        Py_BEGIN_ALLOW_THREADS
        status = gemma_pages_compact(c.p.data(), c.n_kv.data(), c.row_bytes.data(), n, t.table,
                                     t.max_pages, page, t.n_pages, t.refs, used, t.batch, wp,
                                     bytes(ws), err, st);
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
    {"attn_tree", fast(attn_tree), METH_FASTCALL, nullptr},
    {"tree_accept", fast(tree_accept), METH_FASTCALL, nullptr},
    {"kv_keep", fast(kv_keep), METH_FASTCALL, nullptr},
    {"pages_free", fast(pages_free), METH_FASTCALL, nullptr},
    {"pages_fork", fast(pages_fork), METH_FASTCALL, nullptr},
    {"pages_reserve", fast(pages_reserve), METH_FASTCALL, nullptr},
    {"pages_compact", fast(pages_compact), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
