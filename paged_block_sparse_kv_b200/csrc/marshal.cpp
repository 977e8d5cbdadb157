// marshal.cpp -- argument marshalling of the 8-bit cache and page calls for Python.
//
// A call of these operators takes 10 to 20 tensors, and its kernels a few microseconds: checking
// types, shapes and devices from Python costs more than they do.  This module does it through
// torch's C++ interface and calls the C entry points of libvx (include/vx.h), whose addresses
// vx.py hands over with bind().  It computes nothing and keeps nothing between calls.  Every
// function takes positional arguments, as vx.py passes them, and returns the vx_status; a bad
// argument raises TypeError or ValueError, as in vx.py.  A decode call's host time went from 38
// to 11 us with it.
#include <Python.h>

#include <initializer_list>
#include <stdexcept>
#include <string>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/vx.h"

namespace {

struct TypeErr : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct ValueErr : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct PyErr {};  // a Python exception is already set

using c10::ScalarType;

constexpr int64_t ANY = -1;  // an extent that is not checked

struct {
    decltype(&vx_quant_update) quant_update;
    decltype(&vx_sparse_decode_quant) sparse_decode_quant;
    decltype(&vx_block_topk_decode_quant) block_topk_decode_quant;
    decltype(&vx_block_topk_decode_append_quant) block_topk_decode_append_quant;
    decltype(&vx_copy_pages) copy_pages;
    decltype(&vx_update_table) update_table;
    decltype(&vx_compact_pages) compact_pages;
} fn;

// a new reference, dropped at scope's end
struct Ref {
    PyObject *p;
    explicit Ref(PyObject *o) : p(o) {
        if (!p) throw PyErr();
    }
    Ref(const Ref &) = delete;
    ~Ref() { Py_DECREF(p); }
};

PyObject *name_of(const char *s) {
    PyObject *o = PyUnicode_InternFromString(s);
    if (!o) throw PyErr();
    return o;
}

int64_t as_int(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PyErr();
    return v;
}

int32_t as_i32(PyObject *o, const char *name) {
    const int64_t v = as_int(o);
    if (v < INT32_MIN || v > INT32_MAX) throw ValueErr(std::string(name) + " does not fit 32 bits");
    return static_cast<int32_t>(v);
}

float as_float(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PyErr();
    return static_cast<float>(v);
}

std::string dims(c10::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + (s[i] == ANY ? std::string("any") : std::to_string(s[i]));
    return t + ")";
}

// The tensors of one call: checks each, and that all lie on one CUDA device.
struct Call {
    int device = -2;  // -2: none seen yet, -1: not a CUDA tensor
    bool mixed = false;

    const at::Tensor *tensor(PyObject *o, const char *name) {
        if (!THPVariable_Check(o)) throw TypeErr(std::string(name) + " must be a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        const int d = t.is_cuda() ? t.get_device() : -1;
        if (device == -2) device = d;
        else if (d != device) mixed = true;
        if (!t.is_contiguous()) throw ValueErr("tensors passed to libvx must be contiguous");
        return &t;
    }
    template <typename T = void>
    T *ptr(PyObject *o, const char *name, ScalarType type, std::initializer_list<int64_t> shape) {
        if (o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, name);
        if (t->scalar_type() != type)
            throw TypeErr(std::string(name) + ": expected " + c10::toString(type) + ", got " + c10::toString(t->scalar_type()));
        const auto have = t->sizes();
        bool same = have.size() == shape.size();
        size_t i = 0;
        for (const int64_t want : shape) {
            if (!same) break;
            same = want == ANY || have[i] == want;
            ++i;
        }
        if (!same) throw ValueErr(std::string(name) + " has shape " + dims(have) + ", expected " + dims(shape));
        return static_cast<T *>(t->data_ptr());
    }
    template <typename T = void>
    T *flat(PyObject *o, const char *name, ScalarType type) {  // any shape
        if (o == Py_None) return nullptr;
        const at::Tensor *t = tensor(o, name);
        if (t->scalar_type() != type)
            throw TypeErr(std::string(name) + ": expected " + c10::toString(type) + ", got " + c10::toString(t->scalar_type()));
        return static_cast<T *>(t->data_ptr());
    }
    void *workspace(PyObject *o, size_t *bytes) {
        const at::Tensor *t = tensor(o, "ws");
        *bytes = t->nbytes();
        return t->data_ptr();
    }
    int32_t *err(PyObject *o) { return flat<int32_t>(o, "err", ScalarType::Int); }

    // Run the call on the tensors' device, on `stream` (None, or (handle, device index))
    template <typename F>
    PyObject *run(PyObject *stream, F f) {
        if (device < 0) throw ValueErr("libvx works on CUDA tensors");
        if (mixed) throw ValueErr("tensors on several devices in one call");
        void *s;
        if (stream == Py_None) {
            s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        } else {
            if (!PyTuple_Check(stream) || PyTuple_GET_SIZE(stream) != 2) throw TypeErr("stream");
            if (as_int(PyTuple_GET_ITEM(stream, 1)) != device) throw ValueErr("the stream lies on another device");
            s = PyLong_AsVoidPtr(PyTuple_GET_ITEM(stream, 0));
            if (!s && PyErr_Occurred()) throw PyErr();
        }
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != device) guard.set_index(static_cast<c10::DeviceIndex>(device));
        vx_status st;
        Py_BEGIN_ALLOW_THREADS;
        st = f(s);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(st);
    }
};

struct Geo : vx_geometry {
    explicit Geo(PyObject *o) {
        static PyObject *n[8] = {name_of("batch"),       name_of("num_q_heads"), name_of("num_kv_heads"),
                                 name_of("head_dim_qk"), name_of("head_dim_v"),  name_of("page_size"),
                                 name_of("mla_shared_kv"), name_of("num_pool_pages")};
        int32_t *to[6] = {&batch, &num_q_heads, &num_kv_heads, &head_dim_qk, &head_dim_v, &page_size};
        for (int i = 0; i < 6; ++i) {
            Ref a(PyObject_GetAttr(o, n[i]));
            *to[i] = as_i32(a.p, "a geometry field");
        }
        Ref m(PyObject_GetAttr(o, n[6]));
        mla_shared_kv = PyObject_IsTrue(m.p) == 1;
        Ref p(PyObject_GetAttr(o, n[7]));
        num_pool_pages = as_int(p.p);
    }
};

struct Table : vx_page_table {
    int64_t entries;  // of page_indices
    Table(Call &c, PyObject *o, int64_t rows) {
        static PyObject *n[4] = {name_of("page_ptr"), name_of("page_indices"), name_of("seq_lens"), name_of("max_pages")};
        Ref p(PyObject_GetAttr(o, n[0])), i(PyObject_GetAttr(o, n[1])), l(PyObject_GetAttr(o, n[2])),
            m(PyObject_GetAttr(o, n[3]));
        page_ptr = c.ptr<int32_t>(p.p, "page_ptr", ScalarType::Int, {rows});
        page_indices = c.flat<int32_t>(i.p, "page_indices", ScalarType::Int);
        entries = i.p == Py_None ? 0 : THPVariable_Unpack(i.p).numel();
        seq_lens = c.ptr<int32_t>(l.p, "seq_lens", ScalarType::Int, {rows});
        max_pages = as_i32(m.p, "max_pages");
    }
};

// [a, a + an) and [b, b + bn) int32 entries have one in common
bool overlap(const int32_t *a, int64_t an, const int32_t *b, int64_t bn) { return a < b + bn && b < a + an; }

ScalarType type_of(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw TypeErr(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o).scalar_type();
}

struct Cache : vx_quant_cache {
    Cache(Call &c, PyObject *o, const Geo &g) {
        static PyObject *n[4] = {name_of("k_cache"), name_of("v_cache"), name_of("k_scale"), name_of("v_scale")};
        Ref k(PyObject_GetAttr(o, n[0])), v(PyObject_GetAttr(o, n[1])), ks(PyObject_GetAttr(o, n[2])),
            vs(PyObject_GetAttr(o, n[3]));
        const ScalarType t = type_of(k.p, "k_cache");
        if (t != ScalarType::Char && t != ScalarType::Float8_e4m3fn)
            throw TypeErr(std::string("k_cache must be int8 or float8_e4m3fn, got ") + c10::toString(t));
        format = t == ScalarType::Char ? VX_QUANT_INT8 : VX_QUANT_E4M3;
        const int64_t N = g.num_pool_pages, H = g.num_kv_heads, P = g.page_size, D = g.head_dim_qk;
        k_cache = c.ptr(k.p, "k_cache", t, {N, H, P, D});
        v_cache = c.ptr(v.p, "v_cache", t, {N, H, P, D});
        k_scale = c.ptr<float>(ks.p, "k_scale", ScalarType::Float, {N, H});
        v_scale = c.ptr<float>(vs.p, "v_scale", ScalarType::Float, {N, H});
    }
};

struct Pool : vx_page_pool {
    ScalarType type;
    Pool(Call &c, PyObject *o, const Geo &g) {
        static PyObject *n[5] = {name_of("k_cache"), name_of("v_cache"), name_of("centroids"), name_of("k_scale"),
                                 name_of("v_scale")};
        Ref k(PyObject_GetAttr(o, n[0])), v(PyObject_GetAttr(o, n[1])), e(PyObject_GetAttr(o, n[2])),
            ks(PyObject_GetAttr(o, n[3])), vs(PyObject_GetAttr(o, n[4]));
        type = type_of(k.p, "k_cache");
        const bool codes = type == ScalarType::Char || type == ScalarType::Float8_e4m3fn;
        if (!codes && type != ScalarType::BFloat16)
            throw TypeErr(std::string("k_cache must be bfloat16, int8 or float8_e4m3fn, got ") + c10::toString(type));
        const at::Tensor &t = THPVariable_Unpack(k.p);
        const int64_t N = t.dim() ? t.size(0) : 0, H = g.num_kv_heads, P = g.page_size;
        k_cache = c.ptr(k.p, "k_cache", type, {N, H, P, g.head_dim_qk});
        v_cache = c.ptr(v.p, "v_cache", type, {N, H, P, g.head_dim_v});
        centroids = c.ptr(e.p, "centroids", ScalarType::BFloat16, {N, H, g.head_dim_qk});
        k_scale = c.ptr<float>(ks.p, "k_scale", ScalarType::Float, {N, H});
        v_scale = c.ptr<float>(vs.p, "v_scale", ScalarType::Float, {N, H});
        elem_bytes = codes ? 1 : 2;
        num_pages = N;
    }
};

uint64_t as_seed(PyObject *o) {
    const unsigned long long v = PyLong_AsUnsignedLongLongMask(o);
    if (v == ~0ull && PyErr_Occurred()) throw PyErr();
    return v;
}

// geo, table, cache, centroids, k_new, v_new, first_pos, err, stream
PyObject *quant_update(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Table t(c, a[1], g.batch);
    const Cache q(c, a[2], g);
    const int64_t n = a[6] == Py_None ? g.batch : ANY, H = g.num_kv_heads, D = g.head_dim_qk;
    void *cen = c.ptr(a[3], "centroids", ScalarType::BFloat16, {g.num_pool_pages, H, D});
    const void *k = c.ptr(a[4], "k_new", ScalarType::BFloat16, {n, H, D});
    const void *v = c.ptr(a[5], "v_new", ScalarType::BFloat16, {n, H, D});
    const int64_t rows = a[4] != Py_None ? THPVariable_Unpack(a[4]).size(0) : 0;
    if (a[5] != Py_None && THPVariable_Unpack(a[5]).size(0) != rows)
        throw ValueErr("k_new and v_new must have the same number of rows");
    const int32_t *first = c.ptr<int32_t>(a[6], "first_pos", ScalarType::Int, {g.batch});
    int32_t *err = c.err(a[7]);
    return c.run(a[8], [&](void *s) { return fn.quant_update(&g, &t, &q, cen, k, v, rows, first, err, s); });
}

// geo, table, q, cache, sel, k, out, ws, lse, sm_scale, num_splits, err, stream
PyObject *sparse_decode_quant(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Table t(c, a[1], g.batch);
    const void *q = c.ptr(a[2], "q", ScalarType::BFloat16, {g.batch, g.num_q_heads, g.head_dim_qk});
    const Cache qc(c, a[3], g);
    const int32_t k = as_i32(a[5], "k");
    const int32_t *sel = c.ptr<int32_t>(a[4], "sel", ScalarType::Int, {g.batch, g.num_kv_heads, k});
    void *out = c.ptr(a[6], "out", ScalarType::BFloat16, {g.batch, g.num_q_heads, g.head_dim_v});
    size_t n;
    void *ws = c.workspace(a[7], &n);
    float *lse = c.ptr<float>(a[8], "lse", ScalarType::Float, {g.batch, g.num_q_heads});
    const float scale = as_float(a[9]);
    const int32_t splits = as_i32(a[10], "num_splits");
    int32_t *err = c.err(a[11]);
    return c.run(a[12], [&](void *s) { return fn.sparse_decode_quant(&g, &t, q, &qc, sel, k, scale, splits, out, lse, ws, n, err, s); });
}

// geo, table, q, cache, centroids, k_new, v_new, k, out, ws, lse, mode, seed, sm_scale, score_dims, num_splits,
// scores_out, sel_out, err, stream; k_new and v_new None: no append
template <bool APPEND>
PyObject *block_topk_decode_quant(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Table t(c, a[1], g.batch);
    const void *q = c.ptr(a[2], "q", ScalarType::BFloat16, {g.batch, g.num_q_heads, g.head_dim_qk});
    const Cache qc(c, a[3], g);
    const int64_t H = g.num_kv_heads, D = g.head_dim_qk;
    void *cen = c.ptr(a[4], "centroids", ScalarType::BFloat16, {g.num_pool_pages, H, D});
    const void *kn = c.ptr(a[5], "k_new", ScalarType::BFloat16, {g.batch, H, D});
    const void *vn = c.ptr(a[6], "v_new", ScalarType::BFloat16, {g.batch, H, D});
    const int32_t k = as_i32(a[7], "k");
    void *out = c.ptr(a[8], "out", ScalarType::BFloat16, {g.batch, g.num_q_heads, g.head_dim_v});
    size_t n;
    void *ws = c.workspace(a[9], &n);
    float *lse = c.ptr<float>(a[10], "lse", ScalarType::Float, {g.batch, g.num_q_heads});
    const int32_t mode = as_i32(a[11], "mode");
    const uint64_t seed = as_seed(a[12]);
    const float scale = as_float(a[13]);
    const int32_t dims = as_i32(a[14], "score_dims"), splits = as_i32(a[15], "num_splits");
    float *sc = c.ptr<float>(a[16], "scores_out", ScalarType::Float, {g.batch, H, t.max_pages});
    int32_t *sel = c.ptr<int32_t>(a[17], "sel_out", ScalarType::Int, {g.batch, H, k});
    int32_t *err = c.err(a[18]);
    return c.run(a[19], [&](void *s) {
        if constexpr (APPEND)
            return fn.block_topk_decode_append_quant(&g, &t, q, &qc, cen, kn, vn, k, mode, seed, scale, dims, splits, out,
                                                     lse, sc, sel, ws, n, err, s);
        else
            return fn.block_topk_decode_quant(&g, &t, q, &qc, cen, k, mode, seed, scale, dims, splits, out, lse, sc, sel,
                                              ws, n, err, s);
    });
}

// geo, src, dst, src_pages, dst_pages, ws, err, stream
PyObject *copy_pages(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Pool src(c, a[1], g), dst(c, a[2], g);
    if (src.type != dst.type) throw TypeErr("the pools must hold the same type");
    const int32_t *s = c.ptr<int32_t>(a[3], "src_pages", ScalarType::Int, {ANY});
    const int64_t count = s || a[3] != Py_None ? THPVariable_Unpack(a[3]).numel() : 0;
    const int32_t *d = c.ptr<int32_t>(a[4], "dst_pages", ScalarType::Int, {count});
    if (count > INT32_MAX) throw ValueErr("src_pages has too many entries");
    size_t n;
    void *ws = c.workspace(a[5], &n);
    int32_t *err = c.err(a[6]);
    return c.run(a[7], [&](void *st) { return fn.copy_pages(&g, &src, &dst, s, d, (int32_t)count, ws, n, err, st); });
}

// geo, pool, table, ref, parent, grow, new_table, new_ref, ws, err, stream
PyObject *update_table(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Pool pool(c, a[1], g);
    const Table t(c, a[2], g.batch);
    const int32_t *ref = c.ptr<int32_t>(a[3], "ref", ScalarType::Int, {g.num_pool_pages});
    const int32_t *parent = c.ptr<int32_t>(a[4], "parent", ScalarType::Int, {ANY});
    const int64_t rows = a[4] != Py_None ? THPVariable_Unpack(a[4]).numel() : 0;
    if (rows > INT32_MAX) throw ValueErr("parent has too many entries");
    const int32_t *grow = c.ptr<int32_t>(a[5], "grow", ScalarType::Int, {rows});
    const Table to(c, a[6], rows);
    int32_t *new_ref = c.ptr<int32_t>(a[7], "new_ref", ScalarType::Int, {g.num_pool_pages});
    size_t n;
    void *ws = c.workspace(a[8], &n);
    int32_t *err = c.err(a[9]);
    if (overlap(to.page_indices, to.entries, t.page_indices, t.entries) ||
        overlap(to.page_indices, to.entries, t.seq_lens, g.batch) || overlap(to.page_indices, to.entries, t.page_ptr, g.batch))
        throw ValueErr("the new table's page_indices must not lie in the old table's memory");
    if (overlap(to.seq_lens, rows, t.page_indices, t.entries) || overlap(to.seq_lens, rows, t.seq_lens, g.batch) ||
        overlap(to.seq_lens, rows, t.page_ptr, g.batch))
        throw ValueErr("the new table's seq_lens must not lie in the old table's memory");
    return c.run(a[10], [&](void *s) {
        return fn.update_table(&g, &pool, &t, ref, parent, grow, (int32_t)rows, to.page_ptr,
                               const_cast<int32_t *>(to.page_indices), to.entries, const_cast<int32_t *>(to.seq_lens),
                               to.max_pages, new_ref, ws, n, err, s);
    });
}

// geo, pool, table, ref, new_indices, new_ref, remap, num_live, ws, err, stream
PyObject *compact_pages(PyObject *const *a) {
    Call c;
    const Geo g(a[0]);
    const Pool pool(c, a[1], g);
    const Table t(c, a[2], g.batch);
    const int64_t N = g.num_pool_pages;
    const int32_t *ref = c.ptr<int32_t>(a[3], "ref", ScalarType::Int, {N});
    int32_t *idx = c.flat<int32_t>(a[4], "new_indices", ScalarType::Int);
    if (idx && THPVariable_Unpack(a[4]).numel() != t.entries)
        throw ValueErr("new_indices must have as many entries as the table's page_indices");
    if (idx && idx != t.page_indices && overlap(idx, t.entries, t.page_indices, t.entries))
        throw ValueErr("new_indices must be the table's page_indices or apart from them");
    int32_t *new_ref = c.ptr<int32_t>(a[5], "new_ref", ScalarType::Int, {N});
    int32_t *remap = c.ptr<int32_t>(a[6], "remap", ScalarType::Int, {N});
    int32_t *live = c.ptr<int32_t>(a[7], "num_live", ScalarType::Int, {1});
    size_t n;
    void *ws = c.workspace(a[8], &n);
    int32_t *err = c.err(a[9]);
    return c.run(a[10], [&](void *s) { return fn.compact_pages(&g, &pool, &t, ref, idx, new_ref, remap, live, ws, n, err, s); });
}

// No C++ exception leaves the module: each becomes a Python one.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *guarded(PyObject *, PyObject *const *args, Py_ssize_t n) {
    try {
        if (n != N) throw TypeErr("wrong number of arguments");
        return F(args);
    } catch (const PyErr &) {
    } catch (const TypeErr &e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const ValueErr &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// addresses of the entry points, in the order of `fn`
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    void **to = reinterpret_cast<void **>(&fn);
    if (n != (Py_ssize_t)(sizeof(fn) / sizeof(void *))) {
        PyErr_SetString(PyExc_TypeError, "wrong number of entry points");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        void *p = PyLong_AsVoidPtr(args[i]);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "NULL entry point");
            return nullptr;
        }
        to[i] = p;
    }
    Py_RETURN_NONE;
}

#define METHOD(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&guarded<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(&bind)), METH_FASTCALL, nullptr},
    METHOD("quant_update", quant_update, 9),
    METHOD("sparse_decode_quant", sparse_decode_quant, 13),
    METHOD("block_topk_decode_quant", block_topk_decode_quant<false>, 20),
    METHOD("block_topk_decode_append_quant", block_topk_decode_quant<true>, 20),
    METHOD("copy_pages", copy_pages, 8),
    METHOD("update_table", update_table, 11),
    METHOD("compact_pages", compact_pages, 11),
    {nullptr, nullptr, 0, nullptr}};
// the docstring says what the module was built for (see build.py)
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vx_marshal", VX_MARSHAL_MARK, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vx_marshal(void) { return PyModule_Create(&module); }
