// Python entry points of the softmax-attention layer's calls: tensors in, the C
// ABI of include/gdn.h called on their current stream, tensors out. The calls
// of a decode step take a few microseconds on the GPU; marshalled in Python
// their arguments cost several times that on the host (17 us of 20 for a
// one-token cache write), so the checks and allocations stand here.
//
// The module links nothing of the library: gated_deltanet_linear_silu_b200
// hands it the addresses of the entry points (bind) after checking the ABI
// version, and the exception class for their status codes.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/gdn.h"

// What this was compiled against (build.py looks for it in the file).
extern "C" __attribute__((used, visibility("default"))) const char gdn_binding_tag[] = GDN_BINDING_TAG;

namespace {

struct Entry {
    decltype(&gdn_qk_norm_rope) qk_norm_rope;
    decltype(&gdn_qk_norm_rope_cache) qk_norm_rope_cache;
    decltype(&gdn_kv_write) kv_write;
    decltype(&gdn_kv_read) kv_read;
    decltype(&gdn_kv_accept) kv_accept;
    decltype(&gdn_tree_attention_workspace_size) tree_size;
    decltype(&gdn_tree_attention) tree;
} g;
PyObject* g_error = nullptr;  // GDNError(status, what)

// A refused argument: ValueError, or TypeError for a type.
struct Refused {
    PyObject* kind;
    std::string what;
};
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
int64_t integer(PyObject* o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return x;
}
int int32(PyObject* o, const char* name) {
    const int64_t x = integer(o);
    if (x < INT32_MIN || x > INT32_MAX) value_error(std::string(name) + " does not fit 32 bits");
    return (int)x;
}
bool truth(PyObject* o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Refused{nullptr, ""};
    return x != 0;
}
double real(PyObject* o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return x;
}

void dense(const at::Tensor& t, at::Device dev, const char* name) {
    if (t.device() != dev) value_error(std::string(name) + ": tensors must be on one CUDA device");
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
at::Device cuda_device(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return t.device();
}
gdn_dtype_t act_type(at::ScalarType t) {
    if (t == at::kBFloat16) return GDN_BF16;
    if (t == at::kFloat) return GDN_F32;
    type_error("unsupported dtype (bfloat16 or float32)");
}

// [T, heads, D] whose rows [heads, D] are dense; its token stride.
int64_t token_stride(const at::Tensor& t, at::Device dev, const char* name) {
    if (t.device() != dev) value_error(std::string(name) + ": tensors must be on one CUDA device");
    if (t.dim() != 3) value_error(std::string(name) + " must be [T, heads, D]");
    const int64_t h = t.size(1), d = t.size(2);
    if (t.size(0) == 0) return 0;
    if (t.size(0) == 1 && t.is_contiguous()) return h * d;
    if (t.stride(2) != 1 || (h > 1 && t.stride(1) != d) || t.stride(0) < h * d)
        value_error(std::string(name) + " must have dense [heads, D] rows (the token stride may be larger)");
    return t.stride(0);
}

struct Cache {
    gdn_kv_cache_t c;
    Cache(PyObject* const* a, at::Device dev) {
        const at::Tensor &k = tensor(a[0], "cache.k"), &v = tensor(a[1], "cache.v");
        if (k.dim() != 4 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
            value_error("the cache's k and v must be [n_pages, Hk, page, D] alike");
        dense(k, dev, "cache.k");
        dense(v, dev, "cache.v");
        c.k = k.data_ptr();
        c.v = v.data_ptr();
        c.k_scale = c.v_scale = nullptr;
        if (k.scalar_type() == at::kFloat8_e4m3fn) {
            const at::Tensor *ks = maybe(a[2], "cache.k_scale"), *vs = maybe(a[3], "cache.v_scale");
            if (!ks || !vs || ks->sizes() != k.sizes().slice(0, 3) || vs->sizes() != k.sizes().slice(0, 3))
                value_error("an e4m3 cache needs k_scale and v_scale [n_pages, Hk, page]");
            if (ks->scalar_type() != at::kFloat || vs->scalar_type() != at::kFloat)
                type_error("the cache's scales must be float32");
            dense(*ks, dev, "cache.k_scale");
            dense(*vs, dev, "cache.v_scale");
            c.k_scale = static_cast<float*>(ks->data_ptr());
            c.v_scale = static_cast<float*>(vs->data_ptr());
            c.dtype = GDN_E4M3;
        } else if (k.scalar_type() == at::kBFloat16) {
            c.dtype = GDN_BF16;
        } else {
            type_error("unsupported cache dtype (float8_e4m3fn or bfloat16)");
        }
        if (k.size(1) > INT32_MAX || k.size(2) > INT32_MAX || k.size(3) > INT32_MAX) value_error("cache too large");
        c.n_pages = k.size(0);
        c.Hk = (int)k.size(1);
        c.page = (int)k.size(2);
        c.D = (int)k.size(3);
    }
};

struct Pages {
    const int32_t *table, *lens, *cu;
    int max_pages, N;
    const at::Tensor* lens_t;
    Pages(PyObject* const* a, at::Device dev) {
        const at::Tensor &t = tensor(a[0], "page_table"), &l = tensor(a[1], "seq_lens"), &c = tensor(a[2], "cu_seqlens");
        if (t.scalar_type() != at::kInt || l.scalar_type() != at::kInt || c.scalar_type() != at::kInt)
            type_error("page_table, seq_lens and cu_seqlens must be int32");
        if (c.dim() != 1 || c.size(0) < 1 || l.dim() != 1 || l.size(0) != c.size(0) - 1 || t.dim() != 2 ||
            t.size(0) != l.size(0) || l.size(0) > INT32_MAX || t.size(1) > INT32_MAX)
            value_error("page_table must be [N, max_pages], seq_lens [N] and cu_seqlens [N + 1]");
        dense(t, dev, "page_table");
        dense(l, dev, "seq_lens");
        dense(c, dev, "cu_seqlens");
        table = static_cast<const int32_t*>(t.data_ptr());
        lens = static_cast<const int32_t*>(l.data_ptr());
        cu = static_cast<const int32_t*>(c.data_ptr());
        max_pages = (int)t.size(1);
        N = (int)l.size(0);
        lens_t = &l;
    }
};

// q_w, k_w, positions, inv_freq
struct Norm {
    const float *q_w, *k_w;
    const int32_t* pos;
    const double* inv_freq;
    int rotary;
    Norm(const at::Tensor& q, const at::Tensor& k, PyObject* const* a, at::Device dev) {
        if (q.dim() != 3 || k.dim() != 3 || k.size(0) != q.size(0) || k.size(2) != q.size(2) ||
            k.scalar_type() != q.scalar_type())
            value_error("q must be [T, H, D] and k [T, Hk, D] of one dtype");
        if (q.size(1) > INT32_MAX || k.size(1) > INT32_MAX || q.size(2) > INT32_MAX)
            value_error("q, k: more heads or elements than 32 bits count");
        const at::Tensor &wq = tensor(a[0], "q_w"), &wk = tensor(a[1], "k_w"), &p = tensor(a[2], "positions"),
                         &f = tensor(a[3], "inv_freq");
        if (wq.dim() != 1 || wq.size(0) != q.size(2) || wk.dim() != 1 || wk.size(0) != q.size(2) ||
            wq.scalar_type() != at::kFloat || wk.scalar_type() != at::kFloat)
            value_error("q_w and k_w must be [D] float32");
        if (p.dim() != 1 || p.size(0) != q.size(0) || p.scalar_type() != at::kInt)
            value_error("positions must be [T] int32");
        if (f.dim() != 1 || f.scalar_type() != at::kDouble || 2 * f.size(0) > q.size(2))
            value_error("inv_freq must be [rotary / 2] float64, rotary at most D");
        dense(wq, dev, "q_w");
        dense(wk, dev, "k_w");
        dense(p, dev, "positions");
        dense(f, dev, "inv_freq");
        q_w = static_cast<const float*>(wq.data_ptr());
        k_w = static_cast<const float*>(wk.data_ptr());
        pos = static_cast<const int32_t*>(p.data_ptr());
        inv_freq = static_cast<const double*>(f.data_ptr());
        rotary = 2 * (int)f.size(0);
    }
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, at::Device dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}
at::Tensor output(PyObject* given, at::IntArrayRef shape, at::ScalarType type, at::Device dev, const char* name) {
    const at::Tensor* t = maybe(given, name);
    if (!t) return empty(shape, type, dev);
    if (t->sizes() != shape || t->scalar_type() != type) value_error(std::string(name) + " has another shape or dtype");
    dense(*t, dev, name);
    return *t;
}
void check(gdn_status_t st, const char* what) {
    if (st == GDN_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "is", (int)st, what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Refused{nullptr, ""};
}
// The C ABI works on the current device: make the tensors' device current.
struct On {
    c10::cuda::CUDAGuard guard;
    void* stream;
    explicit On(at::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};
PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
    PyObject* t = PyTuple_New(2);
    if (!t) throw Refused{nullptr, ""};
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    return t;
}

// Runs a call; what it throws becomes a Python exception.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
    if (got != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
        return nullptr;
    }
    try {
        return f();
    } catch (const Refused& r) {
        if (r.kind) PyErr_SetString(r.kind, r.what.c_str());
    } catch (const c10::OutOfMemoryError& e) {
        PyObject* torch = PyImport_ImportModule("torch");
        PyObject* kind = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (kind) PyErr_SetString(kind, e.what_without_backtrace());
        Py_XDECREF(kind);
        Py_XDECREF(torch);
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// q, k, q_w, k_w, positions, inv_freq, eps, interleaved, out_q, out_k -> (q, k)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&] {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
        const at::Device dev = cuda_device(q, "q");
        const Norm m(q, k, a + 2, dev);
        const gdn_dtype_t type = act_type(q.scalar_type());
        const int64_t ld_q = token_stride(q, dev, "q"), ld_k = token_stride(k, dev, "k");
        const at::Tensor oq = output(a[8], q.sizes(), q.scalar_type(), dev, "out_q");
        const at::Tensor ok = output(a[9], k.sizes(), k.scalar_type(), dev, "out_k");
        const On on(dev);
        check(g.qk_norm_rope(q.data_ptr(), k.data_ptr(), type, q.size(0), (int)q.size(1), (int)k.size(1),
                             (int)q.size(2), ld_q, ld_k, m.q_w, m.k_w, (float)real(a[6]), m.pos, m.inv_freq, m.rotary,
                             truth(a[7]), oq.data_ptr(), ok.data_ptr(), on.stream),
              "gdn_qk_norm_rope");
        return pair(oq, ok);
    });
}

// q, k, v, q_w, k_w, positions, inv_freq, cache (4), pages (3), eps, interleaved, out_q -> q
PyObject* qk_norm_rope_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 17, [&] {
        const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const at::Device dev = cuda_device(q, "q");
        const Norm m(q, k, a + 3, dev);
        const Cache c(a + 7, dev);
        const Pages p(a + 11, dev);
        const gdn_dtype_t type = act_type(q.scalar_type());
        if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || k.size(1) != c.c.Hk || k.size(2) != c.c.D)
            value_error("k and v must be [T, Hk, D] of one dtype, Hk and D the cache's");
        const int64_t ld_q = token_stride(q, dev, "q"), ld_k = token_stride(k, dev, "k"), ld_v = token_stride(v, dev, "v");
        const at::Tensor oq = output(a[16], q.sizes(), q.scalar_type(), dev, "out_q");
        const On on(dev);
        check(g.qk_norm_rope_cache(q.data_ptr(), k.data_ptr(), v.data_ptr(), type, q.size(0), (int)q.size(1), ld_q, ld_k,
                                   ld_v, m.q_w, m.k_w, (float)real(a[14]), m.pos, m.inv_freq, m.rotary,
                                   truth(a[15]), &c.c, p.table, p.max_pages, p.lens, p.cu, p.N, oq.data_ptr(),
                                   on.stream),
              "gdn_qk_norm_rope_cache");
        return THPVariable_Wrap(oq);
    });
}

// k, v, cache (4), pages (3) -> None
PyObject* kv_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
        const at::Device dev = cuda_device(k, "k");
        const Cache c(a + 2, dev);
        const Pages p(a + 6, dev);
        const gdn_dtype_t type = act_type(k.scalar_type());
        if (k.dim() != 3 || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || k.size(1) != c.c.Hk ||
            k.size(2) != c.c.D)
            value_error("k and v must be [T, Hk, D] of one dtype, Hk and D the cache's");
        const int64_t ld_k = token_stride(k, dev, "k"), ld_v = token_stride(v, dev, "v");
        const On on(dev);
        check(g.kv_write(k.data_ptr(), v.data_ptr(), type, k.size(0), ld_k, ld_v, &c.c, p.table, p.max_pages, p.lens,
                         p.cu, p.N, on.stream),
              "gdn_kv_write");
        Py_RETURN_NONE;
    });
}

// cache (4), pages (3), n_tokens, bf16, out_k, out_v -> (k, v)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&] {
        const at::Device dev = cuda_device(tensor(a[0], "cache.k"), "cache.k");
        const Cache c(a, dev);
        const Pages p(a + 4, dev);
        const int64_t T = integer(a[7]);
        if (T < 0) value_error("n_tokens must not be negative");
        const bool bf16 = truth(a[8]);
        const int64_t shape[3] = {T, c.c.Hk, c.c.D};
        const at::ScalarType type = bf16 ? at::kBFloat16 : at::kFloat;
        const at::Tensor k = output(a[9], shape, type, dev, "out_k"), v = output(a[10], shape, type, dev, "out_v");
        const On on(dev);
        check(g.kv_read(&c.c, p.table, p.max_pages, p.lens, p.cu, p.N, T, bf16 ? GDN_BF16 : GDN_F32, k.data_ptr(),
                        v.data_ptr(), on.stream),
              "gdn_kv_read");
        return pair(k, v);
    });
}

// cache (4), pages (3), accepted, out_seq_lens -> seq_lens
PyObject* kv_accept(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const at::Device dev = cuda_device(tensor(a[0], "cache.k"), "cache.k");
        const Cache c(a, dev);
        const Pages p(a + 4, dev);
        const at::Tensor& x = tensor(a[7], "accepted");
        if (x.dim() != 2 || x.size(0) != p.N || x.scalar_type() != at::kInt || x.size(1) > INT32_MAX)
            value_error("accepted must be [N, M] int32");
        dense(x, dev, "accepted");
        const at::Tensor out = output(a[8], p.lens_t->sizes(), at::kInt, dev, "out_seq_lens");
        const On on(dev);
        check(g.kv_accept(&c.c, p.table, p.max_pages, p.lens, p.cu, p.N, static_cast<const int32_t*>(x.data_ptr()),
                          (int)x.size(1), static_cast<int32_t*>(out.data_ptr()), on.stream),
              "gdn_kv_accept");
        return THPVariable_Wrap(out);
    });
}

// q, cache (4), pages (3), max_nodes, mask, scale (or None), gate, return_lse, out, workspace -> o or (o, lse)
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&] {
        const at::Tensor& q = tensor(a[0], "q");
        const at::Device dev = cuda_device(q, "q");
        const Cache c(a + 1, dev);
        const Pages p(a + 5, dev);
        const int max_nodes = int32(a[8], "max_nodes");
        const at::Tensor *mask = maybe(a[9], "mask"), *gate = maybe(a[11], "gate"), *given = maybe(a[14], "workspace");
        if (q.dim() != 3 || q.size(2) != c.c.D || q.size(1) > INT32_MAX) value_error("q must be [T, H, D], D the cache's");
        const gdn_dtype_t type = act_type(q.scalar_type());
        const int64_t T = q.size(0), ld = token_stride(q, dev, "q");
        const int H = (int)q.size(1);
        if (mask) {
            if (mask->dim() != 1 || mask->size(0) != T || mask->scalar_type() != at::kLong)
                value_error("mask must be [T] int64");
            dense(*mask, dev, "mask");
        }
        if (gate) {
            if (gate->sizes() != q.sizes() || gate->scalar_type() != q.scalar_type())
                value_error("gate must be [T, H, D] in the dtype of q");
            dense(*gate, dev, "gate");
        }
        const float scale = a[10] == Py_None ? 1.f / std::sqrt((float)c.c.D) : (float)real(a[10]);
        const at::Tensor o = output(a[13], q.sizes(), q.scalar_type(), dev, "out");
        const bool want_lse = truth(a[12]);
        at::Tensor lse;
        const int64_t lse_shape[2] = {T, H};
        if (want_lse) lse = empty(lse_shape, at::kFloat, dev);
        const On on(dev);
        at::Tensor ws;
        if (given) {
            dense(*given, dev, "workspace");
            ws = *given;
        } else {
            const int64_t bytes = (int64_t)g.tree_size(&c.c, p.N, H, max_nodes);
            ws = empty(bytes, at::kByte, dev);
        }
        check(g.tree(q.data_ptr(), type, T, ld, H, &c.c, p.table, p.max_pages, p.lens, p.cu, p.N,
                     mask ? static_cast<const int64_t*>(mask->data_ptr()) : nullptr, max_nodes, scale,
                     gate ? gate->data_ptr() : nullptr, o.data_ptr(),
                     want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws.data_ptr(), ws.nbytes(), on.stream),
              "gdn_tree_attention");
        return want_lse ? pair(o, lse) : THPVariable_Wrap(o);
    });
}

// (addresses of the entry points, exception class)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 8) {
        PyErr_SetString(PyExc_TypeError, "bind takes seven addresses and the exception class");
        return nullptr;
    }
    void* p[7];
    for (int i = 0; i < 7; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
            return nullptr;
        }
    }
    g.qk_norm_rope = reinterpret_cast<decltype(g.qk_norm_rope)>(p[0]);
    g.qk_norm_rope_cache = reinterpret_cast<decltype(g.qk_norm_rope_cache)>(p[1]);
    g.kv_write = reinterpret_cast<decltype(g.kv_write)>(p[2]);
    g.kv_read = reinterpret_cast<decltype(g.kv_read)>(p[3]);
    g.kv_accept = reinterpret_cast<decltype(g.kv_accept)>(p[4]);
    g.tree_size = reinterpret_cast<decltype(g.tree_size)>(p[5]);
    g.tree = reinterpret_cast<decltype(g.tree)>(p[6]);
    Py_INCREF(a[7]);
    g_error = a[7];
    Py_RETURN_NONE;
}

#define ENTRY(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind),      ENTRY(qk_norm_rope), ENTRY(qk_norm_rope_cache),
                         ENTRY(kv_write),  ENTRY(kv_read),      ENTRY(kv_accept),
                         ENTRY(tree_attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
