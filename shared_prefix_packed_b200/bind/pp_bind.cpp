// pp_bind.cpp - the checks of tensor arguments before the calls of q/k norm and of the paged cache, and the calls.
//
// These run once a layer on a few microseconds of GPU work. In Python the checks of a call's 7 to 12 tensors took 6 to
// 12 us, as long as the kernels; here they take about 1. Measured in a row of calls, outputs allocated: 128 tokens through
// pp_qk_norm_rope 11.5 -> 6.2 us, its fp32 gradients 24.9 -> 14.0, pp_pages_resize of a step 22.9 -> 12.2,
// pp_paged_decode of one response 24.0 -> 19.7 (the GPU bounds it then). A function takes its arguments by position, raises
// TypeError or ValueError where they do not fit, and else returns the call's pp_status. The library's functions are
// given by address (init), so that there is one libpp.so, the one that _lib.py has loaded.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/pp.h"

namespace {

using at::ScalarType;
using at::Tensor;

decltype(&pp_qk_norm_rope) g_norm;
decltype(&pp_qk_norm_rope_bwd) g_norm_bwd;
decltype(&pp_pages_resize) g_resize;
decltype(&pp_cache_store) g_store;
decltype(&pp_paged_decode) g_decode;

struct Raised {};                                          // a Python error is set
[[noreturn]] void raise(PyObject *type, const std::string &text) {
    PyErr_SetString(type, text.c_str());
    throw Raised{};
}
[[noreturn]] void type_error(const std::string &text) { raise(PyExc_TypeError, text); }
[[noreturn]] void value_error(const std::string &text) { raise(PyExc_ValueError, text); }

std::string dtype_name(ScalarType t) {
    switch (t) {
        case ScalarType::BFloat16: return "torch.bfloat16";
        case ScalarType::Float: return "torch.float32";
        case ScalarType::Double: return "torch.float64";
        case ScalarType::Half: return "torch.float16";
        case ScalarType::Char: return "torch.int8";
        case ScalarType::Int: return "torch.int32";
        case ScalarType::Long: return "torch.int64";
        case ScalarType::Byte: return "torch.uint8";
        case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
        default: return std::string("torch.") + c10::toString(t);
    }
}
constexpr int64_t ANY = -1;
template <typename L> std::string shape_name(const L &shape) {
    std::string s = "[";
    for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + (n == ANY ? std::string("None") : std::to_string(n));
    return s + "]";
}

// The tensors of a call: looked through in order, and at the end found to lie on one GPU.
struct Call {
    static constexpr int MAX = 16;
    const Tensor *t[MAX];
    const char *name[MAX];
    int n = 0;

    // An argument, nullptr for None where it may be that.
    const Tensor *arg(PyObject *o, const char *what, bool optional = false) {
        if (optional && o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) type_error(std::string(what) + " must be a tensor (got " + Py_TYPE(o)->tp_name + ")");
        name[n] = what;
        return t[n++] = &THPVariable_Unpack(o);
    }
    void of_type(const Tensor &x, const char *what, ScalarType dt) {
        if (x.scalar_type() != dt) type_error(std::string(what) + " must be " + dtype_name(dt) + " (got " + dtype_name(x.scalar_type()) + ")");
    }
    [[noreturn]] void bad_shape(const Tensor &x, const char *what, std::initializer_list<int64_t> shape) {
        value_error(std::string(what) + " must have shape " + shape_name(shape) + " (got " + shape_name(x.sizes()) + ")");
    }
    // x is dense, of the type and of the shape (ANY: any size there).
    void need(const Tensor &x, const char *what, ScalarType dt, std::initializer_list<int64_t> shape) {
        of_type(x, what, dt);
        bool same = x.dim() == int64_t(shape.size());
        int i = 0;
        for (int64_t w : shape) same = same && (w == ANY || x.size(i) == w), ++i;
        if (!same) bad_shape(x, what, shape);
        if (!x.is_contiguous()) value_error(std::string(what) + " must be contiguous");
    }
    const Tensor &need(PyObject *o, const char *what, ScalarType dt, std::initializer_list<int64_t> shape) {
        const Tensor &x = *arg(o, what);
        need(x, what, dt, shape);
        return x;
    }
    const Tensor &scratch(PyObject *o) {
        const Tensor &x = *arg(o, "workspace");
        if (!x.is_contiguous()) value_error("workspace must be contiguous");      // its bytes are those of its elements
        return x;
    }
    // The token stride of x [T, heads, d], whose heads and elements are dense.
    int64_t rows(const Tensor &x, const char *what, int64_t T, int64_t heads, int64_t d, ScalarType dt) {
        of_type(x, what, dt);
        if (x.dim() != 3 || x.size(0) != T || x.size(1) != heads || x.size(2) != d) bad_shape(x, what, {T, heads, d});
        if ((d > 1 && x.stride(2) != 1) || (heads > 1 && x.stride(1) != d))
            value_error(std::string(what) + ": the heads of a token must be dense");
        return T > 1 ? x.stride(0) : heads * d;
    }

    // fn(stream) on the tensors' device, on the stream given or that device's current one.
    template <typename F> PyObject *run(PyObject *stream, F fn) {
        int dev = -1;
        for (int i = 0; i < n; ++i) {
            if (!t[i]->is_cuda()) value_error(std::string(name[i]) + " must be a CUDA tensor (got " + t[i]->device().str() + ")");
            const int d = t[i]->get_device();
            if (dev >= 0 && d != dev)
                value_error(std::string("the tensors must lie on one device: ") + name[i] + " is on " + t[i]->device().str() +
                            ", others on cuda:" + std::to_string(dev));
            dev = d;
        }
        void *raw;
        if (stream == Py_None) {
            raw = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
        } else if (PyLong_Check(stream)) {
            raw = PyLong_AsVoidPtr(stream);
        } else {
            auto field = [](PyObject *o, const char *what) {
                PyObject *x = PyObject_GetAttrString(o, what);
                if (!x) throw Raised{};
                return x;
            };
            PyObject *device = field(stream, "device"), *index = nullptr, *handle = nullptr;
            index = PyObject_GetAttrString(device, "index");
            Py_DECREF(device);
            if (!index) throw Raised{};
            const long at = PyLong_AsLong(index);
            Py_DECREF(index);
            if (PyErr_Occurred()) throw Raised{};
            if (at != dev)
                value_error("the stream is of cuda:" + std::to_string(at) + ", the tensors of cuda:" + std::to_string(dev));
            handle = field(stream, "cuda_stream");
            raw = PyLong_AsVoidPtr(handle);
            Py_DECREF(handle);
        }
        if (PyErr_Occurred()) throw Raised{};
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev) guard.set_index(c10::DeviceIndex(dev));
        pp_status st;
        Py_BEGIN_ALLOW_THREADS
        st = fn(raw);
        Py_END_ALLOW_THREADS
        return PyLong_FromLong(st);
    }
};

template <typename T = void> T *at_of(const Tensor *t) { return t ? static_cast<T *>(t->data_ptr()) : nullptr; }
template <typename T = void> T *at_of(const Tensor &t) { return static_cast<T *>(t.data_ptr()); }
float number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return float(x);
}
int32_t integer(PyObject *o) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Raised{};
    if (x != int32_t(x)) value_error("an integer beyond 32 bits");
    return int32_t(x);
}
int32_t size32(int64_t n, const char *what) {
    if (n != int32_t(n)) value_error(std::string(what) + ": a size beyond 32 bits");
    return int32_t(n);
}
pp_dtype real_code(const Tensor &x) {
    if (x.scalar_type() == ScalarType::BFloat16) return PP_BF16;
    if (x.scalar_type() == ScalarType::Float) return PP_FP32;
    type_error("unsupported dtype " + dtype_name(x.scalar_type()));
}

// A function of n arguments, by position; what it throws becomes a Python error.
template <int N, PyObject *(*F)(PyObject *const *)> PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// q, k, wq, wk, pos_ids: what both directions of the norm share.
struct Norm {
    const Tensor *q, *k, *wq, *wk, *pos;
    int64_t T, qs = 0, ks = 0;
    int32_t hq, hkv, d;
    ScalarType dt;
    pp_dtype code;
    Norm(Call &c, PyObject *const *a) {
        q = c.arg(a[0], "q", true);
        k = c.arg(a[1], "k", true);
        const Tensor *ref = q ? q : k;
        if (!ref) value_error("q and k are both None");
        if (ref->dim() != 3 || (k && k->dim() != 3)) value_error("q and k must have shape [T, heads, d]");
        T = ref->size(0);
        hq = size32(ref->size(1), "heads");
        hkv = size32((k ? k : q)->size(1), "heads");
        d = size32(ref->size(2), "d");
        code = real_code(*ref);
        dt = ref->scalar_type();
        if (q) qs = c.rows(*q, "q", T, hq, d, dt);
        if (k) ks = c.rows(*k, "k", T, hkv, d, dt);
        wq = c.arg(a[2], "wq", true);
        wk = c.arg(a[3], "wk", true);
        if (q && wq) c.need(*wq, "wq", dt, {d});
        if (k && wk) c.need(*wk, "wk", dt, {d});
    }
    void positions(Call &c, PyObject *o) {
        pos = &c.need(o, "pos_ids_d", ScalarType::Int, {ANY});
        if (pos->size(0) < T)
            value_error("pos_ids_d holds " + std::to_string(pos->size(0)) + " positions for " + std::to_string(T) + " tokens");
    }
};

// q, k, wq, wk, pos_ids, q_out, k_out, eps, theta, stream
PyObject *norm(PyObject *const *a) {
    Call c;
    Norm s(c, a);
    const Tensor *qo = c.arg(a[5], "q_out", !s.q), *ko = c.arg(a[6], "k_out", !s.k);
    const int64_t qos = s.q ? c.rows(*qo, "q_out", s.T, s.hq, s.d, s.dt) : 0, kos = s.k ? c.rows(*ko, "k_out", s.T, s.hkv, s.d, s.dt) : 0;
    s.positions(c, a[4]);
    const float eps = number(a[7]), theta = number(a[8]);
    return c.run(a[9], [&](void *stream) {
        return g_norm(at_of(s.q), at_of(s.k), s.qs, s.ks, at_of(s.wq), at_of(s.wk), at_of<int32_t>(s.pos), s.T, s.hq, s.hkv, s.d, eps,
                      theta, s.code, at_of(qo), at_of(ko), qos, kos, stream);
    });
}

// q, k, wq, wk, pos_ids, gq, gk, dq, dk, dwq, dwk, workspace, eps, theta, stream
PyObject *norm_bwd(PyObject *const *a) {
    Call c;
    Norm s(c, a);
    const Tensor *gq = c.arg(a[5], "gq", !s.q), *gk = c.arg(a[6], "gk", !s.k), *dq = c.arg(a[7], "dq", !s.q), *dk = c.arg(a[8], "dk", !s.k);
    int64_t gqs = 0, gks = 0, dqs = 0, dks = 0;
    if (s.q) {
        gqs = c.rows(*gq, "gq", s.T, s.hq, s.d, s.dt);
        dqs = c.rows(*dq, "dq", s.T, s.hq, s.d, s.dt);
    }
    if (s.k) {
        gks = c.rows(*gk, "gk", s.T, s.hkv, s.d, s.dt);
        dks = c.rows(*dk, "dk", s.T, s.hkv, s.d, s.dt);
    }
    const Tensor *dwq = c.arg(a[9], "dwq", true), *dwk = c.arg(a[10], "dwk", true);
    if (dwq) c.need(*dwq, "dwq", ScalarType::Float, {s.d});
    if (dwk) c.need(*dwk, "dwk", ScalarType::Float, {s.d});
    s.positions(c, a[4]);
    const Tensor &ws = c.scratch(a[11]);
    const float eps = number(a[12]), theta = number(a[13]);
    return c.run(a[14], [&](void *stream) {
        return g_norm_bwd(at_of(s.q), at_of(s.k), s.qs, s.ks, at_of(s.wq), at_of(s.wk), at_of<int32_t>(s.pos), s.T, s.hq, s.hkv, s.d,
                          eps, theta, s.code, at_of(gq), at_of(gk), gqs, gks, at_of(dq), at_of(dk), dqs, dks, at_of<float>(dwq),
                          at_of<float>(dwk), at_of(ws), int64_t(ws.nbytes()), stream);
    });
}

struct Groups {
    const Tensor &start, &seg;
    int32_t G, nseg;
    Groups(Call &c, PyObject *s, PyObject *g)
        : start(c.need(s, "group_start_d", ScalarType::Int, {ANY})), seg(c.need(g, "seg_group_d", ScalarType::Int, {ANY})) {
        G = size32(start.size(0) - 1, "group_start_d");
        if (G < 1) value_error("group_start_d must hold num_groups + 1 >= 2 entries");
        nseg = size32(seg.size(0), "seg_group_d");
    }
};

// group_start, seg_group, old_lens, new_lens, page_size, page_table, free_pages, n_free_in, n_free_out, slots, pos_ids,
// counts, stream
PyObject *resize(PyObject *const *a) {
    Call c;
    const auto I = ScalarType::Int;
    Groups g(c, a[0], a[1]);
    const Tensor &old_lens = c.need(a[2], "old_lens_d", I, {g.nseg}), &new_lens = c.need(a[3], "new_lens_d", I, {g.nseg});
    const int32_t page = integer(a[4]);
    const Tensor &table = c.need(a[5], "page_table_d", I, {g.nseg, ANY}), &free_pages = c.need(a[6], "free_pages_d", I, {ANY});
    const Tensor &n_in = c.need(a[7], "n_free_in", I, {1}), &n_out = c.need(a[8], "n_free_out", I, {1});
    const Tensor &slots = c.need(a[9], "slots_d", I, {ANY});
    const int64_t capacity = slots.size(0);
    const Tensor &pos = c.need(a[10], "pos_ids_d", I, {capacity}), &counts = c.need(a[11], "counts_d", I, {4});
    const int32_t pool = size32(free_pages.size(0), "free_pages_d");
    return c.run(a[12], [&](void *stream) {
        return g_resize(at_of<int32_t>(g.start), g.G, at_of<int32_t>(g.seg), g.nseg, at_of<int32_t>(old_lens), at_of<int32_t>(new_lens),
                        page, at_of<int32_t>(table), table.size(1), at_of<int32_t>(free_pages), pool, at_of<int32_t>(n_in),
                        at_of<int32_t>(n_out), at_of<int32_t>(slots), at_of<int32_t>(pos), capacity, at_of<int32_t>(counts), stream);
    });
}

struct Pool {
    const Tensor &k, &v, &ks, &vs;
    pp_dtype codes;
    int32_t num_pages, hkv, page, d;
    Pool(Call &c, PyObject *const *a) : k(*c.arg(a[0], "k_pages")), v(*c.arg(a[1], "v_pages")), ks(*c.arg(a[2], "k_scale")), vs(*c.arg(a[3], "v_scale")) {
        const ScalarType dt = k.scalar_type();
        if (dt == ScalarType::Float8_e4m3fn) codes = PP_E4M3;
        else if (dt == ScalarType::Char) codes = PP_INT8;
        else type_error("k_pages must be float8_e4m3fn or int8 (got " + dtype_name(dt) + ")");
        if (k.dim() != 4) value_error("k_pages must have shape [num_pages, hkv, page_size, d]");
        if (!k.is_contiguous()) value_error("k_pages must be contiguous");
        num_pages = size32(k.size(0), "k_pages");
        hkv = size32(k.size(1), "k_pages");
        page = size32(k.size(2), "k_pages");
        d = size32(k.size(3), "k_pages");
        c.need(v, "v_pages", dt, {num_pages, hkv, d, page});
        c.need(ks, "k_scale", ScalarType::Float, {num_pages, hkv});
        c.need(vs, "v_scale", ScalarType::Float, {num_pages, hkv});
    }
};

// k, v, slots, k_pages, v_pages, k_scale, v_scale, stream
PyObject *store(PyObject *const *a) {
    Call c;
    Pool p(c, a + 3);
    const Tensor &k = *c.arg(a[0], "k"), &v = *c.arg(a[1], "v");
    if (k.dim() != 3) value_error("k and v must have shape [n, hkv, d]");
    const int64_t n = k.size(0);
    const pp_dtype code = real_code(k);
    const int64_t ks = c.rows(k, "k", n, p.hkv, p.d, k.scalar_type()), vs = c.rows(v, "v", n, p.hkv, p.d, k.scalar_type());
    const Tensor &slots = c.need(a[2], "slots_d", ScalarType::Int, {n});
    return c.run(a[7], [&](void *stream) {
        return g_store(at_of(k), at_of(v), ks, vs, code, at_of<int32_t>(slots), n, p.hkv, p.d, at_of(p.k), at_of(p.v),
                       at_of<float>(p.ks), at_of<float>(p.vs), p.codes, p.num_pages, p.page, stream);
    });
}

// q, k_pages, v_pages, k_scale, v_scale, group_start, seg_group, lens, page_table, o, lse, workspace, softmax_scale, stream
PyObject *decode(PyObject *const *a) {
    Call c;
    Pool p(c, a + 1);
    Groups g(c, a[5], a[6]);
    const Tensor &q = *c.arg(a[0], "q");
    if (q.dim() != 3) value_error("q must have shape [n_resp, hq, d]");
    const int32_t hq = size32(q.size(1), "q"), n_resp = g.nseg - g.G;
    c.need(q, "q", ScalarType::BFloat16, {n_resp, hq, p.d});
    const Tensor &o = c.need(a[9], "o", ScalarType::BFloat16, {n_resp, hq, p.d}), &lse = c.need(a[10], "lse", ScalarType::Float, {hq, n_resp});
    const Tensor &lens = c.need(a[7], "lens_d", ScalarType::Int, {g.nseg}), &table = c.need(a[8], "page_table_d", ScalarType::Int, {g.nseg, ANY});
    const Tensor &ws = c.scratch(a[11]);
    const float scale = number(a[12]);
    return c.run(a[13], [&](void *stream) {
        return g_decode(at_of(q), at_of(p.k), at_of(p.v), at_of<float>(p.ks), at_of<float>(p.vs), p.codes, p.num_pages, p.page,
                        at_of<int32_t>(g.start), g.G, at_of<int32_t>(g.seg), g.nseg, at_of<int32_t>(lens), at_of<int32_t>(table),
                        table.size(1), hq, p.hkv, p.d, scale, at_of(o), at_of<float>(lse), at_of(ws), int64_t(ws.nbytes()), stream);
    });
}

// The addresses of the five calls in the order above.
PyObject *init(PyObject *const *a) {
    void *at[5];
    for (int i = 0; i < 5; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) throw Raised{};
    }
    g_norm = reinterpret_cast<decltype(g_norm)>(at[0]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(at[1]);
    g_resize = reinterpret_cast<decltype(g_resize)>(at[2]);
    g_store = reinterpret_cast<decltype(g_store)>(at[3]);
    g_decode = reinterpret_cast<decltype(g_decode)>(at[4]);
    Py_RETURN_NONE;
}

template <int N, PyObject *(*F)(PyObject *const *)> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<N, F>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<5, init>("init"),
                         method<10, norm>("qk_norm_rope"),
                         method<15, norm_bwd>("qk_norm_rope_bwd"),
                         method<13, resize>("pages_resize"),
                         method<8, store>("cache_store"),
                         method<14, decode>("paged_decode"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() { return PyModule_Create(&module); }
