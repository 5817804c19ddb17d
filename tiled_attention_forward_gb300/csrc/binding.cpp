// binding.cpp -- argument marshalling of the serving calls for Python
// (fwd_packed, cache_append, cache_append_kv4, decode, decode_kv4): torch
// tensors in, the C ABI of include/fattn.h out, nothing else.
//
// A decode step's kernels take 3 to 9 us, and checking and converting a dozen
// tensors in Python took 8 to 14 us of every call; here it takes under 1 us.
// Each function returns the library's status; what it can see to be wrong with
// the tensors themselves (shape, type, device, layout) raises ValueError before
// the library is called.  Tensors that may be absent are None.
#include <Python.h>

#include <exception>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fattn.h"

namespace {

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};

std::string shape_text(std::initializer_list<int64_t> shape) {
    std::string s = "[";
    for (int64_t n : shape) s += (s.size() > 1 ? ", " : "") + std::to_string(n);
    return s + "]";
}

// The call's arguments, taken in order.
struct Args {
    PyObject* const* at;
    Py_ssize_t left;
    PyObject* next() {
        if (left-- <= 0) throw Refused("too few arguments");
        return *at++;
    }
    const at::Tensor* maybe(const char* name) {
        PyObject* o = next();
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) throw Refused(std::string(name) + " must be a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided) throw Refused(std::string(name) + " must be a strided tensor");
        return &t;
    }
    const at::Tensor& tensor(const char* name) {
        const at::Tensor* t = maybe(name);
        if (!t) throw Refused(std::string(name) + " must be a tensor");
        return *t;
    }
    int64_t integer() {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Refused("an argument must be an integer");
        return v;
    }
    double number() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Refused("scale must be a number");
        return v;
    }
    void done() const {
        if (left != 0) throw Refused("too many arguments");
    }
};

// What every tensor of a call shares.
struct Place {
    int device;
    at::ScalarType type;
    int dtype;  // fattn_dtype

    explicit Place(const at::Tensor& t, const char* name, int64_t dims) {
        if (!t.is_cuda() || t.dim() != dims)
            throw Refused(std::string(name) + " must be a CUDA tensor of " + std::to_string(dims) + " dimensions");
        device = t.get_device();
        type = t.scalar_type();
        if (type == at::kHalf)
            dtype = FATTN_F16;
        else if (type == at::kBFloat16)
            dtype = FATTN_BF16;
        else
            throw Refused(std::string(name) + " must be float16 or bfloat16");
    }

    void shaped(const char* name, const at::Tensor& t, at::ScalarType want, std::initializer_list<int64_t> shape) const {
        bool ok = t.is_cuda() && t.get_device() == device && t.scalar_type() == want &&
                  t.dim() == static_cast<int64_t>(shape.size());
        int64_t i = 0;
        for (int64_t n : shape) ok = ok && t.size(i++) == n;
        if (!ok)
            throw Refused(std::string(name) + " must be " + shape_text(shape) + " " + at::toString(want) + " on cuda:" +
                          std::to_string(device));
    }

    // Strides of 16-bit rows, contiguous along the last dimension; 0 stands for
    // that of a dimension of one element, which is never used.
    void rows(const char* name, const at::Tensor* t, std::initializer_list<int64_t> shape, int64_t* strides) const {
        const int64_t outer = static_cast<int64_t>(shape.size()) - 1;
        if (!t) {
            for (int64_t i = 0; i < outer; ++i) strides[i] = 0;
            return;
        }
        shaped(name, *t, type, shape);
        if (t->stride(outer) != 1) throw Refused(std::string(name) + " must be contiguous along its last dimension");
        for (int64_t i = 0; i < outer; ++i) strides[i] = t->size(i) == 1 ? 0 : t->stride(i);
    }

    void* dense(const char* name, const at::Tensor& t, at::ScalarType want, std::initializer_list<int64_t> shape) const {
        shaped(name, t, want, shape);
        if (!t.is_contiguous()) throw Refused(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }

    void* workspace(const at::Tensor& t, int64_t* bytes) const {
        if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
            throw Refused("workspace must be contiguous on cuda:" + std::to_string(device));
        *bytes = t.numel() * static_cast<int64_t>(t.element_size());
        return t.data_ptr();
    }
};

void* ptr(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

// A 16-bit cache: one stride between the pages of K and of V, each page dense.
struct Pages {
    void* k;
    void* v;
    int64_t stride, pages, page_size;

    Pages(const Place& p, const at::Tensor& kp, const at::Tensor& vp, int64_t Hkv, int64_t D) {
        pages = kp.dim() == 4 ? kp.size(0) : 0;
        page_size = kp.dim() == 4 ? kp.size(2) : 0;
        p.shaped("k_pages", kp, p.type, {pages, Hkv, page_size, D});
        p.shaped("v_pages", vp, p.type, {pages, Hkv, page_size, D});
        int64_t s[2];
        int i = 0;
        for (const at::Tensor* t : {&kp, &vp}) {
            if (t->stride(3) != 1 || (page_size > 1 && t->stride(2) != D) || (Hkv > 1 && t->stride(1) != page_size * D))
                throw Refused("each page of the cache must be contiguous");
            s[i++] = pages > 1 ? t->stride(0) : Hkv * page_size * D;
        }
        if (s[0] != s[1]) throw Refused("k_pages and v_pages must have one page stride");
        stride = s[0];
        k = kp.data_ptr();
        v = vp.data_ptr();
    }
};

// A 4-bit cache, dense.
struct PagesKv4 {
    void *kc, *ks, *vc, *vs;
    int64_t pages, page_size;

    PagesKv4(const Place& p, const at::Tensor& k_codes, const at::Tensor& k_scales, const at::Tensor& v_codes,
             const at::Tensor& v_scales, int64_t Hkv, int64_t D) {
        pages = k_codes.dim() == 4 ? k_codes.size(0) : 0;
        page_size = k_codes.dim() == 4 ? k_codes.size(2) : 0;
        kc = p.dense("k_codes", k_codes, at::kByte, {pages, Hkv, page_size, D / 2});
        ks = p.dense("k_scales", k_scales, at::kHalf, {pages, Hkv, page_size, D / 32, 2});
        vc = p.dense("v_codes", v_codes, at::kByte, {pages, Hkv, page_size, D / 2});
        vs = p.dense("v_scales", v_scales, at::kHalf, {pages, Hkv, page_size, D / 32, 2});
    }
};

// Calls the library with `device` current, on `stream` (-1: torch's current one).
template <typename F>
PyObject* run(const Place& p, int64_t stream, F&& call) {
    const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(p.device)));
    const fattn_stream_t s = stream == -1
                                 ? c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(p.device)).stream()
                                 : reinterpret_cast<fattn_stream_t>(stream);
    return PyLong_FromLong(call(s));
}

// No C++ exception leaves a function.
template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const Refused& e) {
        PyErr_Clear();
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_Clear();
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject* py_fwd_packed(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a{args, n};
        const at::Tensor &q = a.tensor("q"), &k = a.tensor("k"), &v = a.tensor("v"), &cu = a.tensor("cu_seqlens");
        const at::Tensor& out = a.tensor("out");
        const at::Tensor* lse = a.maybe("lse");
        const at::Tensor& ws = a.tensor("workspace");
        const float scale = static_cast<float>(a.number());
        const int causal = static_cast<int>(a.integer());
        const int64_t stream = a.integer();
        a.done();
        const Place p(q, "q", 3);
        const int64_t T = q.size(0), H = q.size(1), D = q.size(2), Hkv = k.dim() == 3 ? k.size(1) : 0;
        const int64_t B = cu.dim() == 1 ? cu.size(0) - 1 : -1;
        if (B < 0) throw Refused("cu_seqlens must be [B + 1]");
        int64_t st[8], ws_bytes;
        p.rows("q", &q, {T, H, D}, st);
        p.rows("k", &k, {T, Hkv, D}, st + 2);
        p.rows("v", &v, {T, Hkv, D}, st + 4);
        p.rows("out", &out, {T, H, D}, st + 6);
        const int32_t* table = static_cast<int32_t*>(p.dense("cu_seqlens", cu, at::kInt, {B + 1}));
        float* l = lse ? static_cast<float*>(p.dense("lse", *lse, at::kFloat, {H, T})) : nullptr;
        void* w = p.workspace(ws, &ws_bytes);
        return run(p, stream, [&](fattn_stream_t s) {
            return fattn_fwd_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), l, st, table, w, ws_bytes, B,
                                    T, H, Hkv, D, scale, causal, p.dtype, s);
        });
    });
}

// What both appends take after the cache: slots, pos, cos, sin, interleaved, q, q_out, k_out.
struct Append {
    int64_t T, H = 0, Hkv, D, max_pos = 0, rot = 0;
    int interleaved;
    const int64_t* slots;
    const int32_t* pos = nullptr;
    const float *cos = nullptr, *sin = nullptr;
    const at::Tensor *q, *q_out, *k_out;
    int64_t strides[12];

    Append(Args& a, const Place& p, const at::Tensor& k, const at::Tensor& v) {
        T = k.size(0);
        Hkv = k.size(1);
        D = k.size(2);
        const at::Tensor& slots_t = a.tensor("slots");
        const at::Tensor *pos_t = a.maybe("pos"), *cos_t = a.maybe("cos"), *sin_t = a.maybe("sin");
        interleaved = static_cast<int>(a.integer());
        q = a.maybe("q");
        q_out = a.maybe("q_out");
        k_out = a.maybe("k_out");
        if ((q != nullptr) != (q_out != nullptr)) throw Refused("q_out needs q");
        if (q) H = q->dim() == 3 ? q->size(1) : -1;
        slots = static_cast<int64_t*>(p.dense("slots", slots_t, at::kLong, {T}));
        if (cos_t || sin_t) {
            if (!cos_t || !sin_t || !pos_t || cos_t->dim() != 2)
                throw Refused("a rotation needs pos, and cos and sin [max_pos, rot/2]");
            max_pos = cos_t->size(0);
            rot = 2 * cos_t->size(1);
            pos = static_cast<int32_t*>(p.dense("pos", *pos_t, at::kInt, {T}));
            cos = static_cast<float*>(p.dense("cos", *cos_t, at::kFloat, {max_pos, rot / 2}));
            sin = static_cast<float*>(p.dense("sin", *sin_t, at::kFloat, {max_pos, rot / 2}));
        }
        p.rows("q", q, {T, H, D}, strides);
        p.rows("k", &k, {T, Hkv, D}, strides + 2);
        p.rows("v", &v, {T, Hkv, D}, strides + 4);
        p.rows("q_out", q_out, {T, H, D}, strides + 6);
        p.rows("k_out", k_out, {T, Hkv, D}, strides + 8);
    }
};

PyObject* py_cache_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a{args, n};
        const at::Tensor &k = a.tensor("k"), &v = a.tensor("v"), &kp = a.tensor("k_pages"), &vp = a.tensor("v_pages");
        const Place p(k, "k", 3);
        const Append x(a, p, k, v);
        const int64_t stream = a.integer();
        a.done();
        const Pages c(p, kp, vp, x.Hkv, x.D);
        return run(p, stream, [&](fattn_stream_t s) {
            return fattn_cache_append(ptr(x.q), k.data_ptr(), v.data_ptr(), ptr(x.q_out), ptr(x.k_out), x.strides, c.k, c.v,
                                      c.stride, c.pages, c.page_size, x.slots, x.pos, x.cos, x.sin, x.max_pos, x.rot,
                                      x.interleaved, x.T, x.H, x.Hkv, x.D, p.dtype, s);
        });
    });
}

PyObject* py_cache_append_kv4(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a{args, n};
        const at::Tensor &k = a.tensor("k"), &v = a.tensor("v"), &kc = a.tensor("k_codes"), &ks = a.tensor("k_scales"),
                         &vc = a.tensor("v_codes"), &vs = a.tensor("v_scales");
        const Place p(k, "k", 3);
        Append x(a, p, k, v);
        const at::Tensor* v_out = a.maybe("v_out");
        const int held = static_cast<int>(a.integer());
        const int64_t stream = a.integer();
        a.done();
        p.rows("v_out", v_out, {x.T, x.Hkv, x.D}, x.strides + 10);
        const PagesKv4 c(p, kc, ks, vc, vs, x.Hkv, x.D);
        return run(p, stream, [&](fattn_stream_t s) {
            return fattn_cache_append_kv4(ptr(x.q), k.data_ptr(), v.data_ptr(), ptr(x.q_out), ptr(x.k_out), ptr(v_out),
                                          x.strides, c.kc, c.ks, c.vc, c.vs, c.pages, c.page_size, x.slots, x.pos, x.cos,
                                          x.sin, x.max_pos, x.rot, x.interleaved, held, x.T, x.H, x.Hkv, x.D, p.dtype, s);
        });
    });
}

// What both decodes take after the cache: block_table, seq_lens, scale, out, lse, workspace.
struct Decode {
    int64_t B, H, Nq, D, width, ws_bytes;
    float scale;
    const int32_t *table, *lens;
    const at::Tensor* out;
    float* lse;
    void* ws;
    int64_t strides[6];

    Decode(Args& a, const Place& p, const at::Tensor& q) {
        B = q.size(0);
        H = q.size(1);
        Nq = q.size(2);
        D = q.size(3);
        const at::Tensor &table_t = a.tensor("block_table"), &lens_t = a.tensor("seq_lens");
        scale = static_cast<float>(a.number());
        out = &a.tensor("out");
        const at::Tensor* lse_t = a.maybe("lse");
        const at::Tensor& ws_t = a.tensor("workspace");
        width = table_t.dim() == 2 ? table_t.size(1) : 0;
        table = static_cast<int32_t*>(p.dense("block_table", table_t, at::kInt, {B, width}));
        lens = static_cast<int32_t*>(p.dense("seq_lens", lens_t, at::kInt, {B}));
        lse = lse_t ? static_cast<float*>(p.dense("lse", *lse_t, at::kFloat, {B, H, Nq})) : nullptr;
        ws = p.workspace(ws_t, &ws_bytes);
        p.rows("q", &q, {B, H, Nq, D}, strides);
        p.rows("out", out, {B, H, Nq, D}, strides + 3);
    }
};

PyObject* py_decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a{args, n};
        const at::Tensor &q = a.tensor("q"), &kp = a.tensor("k_pages"), &vp = a.tensor("v_pages");
        const Place p(q, "q", 4);
        const Decode x(a, p, q);
        const int64_t stream = a.integer();
        a.done();
        const int64_t Hkv = kp.dim() == 4 ? kp.size(1) : 0;
        const Pages c(p, kp, vp, Hkv, x.D);
        return run(p, stream, [&](fattn_stream_t s) {
            return fattn_decode(q.data_ptr(), x.out->data_ptr(), x.lse, x.strides, c.k, c.v, c.stride, c.pages, c.page_size,
                                x.table, x.width, x.lens, x.ws, x.ws_bytes, x.B, x.H, Hkv, x.Nq, x.D, x.scale, p.dtype, s);
        });
    });
}

PyObject* py_decode_kv4(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a{args, n};
        const at::Tensor &q = a.tensor("q"), &kc = a.tensor("k_codes"), &ks = a.tensor("k_scales"), &vc = a.tensor("v_codes"),
                         &vs = a.tensor("v_scales");
        const Place p(q, "q", 4);
        const Decode x(a, p, q);
        const int64_t stream = a.integer();
        a.done();
        const int64_t Hkv = kc.dim() == 4 ? kc.size(1) : 0;
        const PagesKv4 c(p, kc, ks, vc, vs, Hkv, x.D);
        return run(p, stream, [&](fattn_stream_t s) {
            return fattn_decode_kv4(q.data_ptr(), x.out->data_ptr(), x.lse, x.strides, c.kc, c.ks, c.vc, c.vs, c.pages,
                                    c.page_size, x.table, x.width, x.lens, x.ws, x.ws_bytes, x.B, x.H, Hkv, x.Nq, x.D,
                                    x.scale, p.dtype, s);
        });
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_fwd_packed>("fwd_packed"),
                         method<py_cache_append>("cache_append"),
                         method<py_cache_append_kv4>("cache_append_kv4"),
                         method<py_decode>("decode"),
                         method<py_decode_kv4>("decode_kv4"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fattn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fattn_binding() { return PyModule_Create(&module_def); }
