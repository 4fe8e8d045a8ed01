// zha_bind.cpp -- argument checks and marshalling of the paged-cache and
// rotary calls for Python: tensors in, one call of the C ABI, its status out.
//
// These calls can take less time on the GPU than Python takes to look at their
// tensors' attributes (8 us of host time with the checks in Python and ctypes,
// of which the launch itself is 3), so the looking is done here, on the
// tensors themselves. Nothing here computes or launches anything; the
// functions of libzha.so are handed over by the binding (init). A call whose
// tensors cannot be passed on raises ValueError and enqueues nothing.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "zha.h"

namespace {

decltype(&zha_rotary_apply) f_rotary;
decltype(&zha_paged_plan) f_plan;
decltype(&zha_paged_write) f_write;
decltype(&zha_paged_write_check) f_write_check;
decltype(&zha_paged_decode) f_decode;
decltype(&zha_paged_workspace_bytes) f_workspace;

PyTypeObject *paged_config_type, *rotary_type;       // zha.PagedConfig and zha.Rotary
PyObject *name_desc, *name_device;

struct Refused : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct WrongType : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct Raised {};                        // a Python error is set

std::string list(at::IntArrayRef v) {
    std::string s = "[";
    for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
    return s + "]";
}
std::string shown(const at::Tensor &t) {
    std::string s = std::string(", got ") + c10::toString(t.scalar_type()) + " " + list(t.sizes());
    if (t.layout() == at::kStrided) s += " (strides " + list(t.strides()) + ")";
    return s + " on " + t.device().str();
}

at::ScalarType type_of(const zha_paged_config *c) { return c->dtype == ZHA_BF16 ? at::kBFloat16 : at::kFloat; }

// One call's arguments: its name for messages, and the device that all its tensors must be on.
struct Call {
    const char *where;
    int dev = -1;

    [[noreturn]] void refuse(const std::string &what) const { throw Refused(std::string(where) + ": " + what); }
    [[noreturn]] void refuse(const char *name, const std::string &what, const at::Tensor &t) const {
        refuse(std::string(name) + " must be " + what + shown(t));
    }

    const at::Tensor &tensor(PyObject *o, const char *name) const {
        if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided) refuse(name, "a strided tensor", t);
        return t;
    }
    // [n, heads, d] with packed heads: its address and its tokens' stride in elements
    void *rows(PyObject *o, const char *name, int64_t n, int64_t heads, int64_t d, at::ScalarType type, int64_t &stride) const {
        const at::Tensor &t = tensor(o, name);
        if (t.dim() != 3 || t.size(0) != n || t.size(1) != heads || t.size(2) != d || t.scalar_type() != type ||
            t.get_device() != dev)
            refuse(name, "[" + std::to_string(n) + ", " + std::to_string(heads) + ", " + std::to_string(d) + "] of the call's type on device " +
                             std::to_string(dev), t);
        if (n > 0 && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))) refuse(name, "a tensor whose heads are packed", t);
        // (a stride of 0 is a broadcast here, and contiguous in the C call)
        if (n > 1 && t.stride(0) < heads * d) refuse(name, "a tensor whose tokens do not overlap", t);
        stride = n > 1 ? t.stride(0) : heads * d;
        return t.data_ptr();
    }
    // contiguous, of at least n elements; None passes
    int32_t *ints(PyObject *o, const char *name, int64_t n) const {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(o, name);
        if (t.scalar_type() != at::kInt || t.get_device() != dev || !t.is_contiguous() || t.numel() < n)
            refuse(name, "a contiguous Int tensor of at least " + std::to_string(n) + " elements on device " + std::to_string(dev), t);
        return static_cast<int32_t *>(t.data_ptr());
    }
    // contiguous, of these dimensions. Neighbouring ones may be one, or split by ones: what leaves the elements in their
    // order (every dimension's stride is one of the array's); other shapes of as many elements are another layout.
    void *array(PyObject *o, const char *name, at::IntArrayRef dims, at::ScalarType type) const {
        const at::Tensor &t = tensor(o, name);
        int64_t total = 1, at = 1;
        for (int64_t d : dims) total *= d;
        bool same = t.numel() == total && t.is_contiguous();
        size_t left = dims.size();
        int64_t stride = 1;                // of dimension `left`, as if it were one of the array's
        for (int64_t i = t.dim() - 1; i >= 0 && same && total > 0; --i) {
            at *= t.size(i);
            while (stride < at && left > 0) stride *= dims[--left];
            same = stride == at;
        }
        if (!same || t.scalar_type() != type || t.get_device() != dev)
            refuse(name, std::string("a contiguous ") + c10::toString(type) + " " + list(dims) + " on device " + std::to_string(dev), t);
        return t.data_ptr();
    }
    void *pool(PyObject *o, const char *name, const zha_paged_config *c) const {
        return array(o, name, {c->n_pages, c->n_kv_heads, c->page_size, c->head_dim}, type_of(c));
    }
    // [batch, max_pages], or flat: a table of another width would be read askew
    int32_t *table(PyObject *o, const zha_paged_config *cfg) const {
        const at::Tensor &t = tensor(o, "table");
        if (t.dim() > 1 && t.size(-1) != cfg->max_pages) refuse("table", "[batch, " + std::to_string(cfg->max_pages) + "]", t);
        return ints(o, "table", (int64_t)cfg->batch * cfg->max_pages);
    }
    void on(const at::Tensor &t) {
        dev = t.get_device();
        if (!t.is_cuda()) refuse("tensors must be on a CUDA device" + shown(t));
    }
    void *stream(PyObject *o) const {
        if (o != Py_None) {
            void *st = PyLong_AsVoidPtr(o);
            if (!st && PyErr_Occurred()) throw Raised();       // not the default stream in its place
            return st;
        }
        return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    }
};


// The memory of a ctypes structure (which its owner keeps). Only of the right type: any other one would be read askew.
template <typename S>
const S *memory(PyObject *o) {
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE)) throw Raised();
    const S *p = b.len >= (Py_ssize_t)sizeof(S) ? static_cast<const S *>(b.buf) : nullptr;
    PyBuffer_Release(&b);
    if (!p) throw WrongType("a structure is too small");
    return p;
}
const zha_paged_config *config(PyObject *o) {
    if (!PyObject_TypeCheck(o, paged_config_type)) throw WrongType(std::string("a PagedConfig is needed, got ") + Py_TYPE(o)->tp_name);
    return memory<zha_paged_config>(o);
}

void is_rotary(PyObject *o) {
    if (!PyObject_TypeCheck(o, rotary_type)) throw WrongType(std::string("a Rotary is needed, got ") + Py_TYPE(o)->tp_name);
}
// The description of a rotation whose table is on the call's device; null for None.
const zha_rotary *rotation(const Call &c, PyObject *o) {
    if (o == Py_None) return nullptr;
    PyObject *device = PyObject_GetAttr(o, name_device), *desc = PyObject_GetAttr(o, name_desc);
    const zha_rotary *r = nullptr;
    long dev = -1;
    if (device && desc) {
        dev = PyLong_AsLong(device);
        try {
            r = memory<zha_rotary>(desc);
        } catch (...) {
            Py_DECREF(device);
            Py_DECREF(desc);               // (the rotation holds it)
            throw;
        }
    }
    Py_XDECREF(device);
    Py_XDECREF(desc);
    if (!r || PyErr_Occurred()) throw Raised();
    if (dev != c.dev) c.refuse("the rotary table is on another device than the tensors");
    return r;
}

template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F &&f) {
    if (n != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        const int code = f();
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(code);
    } catch (const Raised &) {
    } catch (const WrongType &e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const Refused &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// rotary, q, k, positions, q_out, k_out, transpose, stream
PyObject *rotary(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        Call c{"zha_rotary_apply"};
        is_rotary(a[0]);
        const bool has_q = a[1] != Py_None, has_k = a[2] != Py_None;
        if (!has_q && !has_k) c.refuse("q or k [n, heads, d] is needed");
        const at::Tensor &one = c.tensor(has_q ? a[1] : a[2], has_q ? "q" : "k");
        if (one.dim() != 3) c.refuse(has_q ? "q" : "k", "[n, heads, d]", one);
        c.on(one);
        const auto type = one.scalar_type();
        if (type != at::kBFloat16 && type != at::kFloat) c.refuse(has_q ? "q" : "k", "bf16 or fp32", one);
        const int64_t tokens = one.size(0), d = one.size(2), hq = has_q ? one.size(1) : 0;
        if (tokens > INT32_MAX || d > INT32_MAX || one.size(1) > INT32_MAX) c.refuse("too large");
        int64_t hk = 0, qs = 0, qos = 0, ks = 0, kos = 0;
        void *qp = nullptr, *qo = nullptr, *kp = nullptr, *ko = nullptr;
        if (has_q) {
            qp = c.rows(a[1], "q", tokens, hq, d, type, qs);
            qo = a[4] == Py_None ? (qos = qs, qp) : c.rows(a[4], "q_out", tokens, hq, d, type, qos);
        }
        if (has_k) {
            const at::Tensor &k = c.tensor(a[2], "k");
            hk = k.dim() == 3 ? k.size(1) : 0;
            kp = c.rows(a[2], "k", tokens, hk, d, type, ks);
            ko = a[5] == Py_None ? (kos = ks, kp) : c.rows(a[5], "k_out", tokens, hk, d, type, kos);
        }
        const int32_t *pos = c.ints(a[3], "positions", tokens);
        const zha_rotary *r = rotation(c, a[0]);
        const int transpose = PyObject_IsTrue(a[6]);
        if (transpose < 0) throw Raised();
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
        return (int)f_rotary(r, (int32_t)d, type == at::kFloat ? ZHA_F32 : ZHA_BF16, (int32_t)tokens, (int32_t)hq, (int32_t)hk,
                             qp, qs, kp, ks, pos, qo, qos, ko, kos, transpose, c.stream(a[7]));
    });
}

// config, table, lens, n_new, free_pages, n_free, positions, slots, seq_ids, cu, lens_out, n_free_out, status, stream
PyObject *paged_plan(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 14, [&] {
        Call c{"zha_paged_plan"};
        const zha_paged_config *cfg = config(a[0]);
        c.on(c.tensor(a[1], "table"));
        const int64_t B = cfg->batch, rows = c.tensor(a[7], "slots").numel();
        if (rows > INT32_MAX) c.refuse("the token buffer is too large");
        zha_token_map m{};
        m.positions = c.ints(a[6], "positions", rows);
        m.slots = c.ints(a[7], "slots", rows);
        m.seq_ids = c.ints(a[8], "seq_ids", rows);
        m.cu_new = c.ints(a[9], "cu", B + 1);
        m.max_tokens = (int32_t)rows;
        int32_t *lens = c.ints(a[2], "lens", B), *n_free = c.ints(a[5], "n_free", 1);
        int32_t *lens_out = a[10] == Py_None ? lens : c.ints(a[10], "lens_out", B);
        int32_t *n_free_out = a[11] == Py_None ? n_free : c.ints(a[11], "n_free_out", 1);
        int32_t *table = c.table(a[1], cfg);
        const int32_t *n_new = c.ints(a[3], "n_new", B);
        int32_t *free_pages = c.ints(a[4], "free_pages", cfg->n_pages), *status = c.ints(a[12], "dev_status", 1);
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
        return (int)f_plan(cfg, table, lens, n_new, free_pages, n_free, lens_out, n_free_out, &m, status, c.stream(a[13]));
    });
}

// config, rotary, q, k_new, v_new, positions, slots, q_out, k_pool, v_pool, status, stream, whether to check
// the arguments and no more
PyObject *paged_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        Call c{"zha_paged_write"};
        const zha_paged_config *cfg = config(a[0]);
        if (a[1] != Py_None) is_rotary(a[1]);
        c.on(c.tensor(a[8], "k_pool"));
        const auto type = type_of(cfg);
        const int64_t d = cfg->head_dim, hkv = cfg->n_kv_heads, hq = cfg->n_q_heads;
        const at::Tensor &k = c.tensor(a[3], "k_new");
        const int64_t tokens = k.dim() ? k.size(0) : 0;
        if (tokens > INT32_MAX) c.refuse("too many tokens");
        int64_t qs = 0, ks = 0, vs = 0;
        const void *kp = c.rows(a[3], "k_new", tokens, hkv, d, type, ks), *vp = c.rows(a[4], "v_new", tokens, hkv, d, type, vs);
        void *qp = nullptr, *qo = nullptr;
        if (a[2] != Py_None) {
            qp = c.rows(a[2], "q", tokens, hq, d, type, qs);
            if (a[7] == Py_None) c.refuse("q_out is needed with q");
            qo = c.array(a[7], "q_out", {tokens, hq, d}, type);
        }
        const int32_t *pos = c.ints(a[5], "positions", tokens), *slots = c.ints(a[6], "slots", tokens);
        void *k_pool = c.pool(a[8], "k_pool", cfg), *v_pool = c.pool(a[9], "v_pool", cfg);
        int32_t *status = c.ints(a[10], "dev_status", 1);
        const zha_rotary *r = rotation(c, a[1]);
        if (a[12] == Py_True)
            return (int)f_write_check(cfg, r, (int32_t)tokens, qp, qs, kp, ks, vp, vs, pos, slots, qo, k_pool, v_pool);
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
        return (int)f_write(cfg, r, (int32_t)tokens, qp, qs, kp, ks, vp, vs, pos, slots, qo, k_pool, v_pool, status,
                            c.stream(a[11]));
    });
}

// config, q, k_pool, v_pool, table, lens, out, workspace, lse, seq_ids, positions, status, stream
PyObject *paged_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 13, [&] {
        Call c{"zha_paged_decode"};
        const zha_paged_config *cfg = config(a[0]);
        const at::Tensor &q = c.tensor(a[1], "q");
        c.on(q);
        const auto type = type_of(cfg);
        const int64_t d = cfg->head_dim, hq = cfg->n_q_heads, B = cfg->batch;
        const int64_t rows = q.dim() == 3 ? q.size(0) : -1;
        if (rows < 0 || rows > INT32_MAX || q.size(1) != hq || q.size(2) != d)
            c.refuse("q", "[n, " + std::to_string(hq) + ", " + std::to_string(d) + "]", q);
        if (a[9] == Py_None && rows > B) c.refuse("q", "of no more rows than sequences where seq_ids is not given", q);
        void *qp = c.array(a[1], "q", {rows, hq, d}, type), *out = c.array(a[6], "out", {rows, hq, d}, type);
        float *lse = a[8] == Py_None ? nullptr : static_cast<float *>(c.array(a[8], "lse", {rows, hq}, at::kFloat));
        const at::Tensor &ws = c.tensor(a[7], "workspace");
        const size_t need = rows ? f_workspace(cfg, (int32_t)rows) : 0;
        if (ws.get_device() != c.dev || !ws.is_contiguous() || ws.nbytes() < need)
            c.refuse("workspace", "contiguous, on the call's device and of at least " + std::to_string(need) + " bytes", ws);
        const void *k_pool = c.pool(a[2], "k_pool", cfg), *v_pool = c.pool(a[3], "v_pool", cfg);
        const int32_t *table = c.table(a[4], cfg), *lens = c.ints(a[5], "lens", B);
        const int32_t *seq = c.ints(a[9], "seq_ids", rows), *pos = c.ints(a[10], "positions", rows);
        int32_t *status = c.ints(a[11], "dev_status", 1);
        c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.dev));
        return (int)f_decode(cfg, (int32_t)rows, qp, k_pool, v_pool, table, lens, seq, pos, out, lse, ws.data_ptr(), status,
                             c.stream(a[12]));
    });
}

// Addresses of libzha.so's functions: rotary_apply, paged_plan, paged_write, paged_decode, paged_workspace_bytes,
// paged_write_check; then the types PagedConfig and Rotary.
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 8, [&] {
        f_rotary = reinterpret_cast<decltype(f_rotary)>(PyLong_AsVoidPtr(a[0]));
        f_plan = reinterpret_cast<decltype(f_plan)>(PyLong_AsVoidPtr(a[1]));
        f_write = reinterpret_cast<decltype(f_write)>(PyLong_AsVoidPtr(a[2]));
        f_decode = reinterpret_cast<decltype(f_decode)>(PyLong_AsVoidPtr(a[3]));
        f_workspace = reinterpret_cast<decltype(f_workspace)>(PyLong_AsVoidPtr(a[4]));
        f_write_check = reinterpret_cast<decltype(f_write_check)>(PyLong_AsVoidPtr(a[5]));
        if (!PyType_Check(a[6]) || !PyType_Check(a[7])) throw WrongType("types are needed");
        Py_INCREF(a[6]);
        Py_INCREF(a[7]);
        paged_config_type = reinterpret_cast<PyTypeObject *>(a[6]);
        rotary_type = reinterpret_cast<PyTypeObject *>(a[7]);
        name_desc = PyUnicode_InternFromString("desc");
        name_device = PyUnicode_InternFromString("device");
        return 0;
    });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(init), FAST(rotary), FAST(paged_plan), FAST(paged_write), FAST(paged_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bind() {
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", ZHA_BIND_KEY)) Py_CLEAR(m);      // zha.py compares it
    return m;
}
