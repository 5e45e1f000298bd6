// heads_binding.cpp -- argument marshalling of the operators on attention heads,
// compiled: these calls take up to fifteen tensors with strides, and a served
// model makes them for single tokens, where reading the tensors' shapes from
// Python takes several times as long as the kernels.  Each function checks its
// tensors (types, shapes, the current device), then calls the C entry point of
// the same name on the current torch stream or the one given.  A status that is
// not NRM_OK raises NrmError.
//
// The functions take positional arguments only; _binding.py gives them their
// names, defaults and documentation.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <string>

#include "libnorm.h"

namespace {

PyObject* g_error = nullptr;  // NrmError

struct Raised {};  // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& text) {
    PyErr_SetString(type, text.c_str());
    throw Raised{};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + (s.size() == 1 ? ",)" : ")");
}
std::string type_text(const at::Tensor& t) { return c10::toString(t.scalar_type()); }

// The tensor of an argument; nullptr for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
    if (optional && o == Py_None) return nullptr;
    if (!THPVariable_Check(o))
        raise(o == Py_None ? PyExc_ValueError : PyExc_TypeError, std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}

nrm_dtype dtype_of(const at::Tensor& t, const char* name) {
    switch (t.scalar_type()) {
    case at::kFloat: return NRM_F32;
    case at::kHalf: return NRM_F16;
    case at::kBFloat16: return NRM_BF16;
    default: raise(PyExc_TypeError, std::string(name) + ": unsupported dtype " + type_text(t));
    }
}

void same_type(const at::Tensor& t, const at::Tensor& like, const char* name) {
    if (t.scalar_type() != like.scalar_type())
        raise(PyExc_TypeError, std::string(name) + " is " + type_text(t) + ", expected " + type_text(like));
}

// [tokens, heads, d] or [batch, tokens, heads, d] whose batch and tokens have one
// stride, with contiguous rows.
struct View {
    nrm_heads c{};
    int64_t tokens = 0, d = 0;
    const nrm_heads* ptr = nullptr;  // &c, or nullptr without a tensor
    View() = default;
    View(const View&) = delete;
    void set(const at::Tensor& t, const char* name, const at::Tensor* like_shape = nullptr,
             const at::Tensor* like_type = nullptr) {
        const auto sh = t.sizes(), st = t.strides();
        const size_t n = sh.size();
        if (like_shape && sh != like_shape->sizes())
            raise(PyExc_ValueError, std::string(name) + " has shape " + shape_text(sh) + ", expected " +
                                        shape_text(like_shape->sizes()));
        if (like_type) same_type(t, *like_type, name);
        int64_t ts = 0;
        if (n == 3) {
            tokens = sh[0];
            ts = st[0];
        } else if (n == 4) {
            ts = sh[1] > 1 ? st[1] : st[0];
            if (sh[0] > 1 && sh[1] > 1 && st[0] != sh[1] * st[1])
                raise(PyExc_ValueError, std::string(name) + ": batch and token dimensions must have one stride");
            tokens = sh[0] * sh[1];
        } else {
            raise(PyExc_ValueError, std::string(name) + " must be [tokens, heads, d] or [batch, tokens, heads, d]");
        }
        d = sh[n - 1];
        if (d > 1 && st[n - 1] != 1) raise(PyExc_ValueError, std::string(name) + ": rows must be contiguous");
        c = nrm_heads{t.data_ptr(), sh[n - 2], ts, st[n - 2]};
        ptr = &c;
    }
};

// A contiguous tensor of n values, or none.
template <bool VECTOR>
void* dense(const at::Tensor* t, const char* name, int64_t n, at::ScalarType type) {
    if (!t) return nullptr;
    if (t->scalar_type() != type)
        raise(PyExc_TypeError, std::string(name) + " is " + type_text(*t) + ", expected " + c10::toString(type));
    if (t->numel() != n || !t->is_contiguous() || (VECTOR && t->dim() != 1))
        raise(PyExc_ValueError, std::string(name) + " must be a contiguous " + (VECTOR ? "vector" : "tensor") + " of " +
                                    std::to_string(n) + " values, got " + shape_text(t->sizes()));
    return t->data_ptr();
}

struct Rope {
    nrm_rope c{};
    const nrm_rope* ptr = nullptr;
    PyObject* bytes = nullptr;  // holds the axis map during the call
    Rope() = default;
    Rope(const Rope&) = delete;
    ~Rope() { Py_XDECREF(bytes); }
    void set(const at::Tensor* pos, const at::Tensor* inv, PyObject* axis, PyObject* pairs, int64_t tokens) {
        if (!inv) return;
        if (inv->scalar_type() != at::kFloat || inv->dim() != 1 || !inv->is_contiguous())
            raise(PyExc_TypeError, "inv_freq must be a contiguous float32 vector");
        if (!pos || pos->scalar_type() != at::kLong) raise(PyExc_TypeError, "pos must be an int64 tensor");
        if (!pos->is_contiguous()) raise(PyExc_ValueError, "pos must be contiguous");
        const int64_t n = inv->numel();
        if (n > (int64_t(1) << 29)) raise(PyExc_ValueError, "inv_freq has too many values");
        const int64_t axes = axis == Py_None ? 1 : (pos->dim() ? pos->size(0) : 1);
        if (pos->numel() != axes * tokens)
            raise(PyExc_ValueError, "pos has " + std::to_string(pos->numel()) + " values, expected " +
                                        std::to_string(axes) + " axes of " + std::to_string(tokens) + " tokens");
        if (axis != Py_None) {
            bytes = PyObject_Bytes(axis);
            if (!bytes) throw Raised{};
            if (PyBytes_GET_SIZE(bytes) != n)
                raise(PyExc_ValueError, "axis has " + std::to_string(PyBytes_GET_SIZE(bytes)) +
                                            " entries, expected one for each of " + std::to_string(n) + " pairs");
            c.axis = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(bytes));
        }
        if (PyUnicode_Check(pairs) && PyUnicode_CompareWithASCIIString(pairs, "half") == 0) c.pairs = NRM_PAIRS_HALF;
        else if (PyUnicode_Check(pairs) && PyUnicode_CompareWithASCIIString(pairs, "pair") == 0)
            c.pairs = NRM_PAIRS_ADJACENT;
        else raise(PyExc_ValueError, "pairs must be 'half' or 'pair'");
        c.pos = pos->data_ptr<int64_t>();
        c.pos_stride = tokens;
        c.inv_freq = inv->data_ptr<float>();
        c.rot = int32_t(2 * n);
        c.axes = int32_t(axes);
        ptr = &c;
    }
};

// Every tensor lies on the current CUDA device, where the call launches.
void on_device(std::initializer_list<const at::Tensor*> tensors) {
    int current = -1;
    for (const at::Tensor* t : tensors) {
        if (!t) continue;
        if (t->is_cuda() && current < 0) current = c10::cuda::current_device();
        if (!t->is_cuda() || t->get_device() != current)
            raise(PyExc_ValueError, "tensors must be on the current CUDA device, got " + t->device().str());
    }
}

nrm_stream_t stream_of(PyObject* o) {
    if (o == Py_None) return reinterpret_cast<nrm_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    PyObject* v = PyObject_HasAttrString(o, "cuda_stream") ? PyObject_GetAttrString(o, "cuda_stream") : PyNumber_Long(o);
    if (!v) throw Raised{};
    void* p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) throw Raised{};
    return static_cast<nrm_stream_t>(p);
}

float number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (PyErr_Occurred()) throw Raised{};
    return float(v);
}

template <typename F>
void call(const char* name, F&& f) {
    nrm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f();
    Py_END_ALLOW_THREADS
    if (st == NRM_OK) return;
    PyObject* e = PyObject_CallFunction(g_error, "iss", int(st), name, nrm_last_error_message());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

// Runs a function's body on its n arguments; no C++ exception leaves it.
template <typename F>
PyObject* entry(PyObject* const* args, Py_ssize_t given, Py_ssize_t n, F&& f) {
    if (given != n) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", n, given);
        return nullptr;
    }
    try {
        f(args);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

// k and its second view, with the queries' tokens, row length and type.
void key_views(View& vk, View& v2, const at::Tensor& k, const char* name, PyObject* second, const char* name2,
               const View& q, const at::Tensor& qt, const at::Tensor*& t2) {
    vk.set(k, name, nullptr, &qt);
    if (vk.tokens != q.tokens || vk.d != q.d)
        raise(PyExc_ValueError, std::string(name) + " is " + std::to_string(vk.tokens) + " tokens of " +
                                    std::to_string(vk.d) + ", the queries " + std::to_string(q.tokens) + " of " +
                                    std::to_string(q.d));
    t2 = tensor(second, name2);
    v2.set(*t2, name2, &k, &k);
}

// (q, k, wq, wk, pos, inv_freq, q_out, k_out, rstd_q, rstd_k, eps, stream, axis, pairs)
PyObject* qk_norm_rope_fwd(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 14, [](PyObject* const* o) {
        const at::Tensor &q = *tensor(o[0], "q"), *k = tensor(o[1], "k", true);
        const at::Tensor *wq = tensor(o[2], "wq", true), *wk = k ? tensor(o[3], "wk", true) : nullptr;
        const at::Tensor *pos = tensor(o[4], "pos", true), *inv = tensor(o[5], "inv_freq", true);
        const at::Tensor &qo = *tensor(o[6], "q_out"), *ko = nullptr;
        const at::Tensor *rq = tensor(o[8], "rstd_q", true), *rk = k ? tensor(o[9], "rstd_k", true) : nullptr;
        View vq, vqo, vk, vko;
        Rope rope;
        vq.set(q, "q");
        vqo.set(qo, "q_out", &q, &q);
        if (k) key_views(vk, vko, *k, "k", o[7], "k_out", vq, q, ko);
        const nrm_dtype dt = dtype_of(q, "q");
        const void* pwq = dense<true>(wq, "wq", vq.d, q.scalar_type());
        const void* pwk = dense<true>(wk, "wk", vq.d, q.scalar_type());
        auto* prq = static_cast<float*>(dense<false>(rq, "rstd_q", vq.tokens * vq.c.heads, at::kFloat));
        auto* prk = static_cast<float*>(dense<false>(rk, "rstd_k", vk.tokens * vk.c.heads, at::kFloat));
        rope.set(pos, inv, o[12], o[13], vq.tokens);
        on_device({&q, k, &qo, ko, wq, wk, inv ? pos : nullptr, inv, rq, rk});
        const float eps = number(o[10]);
        const nrm_stream_t s = stream_of(o[11]);
        call("nrm_qk_norm_rope_fwd", [&] {
            return nrm_qk_norm_rope_fwd(vq.ptr, vk.ptr, pwq, pwk, rope.ptr, vqo.ptr, vko.ptr, prq, prk, vq.tokens, vq.d,
                                        eps, dt, s);
        });
    });
}

// (dq_out, dk_out, q, k, wq, wk, rstd_q, rstd_k, pos, inv_freq, dq, dk, dwq, dwk, workspace, stream, axis, pairs)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 18, [](PyObject* const* o) {
        const at::Tensor &dqo = *tensor(o[0], "dq_out"), &q = *tensor(o[2], "q"), *k = tensor(o[3], "k", true);
        const at::Tensor *wq = tensor(o[4], "wq", true), *wk = k ? tensor(o[5], "wk", true) : nullptr;
        const at::Tensor *rq = tensor(o[6], "rstd_q", true), *rk = k ? tensor(o[7], "rstd_k", true) : nullptr;
        const at::Tensor *pos = tensor(o[8], "pos", true), *inv = tensor(o[9], "inv_freq", true);
        const at::Tensor &dq = *tensor(o[10], "dq"), *dko = nullptr, *dk = nullptr;
        const at::Tensor *dwq = tensor(o[12], "dwq", true), *dwk = tensor(o[13], "dwk", true);
        const at::Tensor* ws = tensor(o[14], "workspace", true);
        View vq, vdqo, vdq, vk, vdko, vdk;
        Rope rope;
        vq.set(q, "q");
        vdqo.set(dqo, "dq_out", &q, &q);
        vdq.set(dq, "dq", &q, &q);
        if (k) {
            key_views(vk, vdko, *k, "k", o[1], "dk_out", vq, q, dko);
            dk = tensor(o[11], "dk");
            vdk.set(*dk, "dk", k, k);
        }
        const nrm_dtype dt = dtype_of(q, "q");
        const at::ScalarType type = q.scalar_type();
        const void *pwq = dense<true>(wq, "wq", vq.d, type), *pwk = dense<true>(wk, "wk", vq.d, type);
        void *pdwq = dense<true>(dwq, "dwq", vq.d, type), *pdwk = dense<true>(dwk, "dwk", vq.d, type);
        auto* prq = static_cast<const float*>(dense<false>(rq, "rstd_q", vq.tokens * vq.c.heads, at::kFloat));
        auto* prk = static_cast<const float*>(dense<false>(rk, "rstd_k", vk.tokens * vk.c.heads, at::kFloat));
        if (ws && !ws->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
        rope.set(pos, inv, o[16], o[17], vq.tokens);
        on_device({&q, k, &dqo, &dq, dko, dk, wq, wk, dwq, dwk, rq, rk, inv ? pos : nullptr, inv, ws});
        const nrm_stream_t s = stream_of(o[15]);
        call("nrm_qk_norm_rope_bwd", [&] {
            return nrm_qk_norm_rope_bwd(vdqo.ptr, vdko.ptr, vq.ptr, vk.ptr, pwq, pwk, prq, prk, rope.ptr, vdq.ptr,
                                        vdk.ptr, pdwq, pdwk, vq.tokens, vq.d, dt, ws ? ws->data_ptr() : nullptr,
                                        ws ? size_t(ws->nbytes()) : 0, s);
        });
    });
}

// (q, k, pos, inv_freq, q_out, k_out, stream, axis, pairs)
PyObject* rope_call(PyObject* const* args, Py_ssize_t given, bool inverse) {
    return entry(args, given, 9, [inverse](PyObject* const* o) {
        const char* n[4] = {inverse ? "dq_out" : "q", inverse ? "dk_out" : "k", inverse ? "dq" : "q_out",
                            inverse ? "dk" : "k_out"};
        const at::Tensor &q = *tensor(o[0], n[0]), *k = tensor(o[1], n[1], true);
        const at::Tensor *pos = tensor(o[2], "pos", true), *inv = tensor(o[3], "inv_freq", true);
        const at::Tensor &qo = *tensor(o[4], n[2]), *ko = nullptr;
        View vq, vqo, vk, vko;
        Rope rope;
        vq.set(q, n[0]);
        vqo.set(qo, n[2], &q, &q);
        if (k) key_views(vk, vko, *k, n[1], o[5], n[3], vq, q, ko);
        const nrm_dtype dt = dtype_of(q, n[0]);
        rope.set(pos, inv, o[7], o[8], vq.tokens);
        on_device({&q, k, &qo, ko, inv ? pos : nullptr, inv});
        const nrm_stream_t s = stream_of(o[6]);
        call(inverse ? "nrm_rope_bwd" : "nrm_rope_fwd", [&] {
            return (inverse ? nrm_rope_bwd : nrm_rope_fwd)(vq.ptr, vk.ptr, rope.ptr, vqo.ptr, vko.ptr, vq.tokens, vq.d,
                                                           dt, s);
        });
    });
}
PyObject* rope_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) { return rope_call(args, n, false); }
PyObject* rope_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) { return rope_call(args, n, true); }

// A KvCache: the address of its C description, and one of its tensors.
struct Cache {
    const nrm_kv_cache* c;
    const at::Tensor* held;
    Cache(PyObject* address, PyObject* tensor_of)
        : c(static_cast<const nrm_kv_cache*>(PyLong_AsVoidPtr(address))), held(tensor(tensor_of, "cache")) {
        if (PyErr_Occurred()) throw Raised{};
    }
    void rows(View& v, const at::Tensor& t, const char* name, const at::Tensor* like_type) const {
        v.set(t, name, nullptr, like_type);
        if (v.d != c->d || v.c.heads != c->heads)
            raise(PyExc_ValueError, std::string(name) + ": rows are " + std::to_string(v.c.heads) + " heads of " +
                                        std::to_string(v.d) + ", the cache's " + std::to_string(c->heads) + " of " +
                                        std::to_string(c->d));
    }
};

const int64_t* slots_ptr(const at::Tensor& t, int64_t tokens) {
    if (t.scalar_type() != at::kLong || t.numel() != tokens || !t.is_contiguous())
        raise(PyExc_ValueError, "slots must be " + std::to_string(tokens) + " contiguous int64 values");
    return t.data_ptr<int64_t>();
}

// (cache address, cache tensor, slots, k, v, stream)
PyObject* cache_call(PyObject* const* args, Py_ssize_t given, bool read) {
    return entry(args, given, 6, [read](PyObject* const* o) {
        const char *nk = read ? "k_out" : "k", *nv = read ? "v_out" : "v";
        const Cache cache(o[0], o[1]);
        const at::Tensor &slots = *tensor(o[2], "slots"), *k = tensor(o[3], nk, true), *v = tensor(o[4], nv, true);
        const at::Tensor* any = k ? k : v;
        if (!any) raise(PyExc_ValueError, std::string(nk) + " and " + nv + " must not both be None");
        View vk, vv;
        if (k) cache.rows(vk, *k, nk, nullptr);
        if (v) cache.rows(vv, *v, nv, any);
        const int64_t tokens = k ? vk.tokens : vv.tokens;
        if (k && v && vk.tokens != vv.tokens)
            raise(PyExc_ValueError, std::string(nv) + " has " + std::to_string(vv.tokens) + " tokens, expected " +
                                        std::to_string(tokens));
        const nrm_dtype dt = dtype_of(*any, nk);
        const int64_t* ps = slots_ptr(slots, tokens);
        on_device({k, v, &slots, cache.held});
        const nrm_stream_t s = stream_of(o[5]);
        if (read)
            call("nrm_kv_cache_read", [&] { return nrm_kv_cache_read(cache.c, ps, vk.ptr, vv.ptr, tokens, dt, s); });
        else
            call("nrm_kv_cache_write", [&] { return nrm_kv_cache_write(vk.ptr, vv.ptr, cache.c, ps, tokens, dt, s); });
    });
}
PyObject* kv_cache_write(PyObject*, PyObject* const* args, Py_ssize_t n) { return cache_call(args, n, false); }
PyObject* kv_cache_read(PyObject*, PyObject* const* args, Py_ssize_t n) { return cache_call(args, n, true); }

// (q, k, v, wq, wk, pos, inv_freq, q_out, k_out, cache address, cache tensor, slots, eps, stream, axis, pairs, norm)
PyObject* qk_norm_rope_cache(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 17, [](PyObject* const* o) {
        const at::Tensor &q = *tensor(o[0], "q"), &k = *tensor(o[1], "k"), &v = *tensor(o[2], "v");
        const at::Tensor *wq = tensor(o[3], "wq", true), *wk = tensor(o[4], "wk", true);
        const at::Tensor *pos = tensor(o[5], "pos", true), *inv = tensor(o[6], "inv_freq", true);
        const at::Tensor &qo = *tensor(o[7], "q_out"), *ko = tensor(o[8], "k_out", true);
        const Cache cache(o[9], o[10]);
        const at::Tensor& slots = *tensor(o[11], "slots");
        View vq, vk, vv, vqo, vko;
        Rope rope;
        vq.set(q, "q");
        vqo.set(qo, "q_out", &q, &q);
        cache.rows(vk, k, "k", &q);
        cache.rows(vv, v, "v", &q);
        if (vk.tokens != vq.tokens || vv.tokens != vq.tokens)
            raise(PyExc_ValueError, "k and v must have the " + std::to_string(vq.tokens) + " tokens of q");
        if (ko) vko.set(*ko, "k_out", &k, &q);
        const nrm_dtype dt = dtype_of(q, "q");
        const void* pwq = dense<true>(wq, "wq", vq.d, q.scalar_type());
        const void* pwk = dense<true>(wk, "wk", vq.d, q.scalar_type());
        rope.set(pos, inv, o[14], o[15], vq.tokens);
        const int64_t* ps = slots_ptr(slots, vq.tokens);
        on_device({&q, &k, &v, &qo, ko, wq, wk, inv ? pos : nullptr, inv, &slots, cache.held});
        const float eps = number(o[12]);
        const int norm = PyObject_IsTrue(o[16]);
        if (norm < 0) throw Raised{};
        const nrm_stream_t s = stream_of(o[13]);
        call("nrm_qk_norm_rope_cache", [&] {
            return nrm_qk_norm_rope_cache(vq.ptr, vk.ptr, vv.ptr, pwq, pwk, rope.ptr, vqo.ptr, vko.ptr, cache.c, ps,
                                          vq.tokens, vq.d, eps, norm, dt, s);
        });
    });
}

// (NrmError)
PyObject* set_error(PyObject*, PyObject* type) {
    Py_INCREF(type);
    Py_XSETREF(g_error, type);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<qk_norm_rope_fwd>("qk_norm_rope_fwd"),
    method<qk_norm_rope_bwd>("qk_norm_rope_bwd"),
    method<rope_fwd>("rope_fwd"),
    method<rope_bwd>("rope_bwd"),
    method<kv_cache_write>("kv_cache_write"),
    method<kv_cache_read>("kv_cache_read"),
    method<qk_norm_rope_cache>("qk_norm_rope_cache"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_heads", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__heads() { return PyModule_Create(&g_module); }
