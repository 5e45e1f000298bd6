// heads_binding.cpp -- argument marshalling of the operators on attention heads, on
// the cached sequences and between the blocks of a residual stream, compiled: these
// calls take up to fifteen tensors with strides, and a served model makes them for
// single tokens, where reading the tensors' shapes from Python takes several times
// as long as the kernels.  Each function checks its
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

// Page tables [sequences, width] with contiguous rows, and a length for each.
int64_t table_stride(const at::Tensor& t, const char* name, int64_t sequences) {
    if (t.scalar_type() != at::kLong || t.dim() != 2)
        raise(PyExc_ValueError, std::string(name) + " must be int64 [sequences, pages]");
    if (t.size(0) != sequences)
        raise(PyExc_ValueError, std::string(name) + " has " + std::to_string(t.size(0)) + " sequences, expected " +
                                    std::to_string(sequences));
    if (t.size(1) > 1 && t.stride(1) != 1) raise(PyExc_ValueError, std::string(name) + ": rows must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
struct Pages {
    nrm_kv_pages c{};
    Pages(const at::Tensor& table, const at::Tensor& lengths, int64_t sequences) {
        c.stride = table_stride(table, "table", sequences);
        c.table = table.data_ptr<int64_t>();
        c.width = table.size(1);
        c.sequences = sequences;
        c.lengths = static_cast<const int64_t*>(dense<true>(&lengths, "lengths", sequences, at::kLong));
    }
};

// [sequences, heads, positions] with contiguous rows, or none.
struct Weights {
    nrm_kv_weights c{};
    const nrm_kv_weights* ptr = nullptr;
    Weights(const at::Tensor* t, const char* name, int64_t sequences, int64_t heads) {
        if (!t) return;
        if (t->scalar_type() != at::kFloat || t->dim() != 3)
            raise(PyExc_ValueError, std::string(name) + " must be float32 [sequences, heads, positions]");
        if (t->size(0) != sequences || t->size(1) != heads)
            raise(PyExc_ValueError, std::string(name) + " has shape " + shape_text(t->sizes()) + ", expected " +
                                        std::to_string(sequences) + " sequences of " + std::to_string(heads) + " heads");
        if (t->size(2) > 1 && t->stride(2) != 1)
            raise(PyExc_ValueError, std::string(name) + ": rows must be contiguous");
        c = nrm_kv_weights{t->data_ptr<float>(), t->size(2), t->stride(0), t->stride(1)};
        ptr = &c;
    }
};

int64_t whole(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) throw Raised{};
    return v;
}

// (q, cache address, cache tensor, table, lengths, out, scale, workspace, stream, window, lse, weights)
PyObject* kv_cache_attention(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 12, [](PyObject* const* o) {
        const at::Tensor& q = *tensor(o[0], "q");
        const Cache cache(o[1], o[2]);
        const at::Tensor &table = *tensor(o[3], "table"), &lengths = *tensor(o[4], "lengths"), &out = *tensor(o[5], "out");
        const at::Tensor *ws = tensor(o[7], "workspace", true), *lse = tensor(o[10], "lse", true);
        const at::Tensor* weights = tensor(o[11], "weights", true);
        View vq, vo;
        vq.set(q, "q");
        vo.set(out, "out", &q, &q);
        if (vq.d != cache.c->d)
            raise(PyExc_ValueError, "q has rows of " + std::to_string(vq.d) + ", the cache of " + std::to_string(cache.c->d));
        const nrm_dtype dt = dtype_of(q, "q");
        const Pages pages(table, lengths, vq.tokens);
        const Weights w(weights, "weights", vq.tokens, cache.c->heads);
        auto* pl = static_cast<float*>(dense<false>(lse, "lse", vq.tokens * vq.c.heads, at::kFloat));
        if (ws && !ws->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
        const float scale = number(o[6]);
        const int64_t window = whole(o[9]);
        on_device({&q, &out, &table, &lengths, ws, lse, weights, cache.held});
        const nrm_stream_t s = stream_of(o[8]);
        call("nrm_kv_cache_attention", [&] {
            return nrm_kv_cache_attention(vq.ptr, cache.c, &pages.c, vo.ptr, scale, window, pl, w.ptr, dt,
                                          ws ? ws->data_ptr() : nullptr, ws ? size_t(ws->nbytes()) : 0, s);
        });
    });
}

// (cache address, cache tensor, table, lengths, weights, new_table, new_lengths, new_weights, kept, stream, first, recent)
PyObject* kv_cache_evict(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 12, [](PyObject* const* o) {
        const Cache cache(o[0], o[1]);
        const at::Tensor &table = *tensor(o[2], "table"), &lengths = *tensor(o[3], "lengths");
        const at::Tensor &weights = *tensor(o[4], "weights"), &new_table = *tensor(o[5], "new_table");
        const at::Tensor &new_lengths = *tensor(o[6], "new_lengths"), *new_weights = tensor(o[7], "new_weights", true);
        const at::Tensor& kept = *tensor(o[8], "kept");
        if (table.dim() != 2) raise(PyExc_ValueError, "table must be int64 [sequences, pages]");
        const int64_t sequences = table.size(0), heads = cache.c->heads;
        const Pages pages(table, lengths, sequences);
        const int64_t new_stride = table_stride(new_table, "new_table", sequences);
        const Weights w(&weights, "weights", sequences, heads), nw(new_weights, "new_weights", sequences, heads);
        auto* pl = static_cast<int64_t*>(dense<true>(&new_lengths, "new_lengths", sequences, at::kLong));
        if (kept.dim() != 3) raise(PyExc_ValueError, "kept must be int64 [sequences, heads, keep]");
        const int64_t keep = kept.size(2);
        if (kept.size(0) != sequences || kept.size(1) != heads)
            raise(PyExc_ValueError, "kept has shape " + shape_text(kept.sizes()) + ", expected " +
                                        std::to_string(sequences) + " sequences of " + std::to_string(heads) + " heads");
        auto* pk = static_cast<int64_t*>(dense<false>(&kept, "kept", sequences * heads * keep, at::kLong));
        const int64_t first = whole(o[10]), recent = whole(o[11]);
        on_device({&table, &lengths, &weights, &new_table, &new_lengths, new_weights, &kept, cache.held});
        const nrm_stream_t s = stream_of(o[9]);
        call("nrm_kv_cache_evict", [&] {
            return nrm_kv_cache_evict(cache.c, &pages.c, w.ptr, new_table.data_ptr<int64_t>(), new_table.size(1),
                                      new_stride, pl, nw.ptr, pk, keep, first, recent, s);
        });
    });
}

// Dense tensors of one shape [..., cols] and type.
struct Rows {
    int64_t rows, cols;
    at::ScalarType type;
    at::IntArrayRef shape;
    nrm_dtype dt;
    Rows(const at::Tensor& t, const char* name) : type(t.scalar_type()), shape(t.sizes()), dt(dtype_of(t, name)) {
        if (t.dim() < 1 || t.size(-1) < 1) raise(PyExc_ValueError, std::string(name) + " must be [..., cols]");
        cols = t.size(-1);
        rows = t.numel() / cols;
    }
    void* at(const at::Tensor* t, const char* name) const {
        if (!t) return nullptr;
        if (t->sizes() != shape)
            raise(PyExc_ValueError, std::string(name) + " has shape " + shape_text(t->sizes()) + ", expected " +
                                        shape_text(shape));
        return dense<false>(t, name, rows * cols, type);
    }
    void* param(const at::Tensor* t, const char* name) const { return dense<true>(t, name, cols, type); }
    // [gates, cols], or [cols] for one gate row
    void* gate(const at::Tensor* t, const char* name, int64_t* gates) const {
        *gates = 0;
        if (!t) return nullptr;
        if (t->dim() < 1 || t->size(-1) != cols)
            raise(PyExc_ValueError, std::string(name) + " must be [gates, " + std::to_string(cols) + "], got " +
                                        shape_text(t->sizes()));
        *gates = t->numel() / cols;
        if (*gates == 0 && rows > 0) raise(PyExc_ValueError, std::string(name) + " has no rows");
        return dense<false>(t, name, t->numel(), type);
    }
};

// (x, f, gate, w_post, w_pre, y, h, rstd_post, rstd_pre, alpha, eps, stream, post)
PyObject* block_norm_fwd(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 13, [](PyObject* const* o) {
        const at::Tensor &x = *tensor(o[0], "x"), &f = *tensor(o[1], "f"), *gate = tensor(o[2], "gate", true);
        const int post = PyObject_IsTrue(o[12]);
        if (post < 0) throw Raised{};
        const at::Tensor *w1 = post ? tensor(o[3], "w_post", true) : nullptr, &y = *tensor(o[5], "y");
        const at::Tensor *h = tensor(o[6], "h", true), *w2 = h ? tensor(o[4], "w_pre", true) : nullptr;
        const at::Tensor* r1 = post ? tensor(o[7], "rstd_post", true) : nullptr;
        const at::Tensor* r2 = h ? tensor(o[8], "rstd_pre", true) : nullptr;
        const Rows rows(x, "x");
        const void *px = rows.at(&x, "x"), *pf = rows.at(&f, "f"), *pw1 = rows.param(w1, "w_post");
        const void* pw2 = rows.param(w2, "w_pre");
        int64_t gates;
        const void* pg = rows.gate(gate, "gate", &gates);
        void *py = rows.at(&y, "y"), *ph = rows.at(h, "h");
        auto* p1 = static_cast<float*>(dense<false>(r1, "rstd_post", rows.rows, at::kFloat));
        auto* p2 = static_cast<float*>(dense<false>(r2, "rstd_pre", rows.rows, at::kFloat));
        on_device({&x, &f, gate, w1, w2, &y, h, r1, r2});
        const float alpha = number(o[9]), eps = number(o[10]);
        const nrm_stream_t s = stream_of(o[11]);
        call("nrm_block_norm_fwd", [&] {
            return nrm_block_norm_fwd(px, pf, pg, pw1, pw2, py, ph, p1, p2, rows.rows, rows.cols, gates, alpha, eps, post,
                                      rows.dt, s);
        });
    });
}

// (dh, dy, f, y, gate, w_post, w_pre, rstd_post, rstd_pre, dx, df, dgate, dw_post, dw_pre, workspace, alpha, stream, post)
PyObject* block_norm_bwd(PyObject*, PyObject* const* args, Py_ssize_t given) {
    return entry(args, given, 18, [](PyObject* const* o) {
        const int post = PyObject_IsTrue(o[17]);
        if (post < 0) throw Raised{};
        const at::Tensor *dh = tensor(o[0], "dh", true), *dy = tensor(o[1], "dy", true), &f = *tensor(o[2], "f");
        const at::Tensor *y = tensor(o[3], "y", !dh), *gate = tensor(o[4], "gate", true);
        const at::Tensor *w1 = post ? tensor(o[5], "w_post", true) : nullptr, *w2 = dh ? tensor(o[6], "w_pre", true) : nullptr;
        const at::Tensor* r1 = post ? tensor(o[7], "rstd_post") : nullptr;
        const at::Tensor* r2 = dh ? tensor(o[8], "rstd_pre") : nullptr;
        const at::Tensor &dx = *tensor(o[9], "dx"), &df = *tensor(o[10], "df");
        const at::Tensor *dgate = tensor(o[11], "dgate", true), *dw1 = tensor(o[12], "dw_post", true);
        const at::Tensor *dw2 = tensor(o[13], "dw_pre", true), *ws = tensor(o[14], "workspace", true);
        const Rows rows(f, "f");
        const void *pdh = rows.at(dh, "dh"), *pdy = rows.at(dy, "dy"), *pf = rows.at(&f, "f"), *py = rows.at(y, "y");
        const void *pw1 = rows.param(w1, "w_post"), *pw2 = rows.param(w2, "w_pre");
        int64_t gates, dgates;
        const void* pg = rows.gate(gate, "gate", &gates);
        void* pdg = rows.gate(dgate, "dgate", &dgates);
        if (dgate && dgates != gates)
            raise(PyExc_ValueError, "dgate has " + std::to_string(dgates) + " rows, expected " + std::to_string(gates));
        void *pdx = rows.at(&dx, "dx"), *pdf = rows.at(&df, "df");
        void *pdw1 = rows.param(dw1, "dw_post"), *pdw2 = rows.param(dw2, "dw_pre");
        const auto* p1 = static_cast<const float*>(dense<false>(r1, "rstd_post", rows.rows, at::kFloat));
        const auto* p2 = static_cast<const float*>(dense<false>(r2, "rstd_pre", rows.rows, at::kFloat));
        if (ws && !ws->is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
        on_device({dh, dy, &f, y, gate, w1, w2, r1, r2, &dx, &df, dgate, dw1, dw2, ws});
        const float alpha = number(o[15]);
        const nrm_stream_t s = stream_of(o[16]);
        call("nrm_block_norm_bwd", [&] {
            return nrm_block_norm_bwd(pdh, pdy, pf, py, pg, pw1, pw2, p1, p2, pdx, pdf, pdg, pdw1, pdw2, rows.rows,
                                      rows.cols, gates, alpha, post, rows.dt, ws ? ws->data_ptr() : nullptr,
                                      ws ? size_t(ws->nbytes()) : 0, s);
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
    method<kv_cache_attention>("kv_cache_attention"),
    method<kv_cache_evict>("kv_cache_evict"),
    method<block_norm_fwd>("block_norm_fwd"),
    method<block_norm_bwd>("block_norm_bwd"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_heads", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__heads() { return PyModule_Create(&g_module); }
