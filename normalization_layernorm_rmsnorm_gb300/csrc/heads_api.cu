// heads_api.cu -- the C ABI of the operators on attention heads (declared in
// include/libnorm.h): argument checks, then dispatch by storage dtype.  The
// kernels live in heads_<dtype>.cu.
#include "heads_check.h"

namespace nrm {

int head_bwd_max_partials(const DevInfo& d) { return row_bwd_max_partials(d); }

namespace {

// The forward of q and k, with or without the norm: the shared checks and arguments.
nrm_status set_fwd(const nrm_heads* q, const nrm_heads* k, const nrm_rope* rope, const nrm_heads* qo,
                   const nrm_heads* ko, bool ko_optional, int64_t tokens, int64_t d, nrm_dtype dt, bool inverse,
                   HeadArgs* a) {
    NRM_TRY(check_sizes(tokens, d, dt));
    NRM_TRY(check_view("q", q, nullptr, tokens, d, dt, false));
    NRM_TRY(check_view("q_out", qo, q, tokens, d, dt, true));
    if (k) {
        NRM_TRY(check_view("k", k, nullptr, tokens, d, dt, false));
        if (ko || !ko_optional) NRM_TRY(check_view("k_out", ko, k, tokens, d, dt, true));
    } else {
        ko = nullptr;
    }
    NRM_TRY(check_place("q_out", qo, q, true, tokens));
    NRM_TRY(check_place("q_out", qo, k, false, tokens));
    NRM_TRY(check_place("k_out", ko, k, true, tokens));
    NRM_TRY(check_place("k_out", ko, q, false, tokens));
    NRM_TRY(check_place("k_out", ko, qo, false, tokens));
    *a = HeadArgs{};
    NRM_TRY(set_rope(rope, tokens, d, inverse, &a->rope));
    a->x[0] = view(q);
    a->x[1] = view(k);
    a->y[0] = view(qo);
    a->y[1] = view(ko);
    a->tokens = tokens;
    a->heads[0] = int(q->heads);
    a->heads[1] = k ? int(k->heads) : 0;
    a->d = int(d);
    return NRM_OK;
}

}  // namespace
}  // namespace nrm

using namespace nrm;

extern "C" {

nrm_status nrm_qk_norm_rope_fwd(const nrm_heads* q, const nrm_heads* k, const void* wq, const void* wk,
                                const nrm_rope* rope, const nrm_heads* q_out, const nrm_heads* k_out, float* rstd_q,
                                float* rstd_k, int64_t tokens, int64_t d, float eps, nrm_dtype dt,
                                nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        HeadArgs a;
        NRM_TRY(set_fwd(q, k, rope, q_out, k_out, false, tokens, d, dt, false, &a));
        NRM_TRY(check_eps(eps));
        if (!k) {
            wk = nullptr;
            rstd_k = nullptr;
        }
        NRM_TRY(check_stats({wq, wk}, dsize(dt)));
        NRM_TRY(check_stats({rstd_q, rstd_k}, 4));
        if (rstd_q && rstd_q == rstd_k) return fail(NRM_ERR_INVALID_ARG, "rstd_q and rstd_k are the same memory");
        a.w[0] = wq;
        a.w[1] = wk;
        a.rstd[0] = rstd_q;
        a.rstd[1] = rstd_k;
        a.eps = eps;
        const int vec = fits_vec({q, k, q_out, k ? k_out : nullptr}, {wq, wk}, tokens, d, a.rope, dt);
        return by_dtype(dt, [&](auto tag) {
            return head_fwd<decltype(tag)>(a, true, false, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

nrm_status nrm_qk_norm_rope_bwd(const nrm_heads* dq_out, const nrm_heads* dk_out, const nrm_heads* q,
                                const nrm_heads* k, const void* wq, const void* wk, const float* rstd_q,
                                const float* rstd_k, const nrm_rope* rope, const nrm_heads* dq, const nrm_heads* dk,
                                void* dwq, void* dwk, int64_t tokens, int64_t d, nrm_dtype dt, void* workspace,
                                size_t workspace_bytes, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        NRM_TRY(check_sizes(tokens, d, dt));
        // beyond it nrm_workspace_bytes has no answer
        if (tokens > kMaxRows / d) return fail(NRM_ERR_UNSUPPORTED, "tokens*d must be <= 2^40");
        NRM_TRY(check_view("q", q, nullptr, tokens, d, dt, false));
        NRM_TRY(check_view("dq_out", dq_out, q, tokens, d, dt, false));
        NRM_TRY(check_view("dq", dq, q, tokens, d, dt, true));
        if (tokens > 0 && !rstd_q) return fail(NRM_ERR_INVALID_ARG, "rstd_q must not be NULL");
        if (k) {
            NRM_TRY(check_view("k", k, nullptr, tokens, d, dt, false));
            NRM_TRY(check_view("dk_out", dk_out, k, tokens, d, dt, false));
            NRM_TRY(check_view("dk", dk, k, tokens, d, dt, true));
            if (tokens > 0 && !rstd_k) return fail(NRM_ERR_INVALID_ARG, "rstd_k must not be NULL");
        } else if (dwk) {
            return fail(NRM_ERR_INVALID_ARG, "dwk without k");
        } else {
            dk_out = dk = nullptr;
            wk = nullptr;
            rstd_k = nullptr;
        }
        if (dwq && dwq == dwk) return fail(NRM_ERR_INVALID_ARG, "dwq and dwk are the same memory");
        for (const nrm_heads* in : {q, k, dq_out, dk_out}) {
            NRM_TRY(check_place("dq", dq, in, false, tokens));
            NRM_TRY(check_place("dk", dk, in, false, tokens));
        }
        NRM_TRY(check_place("dk", dk, dq, false, tokens));
        NRM_TRY(check_stats({wq, wk, dwq, dwk}, dsize(dt)));
        NRM_TRY(check_stats({rstd_q, rstd_k}, 4));
        HeadArgs a{};
        NRM_TRY(set_rope(rope, tokens, d, true, &a.rope));
        const DevInfo* dev = dev_info();
        if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
        if ((dwq || dwk) && tokens > 0) {
            const size_t need = nrm_workspace_bytes(NRM_OP_QK_NORM_BWD, tokens, d, dt);
            if (!workspace || !aligned(workspace, 16))
                return fail(NRM_ERR_WORKSPACE, "workspace must be non-NULL and 16-byte aligned");
            if (workspace_bytes < need)
                return fail(NRM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed",
                            workspace_bytes, need);
            a.ws = static_cast<float*>(workspace);
        }
        a.x[0] = view(q);
        a.x[1] = view(k);
        a.dy[0] = view(dq_out);
        a.dy[1] = view(dk_out);
        a.y[0] = view(dq);
        a.y[1] = view(dk);
        a.w[0] = wq;
        a.w[1] = wk;
        a.rstd[0] = const_cast<float*>(rstd_q);
        a.rstd[1] = const_cast<float*>(rstd_k);
        a.dw[0] = dwq;
        a.dw[1] = dwk;
        a.tokens = tokens;
        a.heads[0] = int(q->heads);
        a.heads[1] = k ? int(k->heads) : 0;
        a.d = int(d);
        const int vec = fits_vec({q, k, dq_out, dk_out, dq, dk}, {wq, wk}, tokens, d, a.rope, dt);
        return by_dtype(dt, [&](auto tag) {
            return head_bwd<decltype(tag)>(a, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

static nrm_status rope_only(const nrm_heads* q, const nrm_heads* k, const nrm_rope* rope, const nrm_heads* qo,
                            const nrm_heads* ko, int64_t tokens, int64_t d, nrm_dtype dt, bool inverse,
                            nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        HeadArgs a;
        NRM_TRY(set_fwd(q, k, rope, qo, ko, false, tokens, d, dt, inverse, &a));
        const int vec = fits_vec({q, k, qo, k ? ko : nullptr}, {}, tokens, d, a.rope, dt);
        return by_dtype(dt, [&](auto tag) {
            return head_fwd<decltype(tag)>(a, false, false, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

nrm_status nrm_rope_fwd(const nrm_heads* q, const nrm_heads* k, const nrm_rope* rope, const nrm_heads* q_out,
                        const nrm_heads* k_out, int64_t tokens, int64_t d, nrm_dtype dt, nrm_stream_t stream) {
    return rope_only(q, k, rope, q_out, k_out, tokens, d, dt, false, stream);
}

nrm_status nrm_rope_bwd(const nrm_heads* dq_out, const nrm_heads* dk_out, const nrm_rope* rope, const nrm_heads* dq,
                        const nrm_heads* dk, int64_t tokens, int64_t d, nrm_dtype dt, nrm_stream_t stream) {
    return rope_only(dq_out, dk_out, rope, dq, dk, tokens, d, dt, true, stream);
}

nrm_status nrm_kv_cache_write(const nrm_heads* k, const nrm_heads* v, const nrm_kv_cache* cache, const int64_t* slots,
                              int64_t tokens, nrm_dtype dt, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        HeadArgs a{};
        NRM_TRY(set_cache(cache, k != nullptr, v != nullptr, true, &a.cache));
        NRM_TRY(check_sizes(tokens, cache->d, dt));
        if (!k && !v) return fail(NRM_ERR_INVALID_ARG, "k and v must not both be NULL");
        const nrm_heads like{nullptr, cache->heads, 0, 0};
        if (k) NRM_TRY(check_view("k", k, &like, tokens, cache->d, dt, false));
        if (v) NRM_TRY(check_view("v", v, &like, tokens, cache->d, dt, false));
        NRM_TRY(check_slots(slots, tokens));
        a.x[1] = view(k);
        a.x[2] = view(v);
        a.tokens = tokens;
        a.heads[1] = int(cache->heads);
        a.d = int(cache->d);
        a.slots = slots;
        const int vec = fits_vec({k, v}, {}, tokens, a.d, a.rope, dt, cache, 2);
        return by_dtype(dt, [&](auto tag) {
            return cache_write<decltype(tag)>(a, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

nrm_status nrm_kv_cache_read(const nrm_kv_cache* cache, const int64_t* slots, const nrm_heads* k_out,
                             const nrm_heads* v_out, int64_t tokens, nrm_dtype dt, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        HeadArgs a{};
        NRM_TRY(set_cache(cache, k_out != nullptr, v_out != nullptr, false, &a.cache));
        NRM_TRY(check_sizes(tokens, cache->d, dt));
        if (!k_out && !v_out) return fail(NRM_ERR_INVALID_ARG, "k_out and v_out must not both be NULL");
        const nrm_heads like{nullptr, cache->heads, 0, 0};
        if (k_out) NRM_TRY(check_view("k_out", k_out, &like, tokens, cache->d, dt, true));
        if (v_out) NRM_TRY(check_view("v_out", v_out, &like, tokens, cache->d, dt, true));
        NRM_TRY(check_place("v_out", v_out, k_out, false, tokens));
        NRM_TRY(check_slots(slots, tokens));
        a.y[0] = view(k_out);
        a.y[1] = view(v_out);
        a.tokens = tokens;
        a.heads[1] = int(cache->heads);
        a.d = int(cache->d);
        a.slots = slots;
        const int vec = fits_vec({k_out, v_out}, {}, tokens, a.d, a.rope, dt, cache);
        return by_dtype(dt, [&](auto tag) {
            return cache_read<decltype(tag)>(a, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

nrm_status nrm_qk_norm_rope_cache(const nrm_heads* q, const nrm_heads* k, const nrm_heads* v, const void* wq,
                                  const void* wk, const nrm_rope* rope, const nrm_heads* q_out,
                                  const nrm_heads* k_out, const nrm_kv_cache* cache, const int64_t* slots,
                                  int64_t tokens, int64_t d, float eps, int norm, nrm_dtype dt,
                                  nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        HeadArgs a;
        if (!k) return fail(NRM_ERR_INVALID_ARG, "k must not be NULL");
        NRM_TRY(set_fwd(q, k, rope, q_out, k_out, true, tokens, d, dt, false, &a));
        NRM_TRY(check_view("v", v, k, tokens, d, dt, false));
        NRM_TRY(check_place("q_out", q_out, v, false, tokens));
        NRM_TRY(check_place("k_out", k_out, v, false, tokens));
        NRM_TRY(set_cache(cache, true, true, true, &a.cache));
        if (cache->heads != k->heads || cache->d != d)
            return fail(NRM_ERR_INVALID_ARG, "the cache has %lld heads of %lld, k %lld of %lld",
                        (long long)cache->heads, (long long)cache->d, (long long)k->heads, (long long)d);
        NRM_TRY(check_slots(slots, tokens));
        if (norm) {
            NRM_TRY(check_eps(eps));
            NRM_TRY(check_stats({wq, wk}, dsize(dt)));
            a.w[0] = wq;
            a.w[1] = wk;
            a.eps = eps;
        }
        a.x[2] = view(v);
        a.heads[2] = int(v->heads);
        a.slots = slots;
        const int vec = fits_vec({q, k, v, q_out, k_out}, {a.w[0], a.w[1]}, tokens, d, a.rope, dt, cache);
        return by_dtype(dt, [&](auto tag) {
            return head_fwd<decltype(tag)>(a, norm != 0, true, vec, reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

}  // extern "C"
