// heads_check.h -- argument checks of the calls on attention heads and on the
// key/value cache, shared by their C ABI files (heads_api.cu, kvattn_api.cu):
// sizes, views, rotations, caches, and the frame that every entry point runs in.
#pragma once

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "heads.h"

namespace nrm {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 40;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxExtent = int64_t(1) << 60;  // elements a view may span
constexpr int64_t kMaxHeads = int64_t(1) << 20;

size_t dsize(nrm_dtype dt) { return dt == NRM_F32 ? 4 : 2; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Offsets stay far from the ends of int64: n steps of `stride` each.
bool spans(int64_t n, int64_t stride, int64_t* extent) {
    if (stride < 0 || stride >= kMaxStride) return false;
    const int64_t steps = n > 0 ? n - 1 : 0;
    if (stride > 0 && steps > kMaxExtent / stride) return false;
    *extent = steps * stride;
    return true;
}

// What every call of this file has: sizes, dtype.
nrm_status check_sizes(int64_t tokens, int64_t d, nrm_dtype dt) {
    if (dt != NRM_F32 && dt != NRM_F16 && dt != NRM_BF16)
        return fail(NRM_ERR_INVALID_ARG, "unknown dtype %d", int(dt));
    if (tokens < 0) return fail(NRM_ERR_INVALID_ARG, "tokens must be >= 0");
    if (tokens >= kMaxRows) return fail(NRM_ERR_UNSUPPORTED, "tokens must be < 2^40");
    if (d < 1) return fail(NRM_ERR_INVALID_ARG, "d must be >= 1");
    if (d > kHeadMaxD) return fail(NRM_ERR_UNSUPPORTED, "d must be <= %d", kHeadMaxD);
    return NRM_OK;
}

// A view and, where it is given, the view whose heads it must match.
nrm_status check_view(const char* name, const nrm_heads* v, const nrm_heads* like, int64_t tokens, int64_t d,
                      nrm_dtype dt, bool output) {
    if (!v) return fail(NRM_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (v->heads < 1) return fail(NRM_ERR_INVALID_ARG, "%s: heads must be >= 1", name);
    if (v->heads > kMaxHeads) return fail(NRM_ERR_UNSUPPORTED, "%s: heads must be <= 2^20", name);
    if (like && v->heads != like->heads)
        return fail(NRM_ERR_INVALID_ARG, "%s has %lld heads, its input %lld", name, (long long)v->heads,
                    (long long)like->heads);
    if (tokens > kMaxRows / v->heads) return fail(NRM_ERR_UNSUPPORTED, "%s: tokens*heads must be < 2^40", name);
    if (tokens > 0 && !v->data) return fail(NRM_ERR_INVALID_ARG, "%s: data must not be NULL", name);
    if (!aligned(v->data, dsize(dt))) return fail(NRM_ERR_INVALID_ARG, "%s must be aligned to its element size", name);
    int64_t et = 0, eh = 0;
    if (!spans(tokens, v->token_stride, &et) || !spans(v->heads, v->head_stride, &eh))
        return fail(NRM_ERR_INVALID_ARG, "%s: strides must be >= 0 and span less than 2^60 elements", name);
    if (output && tokens > 0) {
        // rows of an output must not overlap: one of the two dimensions steps over all of the other
        const bool heads_inside = (v->heads == 1 || v->head_stride >= d) && (tokens == 1 || v->token_stride >= eh + d);
        const bool tokens_inside = (tokens == 1 || v->token_stride >= d) && (v->heads == 1 || v->head_stride >= et + d);
        if (!heads_inside && !tokens_inside) return fail(NRM_ERR_INVALID_ARG, "%s: rows overlap", name);
    }
    return NRM_OK;
}

// An output may be `in` itself where in_place says so, and no other input or output.
nrm_status check_place(const char* name, const nrm_heads* out, const nrm_heads* in, bool in_place, int64_t tokens) {
    if (!out || !in || tokens == 0 || out->data != in->data) return NRM_OK;
    if (in_place && (tokens == 1 || out->token_stride == in->token_stride) &&
        (out->heads == 1 || out->head_stride == in->head_stride) && out->heads == in->heads)
        return NRM_OK;
    return fail(NRM_ERR_INVALID_ARG, "%s overlaps an input or another output", name);
}

HeadView view(const nrm_heads* v) { return v ? HeadView{v->data, v->token_stride, v->head_stride} : HeadView{}; }

nrm_status set_rope(const nrm_rope* r, int64_t tokens, int64_t d, bool inverse, RopeDev* out) {
    *out = RopeDev{};
    if (!r || r->rot == 0) return NRM_OK;
    if (r->rot < 0 || r->rot > d || r->rot % 2) return fail(NRM_ERR_INVALID_ARG, "rot must be even and in [0, d]");
    if (r->axes < 1 || r->axes > kHeadMaxAxes)
        return fail(NRM_ERR_INVALID_ARG, "axes must be in [1, %d]", kHeadMaxAxes);
    if (r->pairs != NRM_PAIRS_HALF && r->pairs != NRM_PAIRS_ADJACENT)
        return fail(NRM_ERR_INVALID_ARG, "unknown pairs %d", int(r->pairs));
    if (!r->inv_freq || (tokens > 0 && !r->pos)) return fail(NRM_ERR_INVALID_ARG, "pos and inv_freq must not be NULL");
    if (!aligned(r->inv_freq, 4) || !aligned(r->pos, 8))
        return fail(NRM_ERR_INVALID_ARG, "pos and inv_freq must be aligned to their element size");
    if (r->axes > 1 && !r->axis) return fail(NRM_ERR_INVALID_ARG, "axis must not be NULL with more than one axis");
    if (r->axes > 1 && (r->pos_stride < tokens || r->pos_stride >= kMaxStride))
        return fail(NRM_ERR_INVALID_ARG, "pos_stride must be >= tokens and < 2^40");
    if (r->axis)
        for (int p = 0; p < r->rot / 2; ++p) {
            if (r->axis[p] >= r->axes)
                return fail(NRM_ERR_INVALID_ARG, "axis[%d] is %d of %d axes", p, int(r->axis[p]), int(r->axes));
            out->axis[p / 16] |= uint32_t(r->axis[p]) << (p % 16 * 2);
        }
    out->pos = r->pos;
    out->pos_stride = r->pos_stride;
    out->inv_freq = r->inv_freq;
    out->rot = r->rot;
    out->axes = r->axes;
    out->adjacent = r->pairs == NRM_PAIRS_ADJACENT;
    out->inverse = inverse;
    return NRM_OK;
}

nrm_status set_cache(const nrm_kv_cache* c, bool keys, bool values, bool written, CacheDev* out) {
    if (!c) return fail(NRM_ERR_INVALID_ARG, "cache must not be NULL");
    if (c->kind != NRM_CACHE_E4M3 && c->kind != NRM_CACHE_INT8 && c->kind != NRM_CACHE_INT4)
        return fail(NRM_ERR_INVALID_ARG, "unknown cache kind %d", int(c->kind));
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1)
        return fail(NRM_ERR_INVALID_ARG, "the cache needs pages, slots and heads");
    if (c->d < 1) return fail(NRM_ERR_INVALID_ARG, "the cache's d must be >= 1");
    if (c->d > kHeadMaxD) return fail(NRM_ERR_UNSUPPORTED, "the cache's d must be <= %d", kHeadMaxD);
    if (c->heads > kMaxHeads || c->pages > kMaxRows / c->page_size || c->pages * c->page_size > kMaxRows / c->heads)
        return fail(NRM_ERR_UNSUPPORTED, "the cache must hold fewer than 2^40 rows and 2^20 heads");
    if (c->group < 1 || c->d % c->group) return fail(NRM_ERR_INVALID_ARG, "group must divide the cache's d");
    if (c->kind == NRM_CACHE_INT4 && c->group % 2)
        return fail(NRM_ERR_INVALID_ARG, "a cache in 4 bits needs an even group");
    const int64_t bytes = c->kind == NRM_CACHE_INT4 ? c->d / 2 : c->d, scales = c->d / c->group;
    int64_t ep = 0, es = 0, eh = 0;
    if (!spans(c->pages, c->page_stride, &ep) || !spans(c->page_size, c->slot_stride, &es) ||
        !spans(c->heads, c->head_stride, &eh) || !spans(c->pages, c->scale_page_stride, &ep) ||
        !spans(c->page_size, c->scale_slot_stride, &es) || !spans(c->heads, c->scale_head_stride, &eh))
        return fail(NRM_ERR_INVALID_ARG, "the cache's strides must be >= 0 and span less than 2^60");
    // rows must not overlap: sorted by stride, each dimension steps over all that lie inside it
    for (int part = 0; part < 2; ++part) {
        int64_t n[3] = {c->pages, c->page_size, c->heads};
        int64_t st[3] = {part ? c->scale_page_stride : c->page_stride, part ? c->scale_slot_stride : c->slot_stride,
                         part ? c->scale_head_stride : c->head_stride};
        int64_t inside = part ? scales : bytes;
        bool done[3] = {n[0] == 1, n[1] == 1, n[2] == 1};
        for (int k = 0; k < 3; ++k) {
            int least = -1;
            for (int i = 0; i < 3; ++i)
                if (!done[i] && (least < 0 || st[i] < st[least])) least = i;
            if (least < 0) break;
            if (st[least] < inside) return fail(NRM_ERR_INVALID_ARG, "the cache's rows overlap");
            inside += (n[least] - 1) * st[least];
            done[least] = true;
        }
    }
    if (keys && (!c->k_codes || !c->k_scales)) return fail(NRM_ERR_INVALID_ARG, "the cache has no keys");
    if (values && (!c->v_codes || !c->v_scales)) return fail(NRM_ERR_INVALID_ARG, "the cache has no values");
    if (written && keys && values && (c->k_codes == c->v_codes || c->k_scales == c->v_scales))
        return fail(NRM_ERR_INVALID_ARG, "the cache's keys and values are the same memory");
    if (!aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return fail(NRM_ERR_INVALID_ARG, "the cache's scales must be aligned to 4 bytes");
    *out = CacheDev{};
    out->codes[0] = static_cast<uint8_t*>(c->k_codes);
    out->codes[1] = static_cast<uint8_t*>(c->v_codes);
    out->scales[0] = c->k_scales;
    out->scales[1] = c->v_scales;
    out->slots = c->pages * c->page_size;
    out->page = make_row_div(c->page_size, c->pages * c->page_size);
    out->flat = (c->pages == 1 || c->page_stride == c->page_size * c->slot_stride) &&
                (c->pages == 1 || c->scale_page_stride == c->page_size * c->scale_slot_stride);
    out->page_stride = c->page_stride;
    out->slot_stride = c->slot_stride;
    out->head_stride = c->head_stride;
    out->scale_page_stride = c->scale_page_stride;
    out->scale_slot_stride = c->scale_slot_stride;
    out->scale_head_stride = c->scale_head_stride;
    out->group = int(c->group);
    out->kind = int(c->kind);
    return NRM_OK;
}

nrm_status check_slots(const int64_t* slots, int64_t tokens) {
    if (tokens > 0 && !slots) return fail(NRM_ERR_INVALID_ARG, "slots must not be NULL");
    if (!aligned(slots, 8)) return fail(NRM_ERR_INVALID_ARG, "slots must be aligned to 8 bytes");
    return NRM_OK;
}

// The widest accesses (16 or 8 bytes, 4 of a 16-bit type; 0: single elements) that fit the views,
// the weights, rows of whole pairs of vectors (at most 32 pairs), and, where
// there is one, the cache's groups and rows of codes (`vectors` vectors' codes
// are moved at once).
int fits_vec(std::initializer_list<const nrm_heads*> views, std::initializer_list<const void*> ptrs, int64_t tokens,
             int64_t d, const RopeDev& r, nrm_dtype dt, const nrm_kv_cache* c = nullptr, int vectors = 1) {
    for (int bytes = 16; bytes >= 2 * int(dsize(dt)); bytes /= 2) {
        const int64_t v = bytes / int64_t(dsize(dt));
        bool ok = d % (2 * v) == 0 && d / (2 * v) <= 32 && r.rot % (2 * v) == 0;
        for (const nrm_heads* h : views)
            if (h && (!aligned(h->data, size_t(bytes)) || (tokens > 1 && h->token_stride % v) ||
                      (h->heads > 1 && h->head_stride % v)))
                ok = false;
        for (const void* p : ptrs) ok = ok && aligned(p, size_t(bytes));
        if (c) {
            // bytes of the codes that a lane stores or loads at once
            const int64_t b = vectors * (c->kind == NRM_CACHE_INT4 ? v / 2 : v);
            ok = ok && c->group % v == 0 && aligned(c->k_codes, size_t(b)) && aligned(c->v_codes, size_t(b)) &&
                 (c->pages == 1 || c->page_stride % b == 0) && (c->page_size == 1 || c->slot_stride % b == 0) &&
                 (c->heads == 1 || c->head_stride % b == 0);
        }
        if (ok) return bytes;
    }
    return 0;
}

template <typename F>
nrm_status by_dtype(nrm_dtype dt, F&& f) {
    switch (dt) {
    case NRM_F32: return f(float{});
    case NRM_F16: return f(__half{});
    default: return f(__nv_bfloat16{});
    }
}

// No exception leaves a C entry point (the caches of kernel attributes allocate).
template <typename F>
nrm_status entry(F&& f) noexcept {
    try {
        clear_error();
        return f();
    } catch (...) {
        return fail(NRM_ERR_CUDA, "out of host memory");
    }
}

#define NRM_TRY(call)                                          \
    do {                                                       \
        if (nrm_status st_ = (call); st_ != NRM_OK) return st_; \
    } while (0)

nrm_status check_stats(std::initializer_list<const void*> ptrs, size_t a) {
    for (const void* p : ptrs)
        if (!aligned(p, a)) return fail(NRM_ERR_INVALID_ARG, "pointers must be aligned to their element size");
    return NRM_OK;
}

nrm_status check_eps(float eps) {
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(NRM_ERR_INVALID_ARG, "eps must be finite and > 0");
    return NRM_OK;
}

}  // namespace
}  // namespace nrm
