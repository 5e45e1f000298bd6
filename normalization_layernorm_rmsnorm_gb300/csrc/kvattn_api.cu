// kvattn_api.cu -- the C ABI of the calls that work on whole cached sequences
// (declared in include/libnorm.h): argument checks, workspace layout, then
// dispatch.  The kernels live in kvattn_<dtype>.cu and kvevict.cu.
#include "heads_check.h"
#include "kvattn.h"

namespace nrm {
namespace {

constexpr int64_t kMaxPositions = int64_t(1) << 40;
constexpr int64_t kMaxSequences = int64_t(1) << 30;
constexpr int64_t kMaxWorkspace = int64_t(1) << 48;

nrm_status check_pages(const char* name, const int64_t* table, int64_t width, int64_t stride, int64_t sequences,
                       int64_t page_size) {
    if (width < 0 || (sequences > 0 && width < 1)) return fail(NRM_ERR_INVALID_ARG, "%s: width must be >= 1", name);
    if (width > kMaxPositions / page_size)
        return fail(NRM_ERR_UNSUPPORTED, "%s: width*page_size must be <= 2^40", name);
    if (sequences > 1 && stride < width) return fail(NRM_ERR_INVALID_ARG, "%s: stride must be >= width", name);
    int64_t extent = 0;
    if (!spans(sequences, sequences > 1 ? stride : 0, &extent))
        return fail(NRM_ERR_INVALID_ARG, "%s: strides must span less than 2^60", name);
    if (sequences > 0 && !table) return fail(NRM_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (!aligned(table, 8)) return fail(NRM_ERR_INVALID_ARG, "%s must be aligned to 8 bytes", name);
    return NRM_OK;
}

// The sequences of a call and, in *cap, the positions that one may have.
nrm_status check_sequences(const nrm_kv_pages* p, const nrm_kv_cache* c, const nrm_kv_weights* w, int64_t* cap) {
    if (!p) return fail(NRM_ERR_INVALID_ARG, "pages must not be NULL");
    if (p->sequences < 0) return fail(NRM_ERR_INVALID_ARG, "sequences must be >= 0");
    if (p->sequences > kMaxSequences) return fail(NRM_ERR_UNSUPPORTED, "sequences must be <= 2^30");
    NRM_TRY(check_pages("table", p->table, p->width, p->stride, p->sequences, c->page_size));
    if (p->sequences > 0 && !p->lengths) return fail(NRM_ERR_INVALID_ARG, "lengths must not be NULL");
    if (!aligned(p->lengths, 8)) return fail(NRM_ERR_INVALID_ARG, "lengths must be aligned to 8 bytes");
    *cap = p->width * c->page_size;
    if (w && w->capacity < *cap) *cap = w->capacity < 0 ? 0 : w->capacity;
    return NRM_OK;
}

nrm_status check_weights(const char* name, const nrm_kv_weights* w, int64_t sequences, int64_t heads) {
    if (w->capacity < 1) return fail(NRM_ERR_INVALID_ARG, "%s: capacity must be >= 1", name);
    if (w->capacity > kMaxPositions) return fail(NRM_ERR_UNSUPPORTED, "%s: capacity must be <= 2^40", name);
    if (sequences > 0 && !w->data) return fail(NRM_ERR_INVALID_ARG, "%s: data must not be NULL", name);
    if (!aligned(w->data, 4)) return fail(NRM_ERR_INVALID_ARG, "%s must be aligned to 4 bytes", name);
    int64_t es = 0, eh = 0;
    if (!spans(sequences, w->sequence_stride, &es) || !spans(heads, w->head_stride, &eh))
        return fail(NRM_ERR_INVALID_ARG, "%s: strides must be >= 0 and span less than 2^60", name);
    // rows must not overlap: one of the two dimensions steps over all of the other
    const int64_t n = w->capacity;
    const bool heads_inside = (heads == 1 || w->head_stride >= n) && (sequences <= 1 || w->sequence_stride >= eh + n);
    const bool sequences_inside = (sequences <= 1 || w->sequence_stride >= n) && (heads == 1 || w->head_stride >= es + n);
    if (!heads_inside && !sequences_inside) return fail(NRM_ERR_INVALID_ARG, "%s: rows overlap", name);
    return NRM_OK;
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Where the parts of the workspace begin, in bytes; [4] is its size.
struct AttnWorkspace {
    int64_t at[5];
    int64_t logit_stride;
};
bool attn_workspace(int64_t sequences, int64_t hq, int64_t hk, int64_t d, int64_t positions, int sms, AttnWorkspace* w) {
    const int64_t n = sequences < kAttnSequences ? sequences : kAttnSequences;
    const int64_t heads = hq / hk < kAttnHeads ? hq / hk : kAttnHeads;
    const int64_t logits = n * attn_most_logits(hq, hk);
    w->logit_stride = positions;
    if (logits > 0 && positions > kMaxWorkspace / (logits * 4)) return false;
    w->at[0] = 0;
    w->at[1] = round16((n + 1) * 4);
    w->at[2] = w->at[1] + round16(n * hq * 4);
    // shares times pairs: no more than workers, or pairs where they are more
    const int64_t parts = std::max<int64_t>(int64_t(sms) * kAttnWarps, attn_most_pairs(hq, hk));
    w->at[3] = w->at[2] + round16(parts * 2 * attn_part_floats(int(heads), int(d)) * 4);
    w->at[4] = w->at[3] + logits * positions * 4;
    return true;
}

}  // namespace
}  // namespace nrm

using namespace nrm;

extern "C" {

size_t nrm_kv_attention_workspace_bytes(int64_t sequences, int64_t heads, const nrm_kv_cache* cache,
                                        int64_t positions) {
    const DevInfo* dev = dev_info();
    AttnWorkspace w;
    if (!dev || !cache || sequences < 0 || sequences > kMaxSequences || heads < 1 || heads > kMaxHeads ||
        cache->heads < 1 || heads % cache->heads || cache->d < 1 || cache->d > kHeadMaxD || positions < 0 ||
        positions > kMaxPositions || !attn_workspace(sequences, heads, cache->heads, cache->d, positions, dev->sms, &w))
        return 0;
    return size_t(w.at[4]);
}

nrm_status nrm_kv_cache_attention(const nrm_heads* q, const nrm_kv_cache* cache, const nrm_kv_pages* pages,
                                  const nrm_heads* out, float scale, int64_t window, float* lse,
                                  const nrm_kv_weights* weights, nrm_dtype dt, void* workspace,
                                  size_t workspace_bytes, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        AttnArgs a{};
        NRM_TRY(set_cache(cache, true, true, false, &a.cache));
        NRM_TRY(check_sequences(pages, cache, weights, &a.cap));
        const int64_t sequences = pages->sequences;
        NRM_TRY(check_sizes(sequences, cache->d, dt));
        NRM_TRY(check_view("q", q, nullptr, sequences, cache->d, dt, false));
        NRM_TRY(check_view("out", out, q, sequences, cache->d, dt, true));
        NRM_TRY(check_place("out", out, q, false, sequences));
        if (q->heads % cache->heads)
            return fail(NRM_ERR_INVALID_ARG, "q has %lld heads, no multiple of the cache's %lld", (long long)q->heads,
                        (long long)cache->heads);
        if (weights) NRM_TRY(check_weights("weights", weights, sequences, cache->heads));
        a.scale_log2 = float(double(scale) * 1.4426950408889634074);
        if (!std::isfinite(a.scale_log2)) return fail(NRM_ERR_INVALID_ARG, "scale*log2(e) must be finite");
        if (window < 0) return fail(NRM_ERR_INVALID_ARG, "window must be >= 0");
        NRM_TRY(check_stats({lse}, 4));
        if (sequences == 0) return NRM_OK;
        // positions are divided by the page's size too, and a sequence may have more of them than the cache has slots
        a.cache.page = make_row_div(cache->page_size, std::max(a.cache.slots, a.cap));
        // the tiles of a launch are counted in 32 bits
        const int64_t tiles = (a.cap / kAttnTile + 1 + kAttnStart) * attn_most_pairs(q->heads, cache->heads);
        if (a.cap / kAttnTile >= kAttnTiles || tiles >= kAttnTiles)
            return fail(NRM_ERR_UNSUPPORTED, "positions*heads of a sequence must be < 2^36");
        const DevInfo* dev = dev_info();
        if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
        AttnWorkspace w;
        if (!attn_workspace(sequences, q->heads, cache->heads, cache->d, weights ? a.cap : 0, dev->sms, &w))
            return fail(NRM_ERR_UNSUPPORTED, "the weights need more than 2^48 bytes of workspace");
        if (!workspace || !aligned(workspace, 16))
            return fail(NRM_ERR_WORKSPACE, "workspace must be non-NULL and 16-byte aligned");
        if (workspace_bytes < size_t(w.at[4]))
            return fail(NRM_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu needed", workspace_bytes,
                        size_t(w.at[4]));
        char* ws = static_cast<char*>(workspace);
        a.prefix = reinterpret_cast<int*>(ws + w.at[0]);
        a.lse2 = reinterpret_cast<float*>(ws + w.at[1]);
        a.part = reinterpret_cast<float*>(ws + w.at[2]);
        a.logits = weights ? reinterpret_cast<float*>(ws + w.at[3]) : nullptr;
        a.logit_stride = w.logit_stride;
        a.q = view(q);
        a.out = view(out);
        a.table_stride = sequences > 1 ? pages->stride : 0;
        a.hq = int(q->heads);
        a.hk = int(cache->heads);
        a.shared = a.hq / a.hk;
        a.d = int(cache->d);
        a.window = window;
        if (weights) {
            a.weight_ts = weights->sequence_stride;
            a.weight_hs = weights->head_stride;
        }
        // rows of codes as whole vectors, groups of whole matrix steps
        int vec = 0;
        const int64_t bytes = cache->kind == NRM_CACHE_INT4 ? cache->d / 2 : cache->d;
        if (cache->d % 16 == 0 && cache->group % 16 == 0)
            for (int64_t b = 16; b >= 8 && !vec; b /= 2)
                if (bytes % b == 0 && aligned(cache->k_codes, size_t(b)) && aligned(cache->v_codes, size_t(b)) &&
                    (cache->pages == 1 || cache->page_stride % b == 0) &&
                    (cache->page_size == 1 || cache->slot_stride % b == 0) &&
                    (cache->heads == 1 || cache->head_stride % b == 0))
                    vec = int(b);
        const int64_t es = int64_t(dsize(dt));
        // (strides below 2^40 times counts whose extents were checked: no overflow)
        const int64_t extent = (cache->pages - 1) * cache->page_stride + (cache->page_size - 1) * cache->slot_stride +
                               (cache->heads - 1) * cache->head_stride;
        a.near = vec == 16 && extent < (int64_t(1) << 36);
        auto whole = [&](const nrm_heads* v) {
            return aligned(v->data, 16) && (sequences == 1 || v->token_stride * es % 16 == 0) &&
                   (v->heads == 1 || v->head_stride * es % 16 == 0);
        };
        a.q_vec = whole(q);
        a.out_vec = whole(out);
        a.scale_vec = cache->d / cache->group % 4 == 0 && aligned(cache->k_scales, 16) && aligned(cache->v_scales, 16) &&
                      (cache->pages == 1 || cache->scale_page_stride % 4 == 0) &&
                      (cache->page_size == 1 || cache->scale_slot_stride % 4 == 0) &&
                      (cache->heads == 1 || cache->scale_head_stride % 4 == 0);
        const int64_t most = std::min<int64_t>(kAttnSequences, (kAttnTiles - 1) / tiles);
        for (int64_t s0 = 0; s0 < sequences; s0 += most) {
            AttnArgs b = a;
            b.sequences = int(std::min(sequences - s0, most));
            b.table = pages->table + s0 * a.table_stride;
            b.lengths = pages->lengths + s0;
            b.q.p = static_cast<char*>(a.q.p) + s0 * a.q.ts * es;
            b.out.p = static_cast<char*>(a.out.p) + s0 * a.out.ts * es;
            b.lse = lse ? lse + s0 * a.hq : nullptr;
            b.weights = weights ? weights->data + s0 * a.weight_ts : nullptr;
            NRM_TRY(by_dtype(dt, [&](auto tag) {
                return kv_attention<decltype(tag)>(b, vec, reinterpret_cast<cudaStream_t>(stream));
            }));
        }
        return NRM_OK;
    });
}

nrm_status nrm_kv_cache_evict(const nrm_kv_cache* cache, const nrm_kv_pages* pages, const nrm_kv_weights* weights,
                              const int64_t* new_table, int64_t new_width, int64_t new_stride, int64_t* new_lengths,
                              const nrm_kv_weights* new_weights, int64_t* kept, int64_t keep, int64_t first,
                              int64_t recent, nrm_stream_t stream) {
    return entry([&]() -> nrm_status {
        EvictArgs a{};
        NRM_TRY(set_cache(cache, true, true, true, &a.cache));
        if (!weights) return fail(NRM_ERR_INVALID_ARG, "weights must not be NULL");
        NRM_TRY(check_sequences(pages, cache, weights, &a.cap));
        const int64_t sequences = pages->sequences;
        NRM_TRY(check_weights("weights", weights, sequences, cache->heads));
        if (keep < 1 || first < 0 || recent < 0 || first > keep || recent > keep - first)
            return fail(NRM_ERR_INVALID_ARG, "keep must be >= 1, first and recent >= 0, and first + recent <= keep");
        if (a.cap > (int64_t(1) << 30)) return fail(NRM_ERR_UNSUPPORTED, "a sequence must have at most 2^30 positions");
        if (keep >= (int64_t(1) << 31)) return fail(NRM_ERR_UNSUPPORTED, "keep must be < 2^31");
        NRM_TRY(check_pages("new_table", new_table, new_width, new_stride, sequences, cache->page_size));
        if (sequences > 0 && new_width * cache->page_size < keep)
            return fail(NRM_ERR_INVALID_ARG, "new_table holds %lld positions, fewer than keep",
                        (long long)(new_width * cache->page_size));
        if (sequences > 0 && (!new_lengths || !kept))
            return fail(NRM_ERR_INVALID_ARG, "new_lengths and kept must not be NULL");
        if (!aligned(new_lengths, 8) || !aligned(kept, 8))
            return fail(NRM_ERR_INVALID_ARG, "new_lengths and kept must be aligned to 8 bytes");
        if (sequences > 0 && (new_lengths == pages->lengths || new_table == pages->table))
            return fail(NRM_ERR_INVALID_ARG, "the new lengths and table are the old ones' memory");
        if (new_weights) {
            NRM_TRY(check_weights("new_weights", new_weights, sequences, cache->heads));
            if (new_weights->capacity < keep)
                return fail(NRM_ERR_INVALID_ARG, "new_weights: capacity is less than keep");
            if (sequences > 0 && new_weights->data == weights->data)
                return fail(NRM_ERR_INVALID_ARG, "weights and new_weights are the same memory");
            a.new_weights = new_weights->data;
            a.new_ts = new_weights->sequence_stride;
            a.new_hs = new_weights->head_stride;
        }
        if (sequences == 0) return NRM_OK;
        if (sequences > kMaxRows / cache->heads || sequences * cache->heads > kMaxRows / keep)
            return fail(NRM_ERR_UNSUPPORTED, "sequences*heads*keep must be < 2^40");
        a.table = pages->table;
        a.table_stride = sequences > 1 ? pages->stride : 0;
        a.lengths = pages->lengths;
        a.new_table = new_table;
        a.new_stride = sequences > 1 ? new_stride : 0;
        a.new_lengths = new_lengths;
        a.weights = weights->data;
        a.weight_ts = weights->sequence_stride;
        a.weight_hs = weights->head_stride;
        a.kept = kept;
        a.sequences = sequences;
        a.heads = int(cache->heads);
        a.d = int(cache->d);
        a.keep = keep;
        a.first = first;
        a.recent = recent;
        return kv_evict(a, reinterpret_cast<cudaStream_t>(stream));
    });
}

}  // extern "C"
