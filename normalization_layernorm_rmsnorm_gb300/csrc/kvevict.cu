// kvevict.cu -- eviction from the cache by accumulated attention weight: which
// positions of each head stay, then the copy of their rows into other pages.
//
// Choosing: a CTA for each head of each sequence.  Weights are compared as
// unsigned integers that order as the numbers do; the border is found by radix,
// eight bits at a time from the top, with counts in shared memory (whole
// numbers: their order does not matter), and a last pass over the positions
// writes those that stay in order.
#include "heads.cuh"
#include "kvattn.h"

namespace nrm {
namespace {

constexpr int kEvictThreads = 1024;
constexpr int kCopyThreads = 256;

// Orders as the numbers do; a NaN is above all, -0 is 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}

// Sum of `mine` over the threads before this one; *all: over all of them.
__device__ __forceinline__ uint32_t cta_before(uint32_t mine, uint32_t* sums, uint32_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    uint32_t s = sums[lane], t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += up;
    }
    *all = __shfl_sync(0xffffffffu, t, 31);
    return __shfl_sync(0xffffffffu, t - s, warp) + run - mine;
}

__global__ void __launch_bounds__(kEvictThreads) evict_choose_kernel(const EvictArgs a) {
    __shared__ uint32_t counts[256], sums[32], found[2];
    pdl_next();
    const int64_t s = blockIdx.x / a.heads;
    const int head = int(blockIdx.x - s * a.heads);
    int64_t n = ld_after(a.lengths + s);
    if (n < 0 || n > a.cap) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrCacheSlot);
        n = n < 0 ? 0 : a.cap;
    }
    if (head == 0 && threadIdx.x == 0) a.new_lengths[s] = n < a.keep ? n : a.keep;
    const float* weights = a.weights + s * a.weight_ts + head * a.weight_hs;
    int64_t* kept = a.kept + (s * a.heads + head) * a.keep;
    float* out = a.new_weights ? a.new_weights + s * a.new_ts + head * a.new_hs : nullptr;
    if (n <= a.keep) {
        for (int64_t i = threadIdx.x; i < a.keep; i += kEvictThreads) {
            kept[i] = i < n ? i : -1;
            if (out && i < n) out[i] = ld_after(weights + i);
        }
        return;
    }
    // the border among the positions between: of those with its key, the first `ties` stay
    const int64_t lo = a.first, hi = n - a.recent;
    uint32_t want = uint32_t(a.keep - a.first - a.recent), border = 0;
    if (want == 0) border = 0xffffffffu;
    else
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = threadIdx.x; i < 256; i += kEvictThreads) counts[i] = 0;
            __syncthreads();
            for (int64_t i = lo + threadIdx.x; i < hi; i += kEvictThreads) {
                const uint32_t k = weight_key(ld_after(weights + i));
                if (shift == 24 || k >> (shift + 8) == border >> (shift + 8)) atomicAdd(&counts[k >> shift & 255u], 1u);
            }
            __syncthreads();
            if (threadIdx.x < 32) {
                // lane l looks after 8 digits, from the largest down
                uint32_t c[8], mine = 0;
                for (int j = 0; j < 8; ++j) {
                    c[j] = counts[255 - (int(threadIdx.x) * 8 + j)];
                    mine += c[j];
                }
                uint32_t run = mine;
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
                    if (threadIdx.x >= o) run += up;
                }
                uint32_t before = run - mine;
                for (int j = 0; j < 8; ++j) {
                    if (before < want && want <= before + c[j]) {
                        found[0] = 255u - (threadIdx.x * 8 + j);
                        found[1] = want - before;
                    }
                    before += c[j];
                }
            }
            __syncthreads();
            border |= found[0] << shift;
            want = found[1];
        }
    // in order: each round takes the next positions, one to a thread
    uint32_t taken = 0, ties = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kEvictThreads) {
        const int64_t i = i0 + threadIdx.x;
        float w = 0.f;
        bool above = false, tie = false;
        if (i < n) {
            w = ld_after(weights + i);
            const uint32_t k = weight_key(w);
            const bool between = i >= lo && i < hi;
            above = !between || (want > 0 && k > border);
            tie = between && want > 0 && k == border;
        }
        uint32_t all_ties, all;
        const uint32_t tie_at = ties + cta_before(tie, sums, &all_ties);
        const bool stays = above || (tie && tie_at < want);
        const uint32_t at = taken + cta_before(stays, sums, &all);
        if (stays) {
            kept[at] = i;
            if (out) out[at] = w;
        }
        ties += all_ties;
        taken += all;
    }
}

// A warp for each row that stays, keys and values.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictArgs a, RowDiv per_sequence, RowDiv by_keep) {
    pdl_next();
    const int lane = threadIdx.x & 31;
    const int64_t rows = a.sequences * a.heads * a.keep, warps = int64_t(gridDim.x) * (kCopyThreads / 32);
    const int bytes = a.cache.kind == NRM_CACHE_INT4 ? a.d / 2 : a.d, scales = a.d / a.cache.group;
    const int64_t pages = a.cache.slots / a.cache.page.d;
    for (int64_t r = int64_t(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
        const int64_t j = ld_after(a.kept + r);
        if (j < 0) continue;
        const int64_t s = row_div(r, per_sequence), in_s = r - s * per_sequence.d;
        const int64_t head = row_div(in_s, by_keep), i = in_s - head * a.keep;
        const int64_t from_entry = row_div(j, a.cache.page), to_entry = row_div(i, a.cache.page);
        const int64_t from_page = ld_after(a.table + s * a.table_stride + from_entry);
        const int64_t to_page = ld_after(a.new_table + s * a.new_stride + to_entry);
        if (from_page < 0 || from_page >= pages || to_page < 0 || to_page >= pages) {
            if (lane == 0) atomicOr(a.err, kErrCacheSlot);
            continue;
        }
        const CacheRow from = cache_row(a.cache, from_page * a.cache.page.d + (j - from_entry * a.cache.page.d), int(head));
        const CacheRow to = cache_row(a.cache, to_page * a.cache.page.d + (i - to_entry * a.cache.page.d), int(head));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            for (int b = lane; b < bytes; b += 32) a.cache.codes[t][to.code + b] = ld_after(a.cache.codes[t] + from.code + b);
            for (int g = lane; g < scales; g += 32)
                a.cache.scales[t][to.scale + g] = ld_after(a.cache.scales[t] + from.scale + g);
        }
    }
}

}  // namespace

nrm_status kv_evict(const EvictArgs& args, cudaStream_t s) {
    EvictArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    const int64_t ctas = a.sequences * a.heads;
    if (ctas >= (int64_t(1) << 31)) return fail(NRM_ERR_UNSUPPORTED, "sequences*heads must be < 2^31");
    void* p[] = {&a};
    nrm_status st = launch_pdl(reinterpret_cast<const void*>(&evict_choose_kernel), dim3(unsigned(ctas)),
                               dim3(kEvictThreads), p, s);
    if (st != NRM_OK) return st;
    const int64_t rows = ctas * a.keep;
    RowDiv per_sequence = make_row_div(a.heads * a.keep, rows), by_keep = make_row_div(a.keep, rows);
    void* q[] = {&a, &per_sequence, &by_keep};
    const int64_t want = (rows + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    return launch_pdl(reinterpret_cast<const void*>(&evict_copy_kernel),
                      dim3(unsigned(std::min<int64_t>(want, int64_t(dev->sms) * 16))), dim3(kCopyThreads), q, s);
}

}  // namespace nrm
