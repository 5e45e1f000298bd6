// kvevict.cu -- eviction from the cache by accumulated attention weight: which
// positions of each head stay, then the copy of their rows into other pages.
//
// Choosing: a cluster of CTAs for each head of each sequence, a part of its
// positions each, whose weights are read once and kept in shared memory as
// unsigned integers that order as the numbers do.  The border is found by radix
// in three rounds (11, 11 and 10 bits from the top: the first has the exponent
// and two bits more, so that weights of like size do not all meet at one
// counter); the CTAs add one another's counts (whole numbers, their order does
// not matter) through distributed shared memory.  The positions that stay are
// then written in order, each CTA behind those before it.
// Bound by latency: three exchanges of the cluster, and a CTA's rounds over its part.
//
// Copying: bound by bytes.  The heads of a slot of the shortened sequence follow
// one another, so that what is written lies together, and what is read nearly so.
#include "heads.cuh"
#include "kvattn.h"

namespace nrm {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictCluster = 8;         // CTAs of a cluster, at most
constexpr int kEvictPart = 2048;         // positions that are worth a CTA more
constexpr int kEvictHeld = 45 * 1024;    // weights that a CTA's shared memory holds
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 4;            // rows of a lane under way

// Orders as the numbers do; a NaN is above all, -0 is 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t warp_before(uint32_t mine, uint32_t* all) {
    const int lane = threadIdx.x & 31;
    uint32_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
    }
    *all = __shfl_sync(0xffffffffu, run, 31);
    return run - mine;
}
// Sum of `mine` over the threads before this one; *all: over all of them.
__device__ __forceinline__ uint32_t cta_before(uint32_t mine, uint32_t* sums, uint32_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t in_warp;
    const uint32_t before = warp_before(mine, &in_warp);
    __syncthreads();
    if (lane == 0) sums[warp] = in_warp;
    __syncthreads();
    const uint32_t other = lane < kEvictWarps ? sums[lane] : 0;
    const uint32_t warps = warp_before(other, all);
    return __shfl_sync(0xffffffffu, warps, warp) + before;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__global__ void __launch_bounds__(kEvictThreads) evict_choose_kernel(const EvictArgs a, int ctas, int held) {
    extern __shared__ uint32_t keys[];  // [held]
    __shared__ uint32_t counts[2][kEvictBins], sums[32], found[2], share[2];
    pdl_next();
    const int64_t which = blockIdx.x / ctas, s = which / a.heads;
    const int part = int(blockIdx.x % ctas), head = int(which - s * a.heads);
    int64_t n = ld_after(a.lengths + s);
    if (n < 0 || n > a.cap) {
        if (threadIdx.x == 0) atomicOr(a.err, kErrCacheSlot);
        n = n < 0 ? 0 : a.cap;
    }
    if (head == 0 && part == 0 && threadIdx.x == 0) a.new_lengths[s] = n < a.keep ? n : a.keep;
    const float* weights = a.weights + s * a.weight_ts + head * a.weight_hs;
    int64_t* kept = a.kept + which * a.keep;
    float* out = a.new_weights ? a.new_weights + s * a.new_ts + head * a.new_hs : nullptr;
    if (n <= a.keep) {
        for (int64_t i = int64_t(part) * kEvictThreads + threadIdx.x; i < a.keep; i += int64_t(ctas) * kEvictThreads) {
            kept[i] = i < n ? i : -1;
            if (out && i < n) out[i] = ld_after(weights + i);
        }
        return;
    }
    auto cluster_sync = [&]() {
        if (ctas > 1) cluster_sync_all();
        else __syncthreads();
    };
    // this CTA's positions, rounded to the warps' strides
    const int64_t each = ((n + ctas - 1) / ctas + kEvictThreads - 1) / kEvictThreads * kEvictThreads;
    const int64_t first = min(n, part * each), last = min(n, first + each), lo = a.first, hi = n - a.recent;
    const bool holds = last - first <= held;
    if (holds) {
        const int count = int(last - first);
        for (int i = threadIdx.x; i < count; i += 4 * kEvictThreads) {
            float w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kEvictThreads < count) w[k] = ld_after(weights + first + i + k * kEvictThreads);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k * kEvictThreads < count) keys[i + k * kEvictThreads] = weight_key(w[k]);
        }
    }
    auto key = [&](int64_t i) { return holds ? keys[i - first] : weight_key(ld_after(weights + i)); };
    // the border among the positions between: of those with its key, the first `want` stay
    uint32_t want = uint32_t(a.keep - a.first - a.recent), border = 0;
    const bool any = want > 0;
#pragma unroll
    for (int round = 0; round < 3; ++round) {
        if (!any) break;
        constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
        const int shift = kShift[round], bits = kBits[round];
        uint32_t* mine = counts[round & 1];
        for (int i = threadIdx.x; i < kEvictBins; i += kEvictThreads) mine[i] = 0;
        __syncthreads();
        for (int64_t i = max(first, lo) + threadIdx.x; i < min(last, hi); i += kEvictThreads) {
            const uint32_t k = key(i);
            if (round == 0 || k >> (shift + bits) == border >> (shift + bits))
                atomicAdd(&mine[k >> shift & ((1u << bits) - 1)], 1u);
        }
        cluster_sync();
        // thread t has the digits 4 t to 4 t + 3 from the largest down
        uint32_t c[4], sum = 0, all;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int digit = kEvictBins - 1 - (int(threadIdx.x) * 4 + j);
            c[j] = 0;
            if (ctas == 1) c[j] = mine[digit];
            else
                for (int r = 0; r < ctas; ++r) c[j] += ld_dsmem_u32(dsmem_addr(&mine[digit], uint32_t(r)));
            sum += c[j];
        }
        static_assert(kEvictBins == 4 * kEvictThreads, "four digits to a thread");
        uint32_t before = cta_before(sum, sums, &all);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (before < want && want <= before + c[j]) {
                found[0] = kEvictBins - 1 - (threadIdx.x * 4 + j);
                found[1] = want - before;
            }
            before += c[j];
        }
        __syncthreads();
        border |= found[0] << shift;
        want = found[1];
        __syncthreads();
    }
    // how many of this CTA's positions stay for sure, and how many lie on the border
    auto stays = [&](int64_t i, bool& tie) {
        const bool between = i >= lo && i < hi;
        const uint32_t k = between && any ? key(i) : 0;
        tie = between && any && k == border;
        return !between || (any && k > border);
    };
    uint32_t above = 0, ties = 0;
    for (int64_t i = first + threadIdx.x; i < last; i += kEvictThreads) {
        bool tie;
        above += stays(i, tie);
        ties += tie;
    }
    uint32_t all_above, all_ties;
    cta_before(above, sums, &all_above);
    cta_before(ties, sums, &all_ties);
    if (threadIdx.x == 0) {
        share[0] = all_above;
        share[1] = all_ties;
    }
    cluster_sync();
    uint32_t taken = 0, tied = 0;
    for (int r = 0; r < part; ++r) {
        taken += ld_dsmem_u32(dsmem_addr(&share[0], uint32_t(r)));
        tied += ld_dsmem_u32(dsmem_addr(&share[1], uint32_t(r)));
    }
    taken += min(tied, want);  // of the ties before this CTA's, those that stay
    // in order: each round takes the next positions, one to a thread
    for (int64_t i0 = first; i0 < last; i0 += kEvictThreads) {
        const int64_t i = i0 + threadIdx.x;
        bool tie = false, sure = false;
        if (i < last) sure = stays(i, tie);
        // both counts in one sum: a round has at most 512 of each
        uint32_t all;
        const uint32_t before = cta_before(uint32_t(sure) | uint32_t(tie) << 16, sums, &all);
        const uint32_t tie_at = tied + (before >> 16);
        if (sure || (tie && tie_at < want)) {
            // the ties before it that stay, and those that are sure
            const uint32_t at = taken + (before & 0xffffu) + (min(tie_at, want) - min(tied, want));
            kept[at] = i;
            if (out) out[at] = ld_after(weights + i);
        }
        taken += (all & 0xffffu) + (min(tied + (all >> 16), want) - min(tied, want));
        tied += all >> 16;
    }
    if (ctas > 1) cluster_sync_all();  // the others may still read this CTA's counts
}

// Which row a lane copies: row r of the shortened sequences, head innermost.
struct CopyDiv {
    RowDiv heads, keep;
};

// VEC bytes at once: neighbouring lanes copy neighbouring vectors of a row of keys and of values.
template <int VEC>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictArgs a, CopyDiv by, int row_bytes) {
    using R = std::conditional_t<VEC == 16, uint4, std::conditional_t<VEC == 8, uint2, uint8_t>>;
    pdl_next();
    const int lane = threadIdx.x & 31;
    const int vecs = row_bytes / VEC, scales = a.d / a.cache.group;
    // lanes of a row: as many as it has vectors (a power of two, at most 32)
    int lanes = 1;
    while (lanes < vecs && lanes < 32) lanes *= 2;
    const int at_once = 32 / lanes, mine = lane & (lanes - 1);
    const int64_t rows = a.sequences * a.heads * a.keep, pages = a.cache.slots / a.cache.page.d;
    const int64_t step = int64_t(gridDim.x) * (kCopyThreads / 32) * at_once;
    int64_t r0 = (int64_t(blockIdx.x) * (kCopyThreads / 32) + (threadIdx.x >> 5)) * at_once + lane / lanes;
    for (; r0 < rows; r0 += step * kCopyAhead) {
        int64_t from_code[kCopyAhead], to_code[kCopyAhead], from_scale[kCopyAhead], to_scale[kCopyAhead];
        int64_t j[kCopyAhead], s[kCopyAhead], i[kCopyAhead], from_page[kCopyAhead], to_page[kCopyAhead];
        int head[kCopyAhead];
#pragma unroll
        for (int k = 0; k < kCopyAhead; ++k) {
            const int64_t r = r0 + k * step;
            j[k] = -1;
            if (r >= rows) continue;
            const int64_t in_seq = row_div(r, by.heads);
            head[k] = int(r - in_seq * a.heads);
            s[k] = row_div(in_seq, by.keep);
            i[k] = in_seq - s[k] * a.keep;
            j[k] = ld_after(a.kept + (s[k] * a.heads + head[k]) * a.keep + i[k]);
        }
#pragma unroll
        for (int k = 0; k < kCopyAhead; ++k) {
            if (j[k] < 0) continue;
            const int64_t from_entry = row_div(j[k], a.cache.page), to_entry = row_div(i[k], a.cache.page);
            from_page[k] = ld_after(a.table + s[k] * a.table_stride + from_entry);
            to_page[k] = ld_after(a.new_table + s[k] * a.new_stride + to_entry);
            j[k] -= from_entry * a.cache.page.d;
            i[k] -= to_entry * a.cache.page.d;
        }
#pragma unroll
        for (int k = 0; k < kCopyAhead; ++k) {
            if (j[k] < 0) continue;
            if (from_page[k] < 0 || from_page[k] >= pages || to_page[k] < 0 || to_page[k] >= pages) {
                atomicOr(a.err, kErrCacheSlot);
                j[k] = -1;
                continue;
            }
            const CacheDev& c = a.cache;
            from_code[k] = from_page[k] * c.page_stride + j[k] * c.slot_stride + head[k] * c.head_stride;
            to_code[k] = to_page[k] * c.page_stride + i[k] * c.slot_stride + head[k] * c.head_stride;
            from_scale[k] = from_page[k] * c.scale_page_stride + j[k] * c.scale_slot_stride + head[k] * c.scale_head_stride;
            to_scale[k] = to_page[k] * c.scale_page_stride + i[k] * c.scale_slot_stride + head[k] * c.scale_head_stride;
        }
        for (int v = mine; v < vecs; v += lanes) {
            R x[kCopyAhead][2];
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) {
                if (j[k] < 0) continue;
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    x[k][t] = ld_after(reinterpret_cast<const R*>(a.cache.codes[t] + from_code[k]) + v);
            }
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) {
                if (j[k] < 0) continue;
#pragma unroll
                for (int t = 0; t < 2; ++t) reinterpret_cast<R*>(a.cache.codes[t] + to_code[k])[v] = x[k][t];
            }
        }
        for (int g = mine; g < 2 * scales; g += lanes) {
            const int t = g >= scales, at = g - t * scales;
            float x[kCopyAhead];
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (j[k] >= 0) x[k] = ld_after(a.cache.scales[t] + from_scale[k] + at);
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k)
                if (j[k] >= 0) a.cache.scales[t][to_scale[k] + at] = x[k];
        }
    }
}

nrm_status choose(EvictArgs& a, const DevInfo* dev, cudaStream_t s) {
    const int64_t pairs = a.sequences * a.heads;
    // CTAs to a head: as its positions are worth, while the GPU has room
    int ctas = 1;
    while (ctas < kEvictCluster && a.cap > int64_t(ctas) * kEvictPart && pairs * ctas * 2 <= 2 * int64_t(dev->sms)) ctas *= 2;
    if (pairs * ctas >= (int64_t(1) << 31)) return fail(NRM_ERR_UNSUPPORTED, "sequences*heads must be < 2^31");
    const int64_t most = ((a.cap + ctas - 1) / ctas + kEvictThreads - 1) / kEvictThreads * kEvictThreads;
    int held = int(most <= kEvictHeld ? most : 0);
    const void* fn = reinterpret_cast<const void*>(&evict_choose_kernel);
    const size_t smem = size_t(held) * 4;
    nrm_status st = prepare_kernel(fn, smem, false);
    if (st != NRM_OK) return st;
    void* p[] = {&a, &ctas, &held};
    if (ctas == 1) return launch_pdl(fn, dim3(unsigned(pairs)), dim3(kEvictThreads), p, s, smem);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(pairs * ctas));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelExC(&cfg, fn, p), "eviction launch");
}

}  // namespace

nrm_status kv_evict(const EvictArgs& args, cudaStream_t s) {
    EvictArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    nrm_status st = choose(a, dev, s);
    if (st != NRM_OK) return st;
    const int64_t rows = a.sequences * a.heads * a.keep;
    CopyDiv by{make_row_div(a.heads, rows), make_row_div(a.keep, rows)};
    int bytes = a.cache.kind == NRM_CACHE_INT4 ? a.d / 2 : a.d, vec = 1;
    for (int b : {16, 8})
        if (vec == 1 && bytes % b == 0 && reinterpret_cast<uintptr_t>(a.cache.codes[0]) % b == 0 &&
            reinterpret_cast<uintptr_t>(a.cache.codes[1]) % b == 0 && a.cache.page_stride % b == 0 &&
            a.cache.slot_stride % b == 0 && a.cache.head_stride % b == 0)
            vec = b;
    int lanes = 1;
    while (lanes < bytes / vec && lanes < 32) lanes *= 2;
    const int64_t at_once = int64_t(kCopyThreads / lanes) * kCopyAhead;
    const int64_t want = (rows + at_once - 1) / at_once;
    void* q[] = {&a, &by, &bytes};
    const void* fn = vec == 16  ? reinterpret_cast<const void*>(&evict_copy_kernel<16>)
                     : vec == 8 ? reinterpret_cast<const void*>(&evict_copy_kernel<8>)
                                : reinterpret_cast<const void*>(&evict_copy_kernel<1>);
    return launch_pdl(fn, dim3(unsigned(std::min<int64_t>(want, int64_t(dev->sms) * 64))), dim3(kCopyThreads), q, s);
}

}  // namespace nrm
