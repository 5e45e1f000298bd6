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
// Bound by latency: three exchanges of the cluster, and a CTA's rounds over its part
// (131072 positions to 65536, 8 heads: 22 us; 4096 to 1024: 7).
//
// Copying: bound by bytes (65536 rows of 8 heads of 128 bytes: 47 us, 0.87 of the
// copy rate).  The heads of a slot of the shortened sequence follow one another, so
// that what is written lies together, and what is read nearly so.
#include "heads.cuh"
#include "kvattn.h"

namespace nrm {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictTurn = 4 * kEvictThreads;  // positions that its threads take at once
constexpr int kEvictBins = 2048;
constexpr int kEvictCluster = 8;         // CTAs of a cluster, at most
constexpr int kEvictPart = 8192;         // positions that are worth a CTA more
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
// Sum of `mine` over the threads before this one.
__device__ __forceinline__ uint32_t cta_before(uint32_t mine, uint32_t* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t in_warp;
    const uint32_t before = warp_before(mine, &in_warp);
    if (lane == 0) sums[warp] = in_warp;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) + before;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__global__ void __launch_bounds__(kEvictThreads) evict_choose_kernel(const EvictArgs a, int ctas, int held) {
    extern __shared__ __align__(16) uint32_t keys[];  // [held]
    __shared__ __align__(16) uint32_t counts[2][kEvictBins];      // this CTA's
    __shared__ __align__(16) uint32_t slices[2][kEvictBins / 2];  // the cluster's, of this CTA's share of the digits
    __shared__ uint32_t sums[32], found[2], share[2];
    static_assert(kEvictWarps <= 32 && kEvictBins == 4 * kEvictThreads, "four digits to a thread");
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
    if (n <= a.keep) {
        for (int64_t i = int64_t(part) * kEvictThreads + threadIdx.x; i < a.keep; i += int64_t(ctas) * kEvictThreads)
            kept[i] = i < n ? i : -1;
        return;
    }
    auto cluster_sync = [&]() {
        if (ctas > 1) cluster_sync_all();
        else __syncthreads();
    };
    // this CTA's positions, whole turns of its threads, and of them those between, [from, to)
    const int each = int((n + ctas * kEvictTurn - 1) / (ctas * kEvictTurn)) * kEvictTurn;
    const int first = min(int(n), part * each), count = min(int(n) - first, each);
    const int from = min(count, max(0, int(a.first) - first)), to = min(count, max(0, int(n - a.recent) - first));
    const bool holds = count <= held;
    weights += first;
    uint32_t want = uint32_t(a.keep - a.first - a.recent), border = 0;
    const bool any = want > 0;
    // of four neighbouring positions, which lie between (a bit each)
    auto lie_between = [&](int i) -> uint32_t {
        if (i >= from && i + 4 <= to) return 15u;
        const int lo = min(4, max(0, from - i)), hi = min(4, max(0, to - i));
        return ((1u << hi) - 1) & ~((1u << lo) - 1);
    };
    const bool vectors = reinterpret_cast<uintptr_t>(weights) % 16 == 0;
    auto load = [&](int i, uint32_t (&k)[4]) {
        if (vectors && i + 4 <= count) {
            const uint4 v = ld_after(reinterpret_cast<const uint4*>(weights + i));
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = i + j < count ? __float_as_uint(ld_after(weights + i + j)) : 0;
        }
    };
    auto four = [&](int i, uint32_t (&k)[4]) {
        if (holds) {
            const uint4 v = *reinterpret_cast<const uint4*>(keys + i);  // (what lies behind the last is not used)
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
            load(i, k);
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = weight_key(__uint_as_float(k[j]));
        }
    };
    auto clear = [&](int round) {
        reinterpret_cast<uint4*>(counts[round & 1])[threadIdx.x] = make_uint4(0, 0, 0, 0);
        reinterpret_cast<uint2*>(slices[round & 1])[threadIdx.x] = make_uint2(0, 0);
        __syncthreads();
    };
    // The border among the positions between: of those with its key, the first `want` stay.
    constexpr int kShift[3] = {21, 10, 0}, kBits[3] = {11, 11, 10};
    clear(0);
    if (holds) {  // the first digits are counted as the weights arrive
        constexpr int AHEAD = 8;
        for (int i0 = 4 * int(threadIdx.x); i0 < count; i0 += AHEAD * kEvictTurn) {
            uint32_t k[AHEAD][4];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
                if (i0 + u * kEvictTurn < count) load(i0 + u * kEvictTurn, k[u]);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = i0 + u * kEvictTurn;
                if (i >= count) break;
#pragma unroll
                for (int j = 0; j < 4; ++j) k[u][j] = weight_key(__uint_as_float(k[u][j]));
                *reinterpret_cast<uint4*>(keys + i) = make_uint4(k[u][0], k[u][1], k[u][2], k[u][3]);
                const uint32_t between = lie_between(i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (between >> j & 1) atomicAdd(&counts[0][k[u][j] >> kShift[0]], 1u);
            }
        }
    }
#pragma unroll
    for (int round = 0; round < 3; ++round) {
        if (!any) break;
        const int shift = kShift[round], bits = kBits[round];
        uint32_t *mine = counts[round & 1], *slice = slices[round & 1];
        if (round > 0) clear(round);
        if (round > 0 || !holds)
            for (int i = 4 * int(threadIdx.x); i < to; i += kEvictTurn) {
                uint32_t k[4];
                four(i, k);
                const uint32_t between = lie_between(i);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((between >> j & 1) && (round == 0 || k[j] >> (shift + bits) == border >> (shift + bits)))
                        atomicAdd(&mine[k[j] >> shift & ((1u << bits) - 1)], 1u);
            }
        cluster_sync();
        // thread t has the digits 4 t to 4 t + 3 from the largest down
        const int at = kEvictBins - 4 - int(threadIdx.x) * 4;
        float4 v;
        if (ctas == 1) {
            v = *reinterpret_cast<const float4*>(mine + at);
        } else {
            // each CTA adds a share of the digits, 16 bytes of one CTA's to a thread; then all read the sums
            const int of = kEvictBins / ctas, part4 = of / 4, r = int(threadIdx.x) / part4, i = (int(threadIdx.x) - r * part4) * 4;
            const float4 theirs = ld_dsmem_f4(dsmem_addr(mine + part * of + i, uint32_t(r)));
            atomicAdd(slice + i, __float_as_uint(theirs.x));
            atomicAdd(slice + i + 1, __float_as_uint(theirs.y));
            atomicAdd(slice + i + 2, __float_as_uint(theirs.z));
            atomicAdd(slice + i + 3, __float_as_uint(theirs.w));
            cluster_sync();
            v = ld_dsmem_f4(dsmem_addr(slice + at % of, uint32_t(at / of)));
        }
        const uint32_t c[4] = {__float_as_uint(v.w), __float_as_uint(v.z), __float_as_uint(v.y), __float_as_uint(v.x)};
        uint32_t before = cta_before(c[0] + c[1] + c[2] + c[3], sums);
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
    }
    // of four positions, which stay for sure and which lie on the border: a bit each
    auto stay = [&](int i, uint32_t& sure, uint32_t& tie) {
        sure = tie = 0;
        if (i >= count) return;
        uint32_t k[4];
        four(i, k);
        const uint32_t between = lie_between(i), there = i + 4 <= count ? 15u : (1u << (count - i)) - 1;
        if (any) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sure |= uint32_t(k[j] > border) << j;
                tie |= uint32_t(k[j] == border) << j;
            }
        }
        sure = (sure & between) | (there & ~between);
        tie &= between;
    };
    // a warp takes a stretch of positions: how many of it stay, then, behind those of the warps before it, which
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int stretch = (count + kEvictTurn - 1) / kEvictTurn * 128, begin = warp * stretch, end = min(count, begin + stretch);
    uint32_t above = 0, ties = 0, sure, tie;
    for (int i = begin + 4 * lane; i < end; i += 128) {
        stay(i, sure, tie);
        above += __popc(sure);
        ties += __popc(tie);
    }
    above = __reduce_add_sync(0xffffffffu, above);
    ties = __reduce_add_sync(0xffffffffu, ties);
    __shared__ uint32_t of_warp[2][kEvictWarps];
    if (lane == 0) {
        of_warp[0][warp] = above;
        of_warp[1][warp] = ties;
    }
    __syncthreads();
    above = lane < kEvictWarps ? of_warp[0][lane] : 0;
    ties = lane < kEvictWarps ? of_warp[1][lane] : 0;
    if (warp == 0) {
        const uint32_t all_above = __reduce_add_sync(0xffffffffu, above), all_ties = __reduce_add_sync(0xffffffffu, ties);
        if (lane == 0) {
            share[0] = all_above;
            share[1] = all_ties;
        }
    }
    uint32_t taken = __reduce_add_sync(0xffffffffu, lane < warp ? above : 0);
    uint32_t tied = __reduce_add_sync(0xffffffffu, lane < warp ? ties : 0);
    if (ctas > 1) {
        cluster_sync_all();
        taken += __reduce_add_sync(0xffffffffu, lane < part ? ld_dsmem_u32(dsmem_addr(&share[0], uint32_t(lane))) : 0);
        tied += __reduce_add_sync(0xffffffffu, lane < part ? ld_dsmem_u32(dsmem_addr(&share[1], uint32_t(lane))) : 0);
    }
    taken += min(tied, want);  // of the ties before, those that stay
    for (int i0 = begin; i0 < end; i0 += 128) {
        const int i = i0 + 4 * lane;
        stay(i, sure, tie);
        uint32_t all;  // both counts in one sum
        const uint32_t before = warp_before(uint32_t(__popc(sure)) | uint32_t(__popc(tie)) << 16, &all);
        // the ties before it, and those that stay
        uint32_t tie_at = tied + (before >> 16);
        uint32_t at = taken + (before & 0xffffu) + (min(tie_at, want) - min(tied, want));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool ties_here = tie >> j & 1;
            if ((sure >> j & 1) || (ties_here && tie_at < want)) kept[at++] = first + i + j;
            tie_at += ties_here;
        }
        taken += (all & 0xffffu) + (min(tied + (all >> 16), want) - min(tied, want));
        tied += all >> 16;
    }
    if (ctas > 1) cluster_sync_all();  // the others may still read this CTA's counts
}

// Few positions: a CTA for each head of each sequence counts for every position those that come before it in weight.
// (180 sequences of 2 positions, 12 heads, with the copy and the read back: 30 us with the kernel above.)
constexpr int kSmallThreads = 128, kSmallMost = 2 * kSmallThreads;
__global__ void __launch_bounds__(kSmallThreads) evict_choose_small_kernel(const EvictArgs a) {
    __shared__ __align__(16) uint32_t keys[kSmallMost];  // 0: not between, which no weight's is
    __shared__ uint32_t of_warp[32];
    pdl_next();
    const int64_t which = blockIdx.x, s = which / a.heads;
    const int head = int(which - s * a.heads), t = int(threadIdx.x), lane = t & 31, warp = t >> 5;
    int64_t length = ld_after(a.lengths + s);
    if (length < 0 || length > a.cap) {
        if (t == 0) atomicOr(a.err, kErrCacheSlot);
        length = length < 0 ? 0 : a.cap;
    }
    const int n = int(length);
    if (head == 0 && t == 0) a.new_lengths[s] = n < a.keep ? n : a.keep;
    int64_t* kept = a.kept + which * a.keep;
    if (n <= a.keep) {
        for (int64_t i = t; i < a.keep; i += kSmallThreads) kept[i] = i < n ? i : -1;
        return;
    }
    const float* weights = a.weights + s * a.weight_ts + head * a.weight_hs;
    const int from = int(a.first), to = n - int(a.recent);
    if (t < 32) of_warp[t] = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = t + j * kSmallThreads;
        keys[i] = i >= from && i < to ? weight_key(ld_after(weights + i)) : 0u;
    }
    __syncthreads();
    // this thread's two neighbouring positions
    const uint32_t want = uint32_t(a.keep - a.first - a.recent), mine[2] = {keys[2 * t], keys[2 * t + 1]};
    uint32_t rank[2] = {};
    for (int j = 0; j < to; j += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(keys + j);
        const uint32_t k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int m = 0; m < 2; ++m) rank[m] += k[u] > mine[m] || (k[u] == mine[m] && j + u < 2 * t + m);
    }
    uint32_t stays[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const int i = 2 * t + m;
        stays[m] = i < n && (i < from || i >= to || rank[m] < want);
    }
    uint32_t all;
    uint32_t at = warp_before(stays[0] + stays[1], &all);
    if (lane == 0) of_warp[warp] = all;
    __syncthreads();
    at += __reduce_add_sync(0xffffffffu, lane < warp ? of_warp[lane] : 0);
    if (stays[0]) kept[at] = 2 * t;
    if (stays[1]) kept[at + stays[0]] = 2 * t + 1;
}

// Which row a lane copies: row r of the shortened sequences, head innermost.
struct CopyDiv {
    RowDiv heads, keep;
};

// VEC bytes at once.  A warp takes 32 rows: each lane finds the places of one (its position, then the pages, which the
// next rows' are asked for ahead of) and copies its scales and its weight; then the lanes share the rows' codes,
// neighbouring lanes neighbouring vectors, a few rows of each lane under way.
template <int VEC>
__global__ void __launch_bounds__(kCopyThreads, 3) evict_copy_kernel(const EvictArgs a, CopyDiv by, int row_bytes) {
    using R = std::conditional_t<VEC == 16, uint4, std::conditional_t<VEC == 8, uint2, uint8_t>>;
    pdl_next();
    const int lane = threadIdx.x & 31;
    const int vecs = row_bytes / VEC, scales = a.d / a.cache.group;
    int lanes = 1, log = 0;  // of a row: as many as it has vectors (a power of two, at most 32)
    while (lanes < vecs && lanes < 32) lanes *= 2, ++log;
    const int mine = lane & (lanes - 1), row_of = lane >> log, at_once = 32 >> log;
    const int64_t rows = a.sequences * a.heads * a.keep;
    const uint64_t pages = uint64_t(a.cache.slots / a.cache.page.d);
    const int64_t step = int64_t(gridDim.x) * kCopyThreads;
    const CacheDev& c = a.cache;
    int64_t s = 0, i = 0, j = -1, from_page = -1, to_page = -1;  // sequence, new position and old one (-1: none), pages
    int head = 0;
    float weight = 0.f;
    auto position = [&](int64_t r) {
        j = -1;
        if (r >= rows) return;
        const int64_t in_seq = row_div(r, by.heads);
        head = int(r - in_seq * a.heads);
        s = row_div(in_seq, by.keep);
        i = in_seq - s * a.keep;
        j = ld_after(a.kept + (s * a.heads + head) * a.keep + i);
    };
    auto look_up = [&]() {
        if (j < 0) return;
        from_page = ld_after(a.table + s * a.table_stride + row_div(j, c.page));
        to_page = ld_after(a.new_table + s * a.new_stride + row_div(i, c.page));
        if (a.new_weights) weight = ld_after(a.weights + s * a.weight_ts + head * a.weight_hs + j);
    };
    int64_t r = int64_t(blockIdx.x) * kCopyThreads + threadIdx.x;
    position(r);
    look_up();
    for (int64_t r0 = r - lane; r0 < rows; r0 += step) {
        bool there = j >= 0;
        if (there && a.new_weights) a.new_weights[s * a.new_ts + head * a.new_hs + i] = weight;
        if (there && (uint64_t(from_page) >= pages || uint64_t(to_page) >= pages)) {
            atomicOr(a.err, kErrCacheSlot);
            there = false;
        }
        int64_t from = 0, to = 0, from_scale = 0, to_scale = 0;
        if (there) {
            const int64_t in_from = j - row_div(j, c.page) * c.page.d, in_to = i - row_div(i, c.page) * c.page.d;
            from = from_page * c.page_stride + in_from * c.slot_stride + head * c.head_stride;
            to = to_page * c.page_stride + in_to * c.slot_stride + head * c.head_stride;
            from_scale = from_page * c.scale_page_stride + in_from * c.scale_slot_stride + head * c.scale_head_stride;
            to_scale = to_page * c.scale_page_stride + in_to * c.scale_slot_stride + head * c.scale_head_stride;
        }
        const uint32_t all = __ballot_sync(0xffffffffu, there);
        r += step;
        position(r);
        // this lane's row's scales: the first of both at once
        if (there) {
            const float k = ld_after(c.scales[0] + from_scale), v = ld_after(c.scales[1] + from_scale);
            c.scales[0][to_scale] = k;
            c.scales[1][to_scale] = v;
            for (int g = 1; g < scales; ++g) {
                const float k2 = ld_after(c.scales[0] + from_scale + g), v2 = ld_after(c.scales[1] + from_scale + g);
                c.scales[0][to_scale + g] = k2;
                c.scales[1][to_scale + g] = v2;
            }
        }
        for (int q0 = 0; q0 < lanes; q0 += kCopyAhead) {
            R x[kCopyAhead][2];
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) {
                const int row = (q0 + k) * at_once + row_of;
                const int64_t at = __shfl_sync(0xffffffffu, from, row & 31);
                if (q0 + k < lanes && (all >> row & 1) && mine < vecs) {
                    x[k][0] = ld_after(reinterpret_cast<const R*>(c.codes[0] + at) + mine);
                    x[k][1] = ld_after(reinterpret_cast<const R*>(c.codes[1] + at) + mine);
                }
            }
#pragma unroll
            for (int k = 0; k < kCopyAhead; ++k) {
                const int row = (q0 + k) * at_once + row_of;
                const int64_t at = __shfl_sync(0xffffffffu, to, row & 31);
                const int64_t at_from = __shfl_sync(0xffffffffu, from, row & 31);
                if (q0 + k < lanes && (all >> row & 1)) {
                    if (mine < vecs) {
                        reinterpret_cast<R*>(c.codes[0] + at)[mine] = x[k][0];
                        reinterpret_cast<R*>(c.codes[1] + at)[mine] = x[k][1];
                    }
                    for (int v = mine + lanes; v < vecs; v += lanes)  // (rows of more than 32 vectors)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            reinterpret_cast<R*>(c.codes[t] + at)[v] =
                                ld_after(reinterpret_cast<const R*>(c.codes[t] + at_from) + v);
                }
            }
            if (q0 == 0) look_up();
        }
    }
}

nrm_status choose(EvictArgs& a, const DevInfo* dev, cudaStream_t s) {
    const int64_t pairs = a.sequences * a.heads;
    if (a.cap <= kSmallMost && pairs < (int64_t(1) << 31)) {
        void* p[] = {&a};
        return launch_pdl(reinterpret_cast<const void*>(&evict_choose_small_kernel), dim3(unsigned(pairs)), dim3(kSmallThreads), p, s);
    }
    // CTAs to a head: as its positions are worth, while the GPU has room
    int ctas = 1;
    while (ctas < kEvictCluster && a.cap > int64_t(ctas) * kEvictPart && pairs * ctas * 2 <= 2 * int64_t(dev->sms)) ctas *= 2;
    if (pairs * ctas >= (int64_t(1) << 31)) return fail(NRM_ERR_UNSUPPORTED, "sequences*heads must be < 2^31");
    const int64_t most = (a.cap + ctas * kEvictTurn - 1) / (ctas * kEvictTurn) * kEvictTurn;
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
    const int64_t want = (rows + kCopyThreads - 1) / kCopyThreads;
    void* q[] = {&a, &by, &bytes};
    const void* fn = vec == 16  ? reinterpret_cast<const void*>(&evict_copy_kernel<16>)
                     : vec == 8 ? reinterpret_cast<const void*>(&evict_copy_kernel<8>)
                                : reinterpret_cast<const void*>(&evict_copy_kernel<1>);
    return launch_pdl(fn, dim3(unsigned(std::min<int64_t>(want, int64_t(dev->sms) * 3))), dim3(kCopyThreads), q, s);
}

}  // namespace nrm
