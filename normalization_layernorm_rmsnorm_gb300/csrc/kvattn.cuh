// kvattn.cuh -- attention of one new token of each sequence over the paged,
// quantised key/value cache.
//
// The work is every position of every head of the cache once, so it is bound by
// the bytes of the codes.  Sequences are cut into tiles of 32 positions, all tiles
// of all sequences are dealt out in equal contiguous shares, and the workers (the
// warps of the GPU) take a share for one pair each (a head of the cache and the
// query heads that read it).  A share may end inside a sequence and begin inside
// another, so short and long sequences of one batch load the GPU evenly, and the
// cut is made on the device, from the lengths that lie there.  The workers of one
// share are neighbours, so that the heads of a slot, which lie side by side, are
// read at one time (one head after the other, 131072 positions in 4 bits read 1.7
// times their bytes).  Each worker runs the softmax with a running maximum and sum
// over its tiles of a sequence.  A sequence that lies in one share is written at
// once; of the others, each worker leaves its maximum, sum and accumulator in the
// workspace (it holds at most two such pieces: its first sequence's end and its
// last one's beginning), and a second kernel joins them.
// With weights, the logits lie in the workspace and a third kernel adds each
// position's weight once its sequence's sum is known.
#pragma once

#include <type_traits>

#include "heads.cuh"
#include "kvattn.h"

namespace nrm {

constexpr int kAttnThreads = 256;    // of a CTA of the kernel for any layout and of the one for the weights
constexpr int kJoinWarps = 16;

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// What a maximum is subtracted as: an empty one (all logits -infinity) as 0.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// The sequences' work, in shared memory, counted in tiles: a sequence's tiles and kAttnStart for its beginning (the
// queries, the first copies' wait, the result), none for one without positions.
struct AttnTable {
    int64_t n[kAttnSequences];        // positions
    int pre[kAttnSequences + 1];      // work before each sequence
    int sums[32];
};
__device__ __forceinline__ int attn_work(const AttnArgs& a, int64_t n) {
    const int64_t seen = a.window > 0 && n > a.window ? a.window : n;
    return seen > 0 ? int((seen + kAttnTile - 1) / kAttnTile) + kAttnStart : 0;
}
// The tile that work `c` of a sequence (from its beginning) belongs to.
__device__ __forceinline__ int attn_tile(int c) { return max(0, c - kAttnStart); }

// All threads of the CTA; CTA 0 writes the tiles to the workspace, for the kernels that follow.
__device__ __forceinline__ void attn_table(const AttnArgs& a, AttnTable& t) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = int(blockDim.x) >> 5;
    int before = 0;
    for (int s0 = 0; s0 < a.sequences; s0 += int(blockDim.x)) {
        const int s = s0 + int(threadIdx.x);
        int tiles = 0;
        if (s < a.sequences) {
            int64_t n = ld_after(a.lengths + s);
            if (n < 0 || n > a.cap) {
                atomicOr(a.err, kErrCacheSlot);
                n = n < 0 ? 0 : a.cap;
            }
            t.n[s] = n;
            tiles = attn_work(a, n);
        }
        int run = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += up;
        }
        if (lane == 31) t.sums[warp] = run;
        __syncthreads();
        const int w = lane < warps ? t.sums[lane] : 0;
        run += before + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
        before += __reduce_add_sync(0xffffffffu, w);
        if (s < a.sequences) {
            t.pre[s + 1] = run;
            if (blockIdx.x == 0) a.prefix[s + 1] = run;
        }
        if (s == 0) {
            t.pre[0] = 0;
            if (blockIdx.x == 0) a.prefix[0] = 0;
        }
        __syncthreads();
    }
}

// The shares of all sequences' work: the first `more` have one more.  Where there are more pairs than workers,
// one share.
struct AttnShares {
    int used, each, more;
    __device__ __forceinline__ AttnShares(const AttnArgs& a, int total) {
        used = max(1, min(total, a.workers / (a.hk * a.chunks)));
        each = total / used;
        more = total - each * used;
    }
    __device__ __forceinline__ int begin(int r) const { return r * each + min(r, more); }
    // the share that holds work t
    __device__ __forceinline__ int owner(int t) const {
        const int longer = more * (each + 1);
        return t < longer ? t / (each + 1) : more + (t - longer) / each;
    }
};
// The sequence that work t belongs to.
__device__ __forceinline__ int attn_sequence(const int* pre, int sequences, int t) {
    int lo = 0, hi = sequences - 1;  // the last s with pre[s] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pre[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A worker's piece of a sequence: tiles [tile0, tile1) of sequence s, for one pair.
struct AttnPiece {
    int s, head, q0, heads;  // head of the cache; query heads q0 .. q0 + heads - 1
    int pair;
    int tile0, tile1;
    bool whole;              // all of the sequence
    int64_t lo, n;           // positions that count
    int64_t part;            // where its partial result goes, if it is not whole
};
// The place of the partial result of share r for a pair: its first sequence's end (0) or its last one's beginning (1).
__device__ __forceinline__ int64_t attn_part(const AttnArgs& a, int r, int pair, int which) {
    return ((int64_t(r) * a.hk * a.chunks + pair) * 2 + which) * attn_part_floats(a.heads, a.d);
}

// Calls f(piece) for each piece of this warp's share.
template <typename F>
__device__ __forceinline__ void attn_pieces(const AttnArgs& a, const AttnTable& table, F&& f) {
    const int pairs = a.hk * a.chunks;
    const int total = table.pre[a.sequences];
    if (total == 0) return;
    const AttnShares shares(a, total);
    // as few warps of a CTA as the work takes, so that it fills the GPU
    const int warps = int(blockDim.x) >> 5, warp = int(threadIdx.x) >> 5;
    const int64_t work = int64_t(shares.used) * pairs;
    const int used_warps = int(min(int64_t(warps), (work + gridDim.x - 1) / gridDim.x));
    if (warp >= used_warps) return;
    // (more pairs than workers: a worker takes several)
    for (int64_t w = int(blockIdx.x) * used_warps + warp; w < work; w += int64_t(gridDim.x) * used_warps) {
        const int r = int(w / pairs), pair = int(w - int64_t(r) * pairs);
        // a share's end: a tile of a sequence, moved to the first one of a sequence that is short
        struct Edge {
            int s, tile;
        };
        auto edge = [&](int t) {
            if (t >= total) return Edge{a.sequences, 0};
            const int s = attn_sequence(table.pre, a.sequences, t), first = table.pre[s];
            return Edge{s, table.pre[s + 1] - first <= a.snap + kAttnStart ? 0 : attn_tile(t - first)};
        };
        const Edge from = edge(shares.begin(r)), to = edge(shares.begin(r + 1));
        const int head = pair / a.chunks, chunk = pair - head * a.chunks;
        for (int s = from.s; s < a.sequences && s <= to.s; ++s) {
            const int tiles = attn_tile(table.pre[s + 1] - table.pre[s]);
            AttnPiece p;
            p.tile0 = s == from.s ? from.tile : 0;
            p.tile1 = s == to.s ? to.tile : tiles;
            if (p.tile0 >= p.tile1) continue;
            p.s = s;
            p.pair = pair;
            p.head = head;
            p.q0 = head * a.shared + chunk * a.heads;
            p.heads = min(a.heads, a.shared - chunk * a.heads);
            p.n = table.n[s];
            p.lo = a.window > 0 && p.n > a.window ? p.n - a.window : 0;
            p.whole = p.tile0 == 0 && p.tile1 == tiles;
            p.part = attn_part(a, r, pair, p.tile0 == 0);
            f(p);
        }
    }
}

// A position's logits of a pair.
__device__ __forceinline__ float* attn_logits(const AttnArgs& a, int s, int pair, int64_t j) {
    return a.logits + ((int64_t(s) * a.hk * a.chunks + pair) * a.logit_stride + j) * a.logit_heads;
}

// Sequences without a position: out is 0, lse -infinity.
template <typename T>
__device__ __forceinline__ void attn_empty(const AttnArgs& a, const AttnTable& table) {
    for (int s = int(blockIdx.x); s < a.sequences; s += int(gridDim.x)) {
        if (table.pre[s + 1] != table.pre[s]) continue;
        typename Io<T>::bits_t* out = static_cast<typename Io<T>::bits_t*>(a.out.p) + s * a.out.ts;
        for (int i = int(threadIdx.x); i < a.hq * a.d; i += int(blockDim.x)) {
            const int h = i / a.d;
            out[h * a.out.hs + (i - h * a.d)] = Io<T>::store(0.f);
        }
        for (int h = int(threadIdx.x); h < a.hq; h += int(blockDim.x))
            if (a.lse) a.lse[int64_t(s) * a.hq + h] = -INFINITY;
    }
}

// The cache's row of position j of sequence s, or -1 (a page outside the cache).
__device__ __forceinline__ int64_t attn_slot(const AttnArgs& a, int s, int64_t j) {
    const int64_t entry = row_div(j, a.cache.page);
    const int64_t page = ld_after(a.table + s * a.table_stride + entry);
    if (page < 0 || page >= a.cache.slots / a.cache.page.d) {
        atomicOr(a.err, kErrCacheSlot);
        return -1;
    }
    return page * a.cache.page.d + (j - entry * a.cache.page.d);
}

__device__ __forceinline__ void attn_write_lse(const AttnArgs& a, int s, int h, float m, float sum) {
    // m and the logarithm in base 2; an empty row is -infinity
    const float l2 = sum == 0.f ? -INFINITY : finite_max(m) + log2f(sum);
    a.lse2[int64_t(s) * a.hq + h] = l2;
    if (a.lse) a.lse[int64_t(s) * a.hq + h] = l2 * 0.693147180559945309f;
}

// ---------------------------------------------------------------------------
// any layout: a lane holds every 32nd element of a row
// ---------------------------------------------------------------------------
__device__ __forceinline__ float code_value(const uint8_t* codes, int i, int kind) {
    if (kind == NRM_CACHE_INT4) {
        const uint32_t b = ld_after(codes + (i >> 1));
        return float(int32_t(b << (i & 1 ? 24 : 28)) >> 28);
    }
    const uint32_t b = ld_after(codes + i);
    return kind == NRM_CACHE_INT8 ? float(int8_t(b)) : e4m3x2_values(b).x;
}

template <typename T>
__global__ void __launch_bounds__(kAttnThreads) attn_scalar_kernel(const AttnArgs a) {
    using bits = typename Io<T>::bits_t;
    constexpr int E = kHeadMaxD / 32, H = kAttnScalarHeads;
    __shared__ AttnTable table;
    pdl_next();
    attn_table(a, table);
    attn_empty<T>(a, table);
    const int lane = threadIdx.x & 31;
    attn_pieces(a, table, [&](const AttnPiece& p) {
        float q[H][E], acc[H][E], m[H], sum[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            m[h] = -INFINITY;
            sum[h] = 0.f;
            const bits* row = static_cast<const bits*>(a.q.p) + p.s * a.q.ts + (p.q0 + h) * a.q.hs;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = lane + 32 * e;
                q[h][e] = h < p.heads && i < a.d ? Io<T>::load(ld_after(row + i)) : 0.f;
                acc[h][e] = 0.f;
            }
        }
        const int64_t j1 = min(p.n, p.lo + int64_t(p.tile1) * kAttnTile);
        for (int64_t j = p.lo + int64_t(p.tile0) * kAttnTile; j < j1; ++j) {
            const int64_t slot = attn_slot(a, p.s, j);
            float l[H];
            if (slot >= 0) {
                const CacheRow at = cache_row(a.cache, slot, p.head);
                float dot[H] = {};
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = lane + 32 * e;
                    if (i >= a.d) break;
                    const float k = code_value(a.cache.codes[0] + at.code, i, a.cache.kind) *
                                    ld_after(a.cache.scales[0] + at.scale + i / a.cache.group);
#pragma unroll
                    for (int h = 0; h < H; ++h) dot[h] = fmaf(q[h][e], k, dot[h]);
                }
                float grow[H], w[H];
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    l[h] = warp_sum(dot[h]) * a.scale_log2;
                    const float top = fmaxf(m[h], l[h]), base = finite_max(top);
                    grow[h] = exp2_approx(m[h] - base);
                    w[h] = exp2_approx(l[h] - base);
                    sum[h] = fmaf(sum[h], grow[h], w[h]);
                    m[h] = top;
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = lane + 32 * e;
                    if (i >= a.d) break;
                    const float v = code_value(a.cache.codes[1] + at.code, i, a.cache.kind) *
                                    ld_after(a.cache.scales[1] + at.scale + i / a.cache.group);
#pragma unroll
                    for (int h = 0; h < H; ++h) acc[h][e] = fmaf(acc[h][e], grow[h], w[h] * v);
                }
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h) l[h] = -INFINITY;
            }
            if (a.logits && lane < p.heads) {
                float mine = l[0];
#pragma unroll
                for (int h = 1; h < H; ++h) mine = lane == h ? l[h] : mine;
                attn_logits(a, p.s, p.pair, j)[lane] = mine;
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if (h >= p.heads) break;
            const float scale = p.whole ? (sum[h] == 0.f ? 0.f : 1.f / sum[h]) : 1.f;
            bits* row = static_cast<bits*>(a.out.p) + p.s * a.out.ts + (p.q0 + h) * a.out.hs;
            float* part = a.part + p.part + h * attn_part_row(a.d);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = lane + 32 * e;
                if (i >= a.d) break;
                if (p.whole) row[i] = Io<T>::store(acc[h][e] * scale);
                else part[i] = acc[h][e];
            }
            if (lane == 0) {
                if (p.whole) {
                    attn_write_lse(a, p.s, p.q0 + h, m[h], sum[h]);
                } else {
                    part[a.d] = m[h];
                    part[a.d + 1] = sum[h];
                }
            }
        }
    });
}

// ---------------------------------------------------------------------------
// joining the pieces of a sequence: a CTA for each pair (blockIdx.x), or, where pairs
// are few and so have many pieces, for each of its heads (blockIdx.y).  Its warps
// share the heads, and the warps of a head its pieces.
// ---------------------------------------------------------------------------
template <typename T, int E>  // E: rows of up to E * 128
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const AttnArgs a) {
    using bits = typename Io<T>::bits_t;
    constexpr int AHEAD = 8 / E;  // pieces of a warp under way
    __shared__ float4 joined[kJoinWarps][E * 32];
    __shared__ float sums[kJoinWarps], tops[kJoinWarps];
    const int warps = int(blockDim.x) >> 5;
    pdl_next();
    const int pairs = a.hk * a.chunks;
    const int s = int(blockIdx.x) / pairs, pair = int(blockIdx.x) - s * pairs;
    const int before = ld_after(a.prefix + s), work = ld_after(a.prefix + s + 1) - before;
    const AttnShares shares(a, ld_after(a.prefix + a.sequences));
    if (work <= a.snap + kAttnStart) return;
    const int w0 = shares.owner(before + kAttnStart), w1 = shares.owner(before + work - 1);
    if (w0 == w1) return;  // written by that worker
    const int head = pair / a.chunks, chunk = pair - head * a.chunks;
    const int heads = min(a.heads, a.shared - chunk * a.heads), q0 = head * a.shared + chunk * a.heads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // heads of this CTA, in rounds of as many as have warps of their own
    const int mine = gridDim.y > 1 ? 1 : heads, at_once = min(mine, warps), each = warps / at_once;
    const int group = warp / each, in_group = warp - group * each;
    for (int h0 = 0; h0 < mine; h0 += at_once) {
        const int h = gridDim.y > 1 ? int(blockIdx.y) : h0 + group;
        const bool there = group < at_once && h0 + group < mine && h < heads;
        // the first worker's piece is the beginning of its last sequence, the others' the end of their first
        auto part = [&](int w) {
            return a.part + attn_part(a, w, pair, w == w0) + h * attn_part_row(a.d);
        };
        if (there) {
            float top = -INFINITY, sum = 0.f;
            float4 acc[E];
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = w0 + in_group; w <= w1; w += AHEAD * each) {
                float m[AHEAD], l[AHEAD];
                uint4 v[AHEAD][E];
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    m[k] = -INFINITY;
                    l[k] = 0.f;
                    if (w + k * each > w1) continue;
                    const float* from = part(w + k * each);
                    m[k] = ld_after(from + a.d);
                    l[k] = ld_after(from + a.d + 1);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (lane * 4 + 128 * e < a.d) v[k][e] = ld_after(reinterpret_cast<const uint4*>(from) + lane + 32 * e);
                }
                float most = top;
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) most = fmaxf(most, m[k]);
                const float base = finite_max(most), grow = exp2_approx(top - base);
                top = most;
                sum *= grow;
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = make_float4(acc[e].x * grow, acc[e].y * grow, acc[e].z * grow, acc[e].w * grow);
#pragma unroll
                for (int k = 0; k < AHEAD; ++k) {
                    if (w + k * each > w1) continue;
                    const float f = exp2_approx(m[k] - base);
                    sum = fmaf(l[k], f, sum);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (lane * 4 + 128 * e >= a.d) break;
                        acc[e].x = fmaf(__uint_as_float(v[k][e].x), f, acc[e].x);
                        acc[e].y = fmaf(__uint_as_float(v[k][e].y), f, acc[e].y);
                        acc[e].z = fmaf(__uint_as_float(v[k][e].z), f, acc[e].z);
                        acc[e].w = fmaf(__uint_as_float(v[k][e].w), f, acc[e].w);
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (lane * 4 + 128 * e < a.d) joined[warp][lane + 32 * e] = acc[e];
            if (lane == 0) {
                sums[warp] = sum;
                tops[warp] = top;
            }
        }
        __syncthreads();
        if (there) {
            float top = -INFINITY, all = 0.f;
            for (int k = 0; k < each; ++k) top = fmaxf(top, tops[group * each + k]);
            const float base = finite_max(top);
            for (int k = 0; k < each; ++k) all = fmaf(sums[group * each + k], exp2_approx(tops[group * each + k] - base), all);
            const float scale = all == 0.f ? 0.f : 1.f / all;
            bits* row = static_cast<bits*>(a.out.p) + s * a.out.ts + (q0 + h) * a.out.hs;
            for (int i = in_group * 32 + lane; i < a.d; i += each * 32) {
                float v = 0.f;
                for (int k = 0; k < each; ++k)
                    v = fmaf(reinterpret_cast<const float*>(joined[group * each + k])[i], exp2_approx(tops[group * each + k] - base), v);
                row[i] = Io<T>::store(v * scale);
            }
            if (in_group == 0 && lane == 0) attn_write_lse(a, s, q0 + h, top, all);
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// each position's weight, from its logits and its sequence's sum
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) attn_weights_kernel(const AttnArgs a) {
    constexpr int AHEAD = 4;
    __shared__ int pre[kAttnSequences + 1];
    pdl_next();
    for (int s = int(threadIdx.x); s <= a.sequences; s += kAttnThreads) pre[s] = ld_after(a.prefix + s);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int total = pre[a.sequences] * a.hk, warps = int(gridDim.x) * (kAttnThreads / 32);
    const int w = int(threadIdx.x >> 5) * int(gridDim.x) + int(blockIdx.x);
    const int each = total / warps, more = total - each * warps;
    int t = w * each + min(w, more);
    const int end = t + each + (w < more);
    if (t >= end) return;
    int s = attn_sequence(pre, a.sequences, t / a.hk);
    while (t < end) {
        while (pre[s + 1] * a.hk <= t) ++s;
        const int work = pre[s + 1] - pre[s], at = t - pre[s] * a.hk;
        const int head = at / work, work0 = at - head * work, work1 = min(work, work0 + (end - t));
        const int tile0 = attn_tile(work0), tile1 = attn_tile(work1);
        const int64_t n = max(int64_t(0), min(a.cap, ld_after(a.lengths + s)));
        const int64_t lo = a.window > 0 && n > a.window ? n - a.window : 0;
        const int64_t j1 = min(n, lo + int64_t(tile1) * kAttnTile);
        float* out = a.weights + s * a.weight_ts + head * a.weight_hs;
        for (int64_t j = lo + int64_t(tile0) * kAttnTile + lane; j < j1; j += 32 * AHEAD) {
            float sum[AHEAD] = {};
            for (int c = 0; c < a.chunks; ++c) {
                const float* lse2 = a.lse2 + int64_t(s) * a.hq + head * a.shared + c * a.heads;
                const int heads = min(a.heads, a.shared - c * a.heads);
                const float* logits = attn_logits(a, s, head * a.chunks + c, j);
                for (int h = 0; h < heads; h += 2) {
                    const float l0 = ld_after(lse2 + h), l1 = h + 1 < heads ? ld_after(lse2 + h + 1) : 0.f;
                    uint2 v[AHEAD];
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k)
                        if (j + 32 * k < j1)
                            v[k] = ld_after(reinterpret_cast<const uint2*>(logits + int64_t(32 * k) * a.logit_heads + h));
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        if (j + 32 * k >= j1) break;
                        const float x = __uint_as_float(v[k].x), y = __uint_as_float(v[k].y);
                        sum[k] += x == -INFINITY ? 0.f : exp2_approx(x - l0);
                        if (h + 1 < heads) sum[k] += y == -INFINITY ? 0.f : exp2_approx(y - l1);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (j + 32 * k < j1) out[j + 32 * k] += sum[k];
        }
        t += work1 - work0;
    }
}

}  // namespace nrm
