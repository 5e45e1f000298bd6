// kvattn.cuh -- attention of one new token of each sequence over the paged,
// quantised key/value cache.
//
// The work is every position of every head of the cache once, so it is bound by
// the bytes of the codes.  Sequences are cut into tiles of 32 positions, and all
// tiles of all sequences and heads are dealt to the warps of the GPU in equal
// contiguous shares: a worker's share may end inside a sequence and begin inside
// another, so short and long sequences of one batch load the GPU evenly, and the
// cut is made on the device, from the lengths that lie there.  Each worker runs
// the softmax with a running maximum and sum over its tiles of a pair (a head of
// the cache and the query heads that read it).  A pair that lies in one worker's
// share is written at once; of the others, each worker leaves its maximum, sum
// and accumulator in the workspace (it holds at most two such pieces: its first
// pair's end and its last pair's beginning), and a second kernel joins them.
// With weights, the logits lie in the workspace and a third kernel adds each
// position's weight once its sequence's sum is known.
#pragma once

#include <type_traits>

#include "heads.cuh"
#include "kvattn.h"

namespace nrm {

constexpr int kAttnThreads = 32 * kAttnWarps;

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// What a maximum is subtracted as: an empty one (all logits -infinity) as 0.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// The positions of sequence s that count: [lo, n).
struct AttnSpan {
    int64_t lo, n;
};
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& a, int s) {
    int64_t n = ld_after(a.lengths + s);
    if (n < 0 || n > a.cap) {
        atomicOr(a.err, kErrCacheSlot);
        n = n < 0 ? 0 : a.cap;
    }
    return AttnSpan{a.window > 0 && n > a.window ? n - a.window : 0, n};
}

// Tiles before each sequence, in shared memory; all threads of the CTA.
__device__ __forceinline__ void attn_prefix(const AttnArgs& a, int64_t* pre, int64_t* sums) {
    constexpr int per = kAttnSequences / kAttnThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t tiles[per], total = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int s = int(threadIdx.x) * per + i;
        tiles[i] = 0;
        if (s < a.sequences) {
            const AttnSpan p = attn_span(a, s);
            tiles[i] = (p.n - p.lo + kAttnTile - 1) / kAttnTile;
        }
        total += tiles[i];
    }
    int64_t run = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    int64_t before = run - total;
    for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int s = int(threadIdx.x) * per + i;
        if (s < a.sequences) pre[s] = before;
        before += tiles[i];
        if (s == a.sequences - 1) pre[a.sequences] = before;
    }
    __syncthreads();
}

// Workers that get a share of `total` tiles, and where shares begin.
__device__ __forceinline__ int64_t attn_used(const AttnArgs& a, int64_t total) {
    const int64_t w = (total + a.min_tiles - 1) / a.min_tiles;
    return w < a.workers ? w : a.workers;
}
__device__ __forceinline__ int64_t attn_begin(int64_t total, int64_t used, int64_t w) { return total * w / used; }
// The worker whose share holds tile t.
__device__ __forceinline__ int64_t attn_owner(int64_t total, int64_t used, int64_t t) {
    return ((t + 1) * used - 1) / total;
}
// The sequence that tile `t` of the sequences' tiles (not their pairs') belongs to.
__device__ __forceinline__ int attn_sequence(const int64_t* pre, int sequences, int64_t t) {
    int lo = 0, hi = sequences - 1;  // the last s with pre[s] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pre[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A worker's piece of one pair: tiles [tile0, tile1) of sequence s.
struct AttnPiece {
    int s, head, q0, heads;  // head of the cache; query heads q0 .. q0 + heads - 1
    int64_t lo, n;           // positions that count
    int64_t tile0, tile1;
    bool whole;              // all of the pair
    int64_t part;            // else: where its partial result goes
};

// Calls f(piece) for each piece of worker w's share.  `pre`: shared memory.
template <typename F>
__device__ __forceinline__ void attn_pieces(const AttnArgs& a, const int64_t* pre, int64_t w, F&& f) {
    const int pairs = a.hk * a.chunks;
    const int64_t total = pre[a.sequences] * pairs, used = attn_used(a, total);
    if (w >= used) return;
    int64_t t = attn_begin(total, used, w);
    const int64_t end = attn_begin(total, used, w + 1);
    int s = attn_sequence(pre, a.sequences, t / pairs);
    while (t < end) {
        while (pre[s + 1] * pairs <= t) ++s;  // (sequences without tiles are passed over)
        const int64_t tiles = pre[s + 1] - pre[s], at = t - pre[s] * pairs;
        const int pair = int(at / tiles);
        AttnPiece p;
        p.s = s;
        p.head = pair / a.chunks;
        const int chunk = pair - p.head * a.chunks;
        p.q0 = p.head * a.shared + chunk * a.heads;
        p.heads = min(a.heads, a.shared - chunk * a.heads);
        const AttnSpan span = attn_span(a, s);
        p.lo = span.lo;
        p.n = span.n;
        p.tile0 = at - pair * tiles;
        p.tile1 = min(tiles, p.tile0 + (end - t));
        p.whole = p.tile0 == 0 && p.tile1 == tiles;
        // its first pair's end, or its last pair's beginning
        p.part = (w * 2 + (p.tile0 == 0 ? 1 : 0)) * attn_part_floats(a.heads, a.d);
        f(p);
        t += p.tile1 - p.tile0;
    }
}

// Sequences without a position: out is 0, lse -infinity.
template <typename T>
__device__ __forceinline__ void attn_empty(const AttnArgs& a, const int64_t* pre) {
    for (int s = int(blockIdx.x); s < a.sequences; s += int(gridDim.x)) {
        if (pre[s + 1] != pre[s]) continue;
        typename Io<T>::bits_t* out = static_cast<typename Io<T>::bits_t*>(a.out.p) + s * a.out.ts;
        for (int i = int(threadIdx.x); i < a.hq * a.d; i += kAttnThreads) {
            const int h = i / a.d;
            out[h * a.out.hs + (i - h * a.d)] = Io<T>::store(0.f);
        }
        for (int h = int(threadIdx.x); h < a.hq; h += kAttnThreads)
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
constexpr int kAttnScalarHeads = 4;  // query heads of a worker

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
    __shared__ int64_t pre[kAttnSequences + 1], sums[kAttnWarps];
    pdl_next();
    attn_prefix(a, pre, sums);
    if (blockIdx.x == 0)
        for (int s = int(threadIdx.x); s <= a.sequences; s += kAttnThreads) a.prefix[s] = pre[s];
    attn_empty<T>(a, pre);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    attn_pieces(a, pre, int64_t(warp) * gridDim.x + blockIdx.x, [&](const AttnPiece& p) {
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
        const int64_t j1 = min(p.n, p.lo + p.tile1 * kAttnTile);
        for (int64_t j = p.lo + p.tile0 * kAttnTile; j < j1; ++j) {
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
                a.logits[(int64_t(p.s) * a.hq + p.q0 + lane) * a.logit_stride + j] = mine;
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
// joining the pieces of a pair: a CTA for each query head
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(const AttnArgs a) {
    using bits = typename Io<T>::bits_t;
    constexpr int E = kHeadMaxD / 32;
    __shared__ float joined[kAttnWarps][kHeadMaxD], sums[kAttnWarps];
    pdl_next();
    const int s = int(blockIdx.x) / a.hq, hq = int(blockIdx.x) - s * a.hq;
    const int head = hq / a.shared, in_head = hq - head * a.shared;
    const int chunk = in_head / a.heads, h = in_head - chunk * a.heads;
    const int pairs = a.hk * a.chunks, pair = head * a.chunks + chunk;
    const int64_t before = ld_after(a.prefix + s), tiles = ld_after(a.prefix + s + 1) - before;
    const int64_t total = ld_after(a.prefix + a.sequences) * pairs;
    if (tiles == 0) return;
    const int64_t used = attn_used(a, total), t0 = before * pairs + pair * tiles;
    const int64_t w0 = attn_owner(total, used, t0), w1 = attn_owner(total, used, t0 + tiles - 1);
    if (w0 == w1) return;  // written by that worker
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the first worker's piece is the beginning of its last pair, the others' the end of their first
    auto part = [&](int64_t w) {
        return a.part + (w * 2 + (w == w0)) * attn_part_floats(a.heads, a.d) + h * attn_part_row(a.d);
    };
    float top = -INFINITY;
    for (int64_t w = w0 + lane; w <= w1; w += 32) {
        const float m = ld_after(part(w) + a.d);
        top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = finite_max(top);
    float acc[E] = {}, sum = 0.f;
    for (int64_t w = w0 + warp; w <= w1; w += kAttnWarps) {
        const float* from = part(w);
        const float f = exp2_approx(ld_after(from + a.d) - base);
        sum = fmaf(ld_after(from + a.d + 1), f, sum);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (lane + 32 * e < a.d) acc[e] = fmaf(ld_after(from + lane + 32 * e), f, acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (lane + 32 * e < a.d) joined[warp][lane + 32 * e] = acc[e];
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    float all = 0.f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) all += sums[w];
    const float scale = all == 0.f ? 0.f : 1.f / all;
    bits* row = static_cast<bits*>(a.out.p) + s * a.out.ts + hq * a.out.hs;
    for (int i = int(threadIdx.x); i < a.d; i += kAttnThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) v += joined[w][i];
        row[i] = Io<T>::store(v * scale);
    }
    if (threadIdx.x == 0) attn_write_lse(a, s, hq, top, all);
}

// ---------------------------------------------------------------------------
// each position's weight, from its logits and its sequence's sum
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) attn_weights_kernel(const AttnArgs a) {
    __shared__ int64_t pre[kAttnSequences + 1];
    pdl_next();
    for (int s = int(threadIdx.x); s <= a.sequences; s += kAttnThreads) pre[s] = ld_after(a.prefix + s);
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int64_t total = pre[a.sequences] * a.hk, warps = int64_t(gridDim.x) * kAttnWarps;
    const int64_t w = int64_t(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    int64_t t = total * w / warps;
    const int64_t end = total * (w + 1) / warps;
    if (t >= end) return;
    int s = attn_sequence(pre, a.sequences, t / a.hk);
    while (t < end) {
        while (pre[s + 1] * a.hk <= t) ++s;
        const int64_t tiles = pre[s + 1] - pre[s], at = t - pre[s] * a.hk;
        const int head = int(at / tiles);
        const int64_t tile0 = at - head * tiles, tile1 = min(tiles, tile0 + (end - t));
        const AttnSpan span = attn_span(a, s);
        const float* lse2 = a.lse2 + int64_t(s) * a.hq + head * a.shared;
        const float* logits = a.logits + (int64_t(s) * a.hq + head * a.shared) * a.logit_stride;
        float* out = a.weights + s * a.weight_ts + head * a.weight_hs;
        for (int64_t j = span.lo + tile0 * kAttnTile + lane; j < min(span.n, span.lo + tile1 * kAttnTile); j += 32) {
            float sum = 0.f;
            for (int h = 0; h < a.shared; ++h) {
                const float l = ld_after(logits + h * a.logit_stride + j);
                sum += l == -INFINITY ? 0.f : exp2_approx(l - ld_after(lse2 + h));
            }
            out[j] += sum;
        }
        t += tile1 - tile0;
    }
}

}  // namespace nrm
