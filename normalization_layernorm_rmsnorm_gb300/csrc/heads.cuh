// heads.cuh -- kernels on attention heads: RMSNorm of each head with the
// position rotation in the same pass, forward and backward, the rotation alone,
// and the quantised key/value cache (written from given rows, from the key the
// norm and rotation just made, and read back).
//
// One row is one token's head of d <= 256 elements.  This first form gives a row
// to a warp: lane l holds the pair slots l, l + 32, ...; a slot is the two
// elements that turn together, or two neighbours past the rotated part.
#pragma once

#include "common.cuh"
#include "heads.h"

namespace nrm {

constexpr int kHeadWarps = 8;                       // warps of a CTA
constexpr int kHeadSlots = kHeadMaxPairs / 32;      // pair slots of a lane

// ---------------------------------------------------------------------------
// angles
// ---------------------------------------------------------------------------

// inv_freq as a fraction of a turn per position, in units of 2^-64 turns: the
// product with an integer position then wraps at whole turns by itself, so the
// angle of a far position is as exact as that of a near one.
__device__ __forceinline__ uint64_t turn_step(float inv_freq) {
    double f = double(inv_freq) * 0.15915494309189533577;  // 1 / (2 pi)
    f -= floor(f);
    return __double2ull_rz(f * 18446744073709551616.0);
}

__device__ __forceinline__ int pair_axis(const RopeDev& r, int p) {
    return int(r.axis[p >> 4] >> ((p & 15) * 2)) & 3;
}

// cos and sin of pair p of token t.  The top 32 bits of the phase, read as
// signed, are the angle in units of 2^-31 half turns.
__device__ __forceinline__ float2 pair_turn(const RopeDev& r, int p, int64_t t) {
    const int64_t pos = __ldg(r.pos + pair_axis(r, p) * r.pos_stride + t);
    const uint64_t phase = uint64_t(pos) * turn_step(__ldg(r.inv_freq + p));
    float s, c;
    sincospif(float(int32_t(phase >> 32)) * 0x1p-31f, &s, &c);
    return make_float2(c, r.inverse ? -s : s);
}

// (u, v) turned by (cos, sin); the products' roundings are spelt out so that
// every kernel that turns the same pair gets the same bits.
__device__ __forceinline__ void turn(float& u, float& v, float2 cs) {
    const float a = fmaf(u, cs.x, -__fmul_rn(v, cs.y));
    const float b = fmaf(v, cs.x, __fmul_rn(u, cs.y));
    u = a;
    v = b;
}

// ---------------------------------------------------------------------------
// quantising a group by its largest magnitude
// ---------------------------------------------------------------------------
__device__ __forceinline__ float cache_qmax(int kind) {
    return kind == NRM_CACHE_E4M3 ? 448.f : (kind == NRM_CACHE_INT8 ? 127.f : 7.f);
}

// A group's scale and what its codes need, from the bits of its largest
// magnitude (compared as integers, so a NaN is the largest of all).
struct GroupQ {
    float scale;
    float m;     // largest magnitude; 0 where every code is 0
    float q;
};
__device__ __forceinline__ GroupQ group_q(uint32_t m_bits, int kind) {
    GroupQ g;
    g.q = cache_qmax(kind);
    g.m = __uint_as_float(m_bits);
    if (m_bits >= 0x7f800000u) {       // a NaN or an infinity: the group reads back as NaN
        g.scale = __uint_as_float(0x7fffffffu);
        g.m = 0.f;
    } else if (g.m < 0x1p-100f) {      // nothing but (almost) zeros
        g.scale = 0.f;
        g.m = 0.f;
    } else {
        g.scale = __fdiv_rn(g.m, g.q);
    }
    return g;
}
// x*q/m, so that the code nearest to the real quotient is the one nearest to
// this.  Groups above 2^100 are divided by 2^32 first and groups below 2^-36
// multiplied by 2^64 (both exact where it matters), so that products stay finite
// and residuals representable.
// 16-bit x: the product is exact and the quotient rounded once, so a value half
// way between two codes is seen as that, and any other quotient of such numbers
// is further from half way than its rounding reaches.
// float32 x: the quotient is rounded to odd (one further step of division first,
// as the rounded product alone leaves it up to 1.5 ulp off): a quotient that is
// not exact never lands on an even number, and so never half way between codes.
template <typename T>
__device__ __forceinline__ float group_scaled(float x, const GroupQ& g) {
    if (g.m == 0.f) return 0.f;
    const float p = g.m > 0x1p100f ? 0x1p-32f : (g.m < 0x1p-36f ? 0x1p64f : 1.f);
    const float a = x * p, m = g.m * p;
    const float n = __fmul_rn(a, g.q);
    float u = __fdiv_rn(n, m);
    if constexpr (sizeof(T) == 4) {
        const float lost = fmaf(a, g.q, -n);             // n + lost == a*q
        u = __fadd_rn(u, __fdiv_rn(fmaf(-u, m, n) + lost, m));
        const float left = fmaf(-u, m, n) + lost;        // its sign: which side of u the quotient lies on
        const int bits = __float_as_int(u);
        if (left != 0.f && (bits & 1) == 0 && fabsf(u) >= 0x1p-24f)
            u = __int_as_float(bits + ((left > 0.f) == (u > 0.f) ? 1 : -1));
    }
    return u;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_values(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t code_of(float u, int kind) {
    if (kind == NRM_CACHE_E4M3) return e4m3x2(u, 0.f) & 0xffu;
    return uint32_t(__float2int_rn(u)) & (kind == NRM_CACHE_INT8 ? 0xffu : 0xfu);
}

// Byte and float offsets of a slot's row.  A slot outside the cache is -1.
struct CacheRow {
    int64_t code, scale;
};
__device__ __forceinline__ int64_t cache_slot(const CacheDev& c, int64_t slot, unsigned int* err) {
    if (slot >= 0 && slot < c.slots) return slot;
    if (slot != -1) atomicOr(err, kErrCacheSlot);
    return -1;
}
__device__ __forceinline__ CacheRow cache_row(const CacheDev& c, int64_t slot, int head) {
    const int64_t page = slot / c.page_size, at = slot - page * c.page_size;
    return CacheRow{page * c.page_stride + at * c.slot_stride + head * c.head_stride,
                    page * c.scale_page_stride + at * c.scale_slot_stride + head * c.scale_head_stride};
}

// Quantises the d values of `row` (of T, as floats in shared memory, visible to
// the warp) into the cache's tensor `which` (0: keys, 1: values).
template <typename T>
__device__ __forceinline__ void quantise_row(const float* row, int d, const CacheDev& c, int which, int64_t slot,
                                             int head, int lane) {
    const CacheRow at = cache_row(c, slot, head);
    uint8_t* codes = c.codes[which] + at.code;
    float* scales = c.scales[which] + at.scale;
    for (int g0 = 0; g0 < d; g0 += c.group) {
        uint32_t m = 0;
        for (int i = lane; i < c.group; i += 32) m = max(m, __float_as_uint(row[g0 + i]) & 0x7fffffffu);
        const GroupQ q = group_q(__reduce_max_sync(0xffffffffu, m), c.kind);
        if (lane == 0) scales[g0 / c.group] = q.scale;
        if (c.kind == NRM_CACHE_INT4) {
            for (int i = 2 * lane; i < c.group; i += 64)
                codes[(g0 + i) / 2] = uint8_t(code_of(group_scaled<T>(row[g0 + i], q), c.kind) |
                                              code_of(group_scaled<T>(row[g0 + i + 1], q), c.kind) << 4);
        } else {
            for (int i = lane; i < c.group; i += 32)
                codes[g0 + i] = uint8_t(code_of(group_scaled<T>(row[g0 + i], q), c.kind));
        }
    }
}

// ---------------------------------------------------------------------------
// any layout: a row per warp, two elements per slot
// ---------------------------------------------------------------------------

// The elements of pair slot j (e1 == d: past the end of an odd row) and whether they turn.
struct SlotAt {
    int e0, e1;
    bool turns;
};
__device__ __forceinline__ SlotAt slot_at(int j, int d, const RopeDev& r) {
    const int half = r.rot >> 1;
    if (j < half) return r.adjacent ? SlotAt{2 * j, 2 * j + 1, true} : SlotAt{j, j + half, true};
    return SlotAt{2 * j, min(2 * j + 1, d), false};
}

template <typename T>
__device__ __forceinline__ float ld_elem(const void* p, int64_t i) {
    return Io<T>::load(reinterpret_cast<const typename Io<T>::bits_t*>(p)[i]);
}
template <typename T>
__device__ __forceinline__ void st_elem(void* p, int64_t i, float v) {
    reinterpret_cast<typename Io<T>::bits_t*>(p)[i] = Io<T>::store(v);
}
template <typename T>
__device__ __forceinline__ float round_to(float v) {
    return Io<T>::load(Io<T>::store(v));
}

template <typename T, bool NORM, bool CACHE>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_fwd_scalar_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ float stage[CACHE ? kHeadWarps : 1][CACHE ? kHeadMaxD : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = a.heads[0] + a.heads[1] + (CACHE ? a.heads[2] : 0);
    const int slots = (a.d + 1) >> 1;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float2 cs[kHeadSlots];
#pragma unroll
        for (int s = 0; s < kHeadSlots; ++s)
            if (2 * (lane + 32 * s) < a.rope.rot) cs[s] = pair_turn(a.rope, lane + 32 * s, t);
        const int64_t slot = CACHE ? cache_slot(a.cache, __ldg(a.slots + t), a.err) : -1;
        for (int hh = warp + int(blockIdx.y) * kHeadWarps; hh < heads; hh += int(gridDim.y) * kHeadWarps) {
            const int which = hh < a.heads[0] ? 0 : (hh < a.heads[0] + a.heads[1] ? 1 : 2);
            const int h = hh - (which > 0 ? a.heads[0] : 0) - (which > 1 ? a.heads[1] : 0);
            const HeadView xv = a.x[which];
            const T* x = reinterpret_cast<const T*>(xv.p) + t * xv.ts + h * xv.hs;
            float u[kHeadSlots], v[kHeadSlots];
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < kHeadSlots; ++s) {
                const int j = lane + 32 * s;
                u[s] = v[s] = 0.f;
                if (j < slots) {
                    const SlotAt e = slot_at(j, a.d, a.rope);
                    u[s] = ld_elem<T>(x, e.e0);
                    if (e.e1 < a.d) v[s] = ld_elem<T>(x, e.e1);
                    if (NORM) sum = fmaf(u[s], u[s], fmaf(v[s], v[s], sum));
                }
            }
            if (which < 2) {
                float r = 1.f;
                if (NORM) {
                    r = rsqrtf(warp_sum(sum) / float(a.d) + a.eps);
                    if (lane == 0 && a.rstd[which]) a.rstd[which][t * a.heads[which] + h] = r;
                }
#pragma unroll
                for (int s = 0; s < kHeadSlots; ++s) {
                    const int j = lane + 32 * s;
                    if (j < slots) {
                        const SlotAt e = slot_at(j, a.d, a.rope);
                        if (NORM) {
                            u[s] = __fmul_rn(u[s], r);
                            v[s] = __fmul_rn(v[s], r);
                            if (a.w[which]) {
                                u[s] = __fmul_rn(u[s], ld_elem<T>(a.w[which], e.e0));
                                if (e.e1 < a.d) v[s] = __fmul_rn(v[s], ld_elem<T>(a.w[which], e.e1));
                            }
                        }
                        if (e.turns) turn(u[s], v[s], cs[s]);
                        const HeadView yv = a.y[which];
                        if (yv.p) {
                            T* y = reinterpret_cast<T*>(yv.p) + t * yv.ts + h * yv.hs;
                            st_elem<T>(y, e.e0, u[s]);
                            if (e.e1 < a.d) st_elem<T>(y, e.e1, v[s]);
                        }
                    }
                }
            }
            if (CACHE && which > 0 && slot >= 0) {
                // the cache stores the key in the activations' type: what a separate write would read
                float* row = stage[warp];
#pragma unroll
                for (int s = 0; s < kHeadSlots; ++s) {
                    const int j = lane + 32 * s;
                    if (j < slots) {
                        const SlotAt e = slot_at(j, a.d, a.rope);
                        row[e.e0] = round_to<T>(u[s]);
                        if (e.e1 < a.d) row[e.e1] = round_to<T>(v[s]);
                    }
                }
                __syncwarp();
                quantise_row<T>(row, a.d, a.cache, which - 1, slot, h, lane);
                __syncwarp();
            }
        }
    }
}

// Backward.  CTAs [0, nq) take q, the others k, so that a thread's sums for dw
// belong to one weight; each CTA writes its partial row [d].
template <typename T>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_bwd_scalar_kernel(const __grid_constant__ HeadArgs a, int nq) {
    __shared__ float part[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = int(blockIdx.x) < nq ? 0 : 1;
    const int cta = int(blockIdx.x) - (which ? nq : 0);
    const int ctas = which ? int(gridDim.x) - nq : nq;
    const int slots = (a.d + 1) >> 1;
    float acc_u[kHeadSlots] = {}, acc_v[kHeadSlots] = {};
    for (int64_t t = cta; t < a.tokens; t += ctas) {
        float2 cs[kHeadSlots];
#pragma unroll
        for (int s = 0; s < kHeadSlots; ++s)
            if (2 * (lane + 32 * s) < a.rope.rot) cs[s] = pair_turn(a.rope, lane + 32 * s, t);
        for (int h = warp; h < a.heads[which]; h += kHeadWarps) {
            const T* x = reinterpret_cast<const T*>(a.x[which].p) + t * a.x[which].ts + h * a.x[which].hs;
            const T* dy = reinterpret_cast<const T*>(a.dy[which].p) + t * a.dy[which].ts + h * a.dy[which].hs;
            T* dx = reinterpret_cast<T*>(a.y[which].p) + t * a.y[which].ts + h * a.y[which].hs;
            const float r = a.rstd[which][t * a.heads[which] + h];
            float u[kHeadSlots], v[kHeadSlots], gu[kHeadSlots], gv[kHeadSlots];
            float sum = 0.f;
#pragma unroll
            for (int s = 0; s < kHeadSlots; ++s) {
                const int j = lane + 32 * s;
                u[s] = v[s] = gu[s] = gv[s] = 0.f;
                if (j < slots) {
                    const SlotAt e = slot_at(j, a.d, a.rope);
                    const bool two = e.e1 < a.d;
                    u[s] = ld_elem<T>(x, e.e0);
                    gu[s] = ld_elem<T>(dy, e.e0);
                    if (two) {
                        v[s] = ld_elem<T>(x, e.e1);
                        gv[s] = ld_elem<T>(dy, e.e1);
                    }
                    if (e.turns) turn(gu[s], gv[s], cs[s]);
                    acc_u[s] = fmaf(gu[s], u[s] * r, acc_u[s]);
                    acc_v[s] = fmaf(gv[s], v[s] * r, acc_v[s]);
                    if (a.w[which]) {
                        gu[s] *= ld_elem<T>(a.w[which], e.e0);
                        if (two) gv[s] *= ld_elem<T>(a.w[which], e.e1);
                    }
                    sum = fmaf(gu[s], u[s], fmaf(gv[s], v[s], sum));
                }
            }
            const float f = warp_sum(sum) / float(a.d) * r * r * r;
#pragma unroll
            for (int s = 0; s < kHeadSlots; ++s) {
                const int j = lane + 32 * s;
                if (j < slots) {
                    const SlotAt e = slot_at(j, a.d, a.rope);
                    st_elem<T>(dx, e.e0, fmaf(-u[s], f, gu[s] * r));
                    if (e.e1 < a.d) st_elem<T>(dx, e.e1, fmaf(-v[s], f, gv[s] * r));
                }
            }
        }
    }
    if (a.ws == nullptr) return;
#pragma unroll
    for (int s = 0; s < kHeadSlots; ++s) {
        const int j = lane + 32 * s;
        if (j < slots) {
            const SlotAt e = slot_at(j, a.d, a.rope);
            part[warp][e.e0] = acc_u[s];
            if (e.e1 < a.d) part[warp][e.e1] = acc_v[s];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kHeadWarps * 32) {
        float sum = 0.f;
        for (int w = 0; w < kHeadWarps; ++w) sum += part[w][i];
        a.ws[int64_t(blockIdx.x) * a.d + i] = sum;
    }
}

// dw of q (blockIdx.y 0) and of k (1): the column sums of their partial rows, in
// a fixed order.  A column's rows are split over the 32 warps of a CTA; the
// partial rows can be much larger than their sum, so both levels carry the
// rounding error along (Neumaier's sum).
constexpr int kHeadSumWarps = 32;
struct CarriedSum {
    float s = 0.f, c = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v;
        c += fabsf(s) >= fabsf(v) ? (s - t) + v : (v - t) + s;
        s = t;
    }
};
template <typename T>
__global__ void __launch_bounds__(kHeadSumWarps * 32)
head_dw_kernel(const float* __restrict__ ws, int d, int nq, int nk, T* dwq, T* dwk) {
    pdl_wait();
    const int which = blockIdx.y;
    T* out = which ? dwk : dwq;
    if (out == nullptr) return;
    const float* rows = ws + (which ? int64_t(nq) * d : 0);
    const int n = which ? nk : nq;
    __shared__ float part[kHeadSumWarps][2][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    CarriedSum sum;
    if (col < d) {
#pragma unroll 4
        for (int p = warp; p < n; p += kHeadSumWarps) sum.add(rows[int64_t(p) * d + col]);
    }
    part[warp][0][lane] = sum.s;
    part[warp][1][lane] = sum.c;
    __syncthreads();
    if (warp == 0 && col < d) {
        CarriedSum tot;
#pragma unroll 8
        for (int w = 0; w < kHeadSumWarps; ++w) {
            tot.add(part[w][0][lane]);
            tot.add(part[w][1][lane]);
        }
        st_elem<T>(out, col, tot.s + tot.c);
    }
}

// ---------------------------------------------------------------------------
// cache rows: one row per warp
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_write_scalar_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ float stage[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.x[1].p ? int(blockIdx.y) : 1;
    const HeadView xv = a.x[1 + which];
    float* row = stage[warp];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = i / heads;
        const int h = int(i - t * heads);
        const int64_t slot = cache_slot(a.cache, __ldg(a.slots + t), a.err);
        if (slot < 0) continue;
        const T* x = reinterpret_cast<const T*>(xv.p) + t * xv.ts + h * xv.hs;
        for (int e = lane; e < a.d; e += 32) row[e] = ld_elem<T>(x, e);
        __syncwarp();
        quantise_row<T>(row, a.d, a.cache, which, slot, h, lane);
        __syncwarp();
    }
}

template <typename T>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_read_scalar_kernel(const __grid_constant__ HeadArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.y[0].p ? int(blockIdx.y) : 1;
    const HeadView yv = a.y[which];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = i / heads;
        const int h = int(i - t * heads);
        const int64_t slot = cache_slot(a.cache, __ldg(a.slots + t), a.err);
        if (slot < 0) continue;
        const CacheRow at = cache_row(a.cache, slot, h);
        const uint8_t* codes = a.cache.codes[which] + at.code;
        const float* scales = a.cache.scales[which] + at.scale;
        T* y = reinterpret_cast<T*>(yv.p) + t * yv.ts + h * yv.hs;
        for (int e = lane; e < a.d; e += 32) {
            float c;
            if (a.cache.kind == NRM_CACHE_E4M3) c = e4m3x2_values(codes[e]).x;
            else if (a.cache.kind == NRM_CACHE_INT8) c = float(int8_t(codes[e]));
            else c = float(int32_t(uint32_t(codes[e >> 1]) << (e & 1 ? 24 : 28)) >> 28);
            st_elem<T>(y, e, c * scales[e / a.cache.group]);
        }
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename T>
nrm_status head_fwd_scalar(const HeadArgs& a, bool norm, bool cache, const DevInfo& d, cudaStream_t s) {
    const void* fn = norm ? (cache ? (const void*)&head_fwd_scalar_kernel<T, true, true>
                                   : (const void*)&head_fwd_scalar_kernel<T, true, false>)
                          : (cache ? (const void*)&head_fwd_scalar_kernel<T, false, true>
                                   : (const void*)&head_fwd_scalar_kernel<T, false, false>);
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head forward kernel cannot be resident");
    const int64_t cap = int64_t(occ) * d.sms;
    const int heads = a.heads[0] + a.heads[1] + (cache ? a.heads[2] : 0);
    // few tokens: their heads are split over CTAs
    const int64_t gx = a.tokens < cap ? a.tokens : cap;
    int64_t gy = (heads + kHeadWarps - 1) / kHeadWarps;
    if (gy > (cap + gx - 1) / gx) gy = (cap + gx - 1) / gx;
    HeadArgs args = a;
    void* kargs[] = {&args};
    return cuda_status(cudaLaunchKernel(fn, dim3(unsigned(gx), unsigned(gy)), dim3(kHeadWarps * 32), kargs, 0, s),
                       "head forward launch");
}

template <typename T>
nrm_status head_fwd(const HeadArgs& a, bool norm, bool cache, bool vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    HeadArgs args = a;
    args.err = d->err;
    (void)vec;
    return head_fwd_scalar<T>(args, norm, cache, *d, s);
}

// Splits `ctas` between q and k by their rows.
inline int head_bwd_split(const HeadArgs& a, int ctas) {
    if (a.heads[1] == 0) return ctas;
    int nq = int(int64_t(ctas) * a.heads[0] / (a.heads[0] + a.heads[1]));
    if (nq < 1) nq = 1;
    return nq < ctas ? nq : ctas - 1;
}

template <typename T>
nrm_status head_bwd(const HeadArgs& a, bool vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) {
        for (void* dw : a.dw)
            if (dw)
                if (nrm_status st = cuda_status(cudaMemsetAsync(dw, 0, size_t(a.d) * sizeof(T), s), "dw zero fill");
                    st != NRM_OK)
                    return st;
        return NRM_OK;
    }
    (void)vec;
    const void* fn = (const void*)&head_bwd_scalar_kernel<T>;
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head backward kernel cannot be resident");
    int64_t ctas = int64_t(occ) * d->sms;
    if (ctas > head_bwd_max_partials(*d)) ctas = head_bwd_max_partials(*d);
    const int64_t most = a.tokens * (a.heads[1] ? 2 : 1);
    if (ctas > most) ctas = most;
    HeadArgs args = a;
    int nq = head_bwd_split(a, int(ctas));
    void* kargs[] = {&args, &nq};
    nrm_status st = cuda_status(cudaLaunchKernel(fn, dim3(unsigned(ctas)), dim3(kHeadWarps * 32), kargs, 0, s),
                                "head backward launch");
    if (st != NRM_OK || a.ws == nullptr) return st;
    const float* ws = a.ws;
    int dd = a.d, nk = int(ctas) - nq;
    T* dwq = reinterpret_cast<T*>(a.dw[0]);
    T* dwk = reinterpret_cast<T*>(a.dw[1]);
    void* sargs[] = {&ws, &dd, &nq, &nk, &dwq, &dwk};
    return launch_pdl((const void*)&head_dw_kernel<T>, dim3(unsigned(a.d + 31) / 32, 2), dim3(kHeadSumWarps * 32),
                      sargs, s);
}

template <typename T>
nrm_status cache_rows_scalar(const HeadArgs& a, const void* fn, bool both, const DevInfo& d, cudaStream_t s) {
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "cache kernel cannot be resident");
    const int64_t rows = a.tokens * a.heads[1];
    int64_t ctas = (rows + kHeadWarps - 1) / kHeadWarps;
    const int64_t cap = int64_t(occ) * d.sms;
    if (ctas > cap) ctas = cap;
    HeadArgs args = a;
    args.err = d.err;
    void* kargs[] = {&args};
    return cuda_status(cudaLaunchKernel(fn, dim3(unsigned(ctas), both ? 2 : 1), dim3(kHeadWarps * 32), kargs, 0, s),
                       "cache launch");
}

template <typename T>
nrm_status cache_write(const HeadArgs& a, bool vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    (void)vec;
    return cache_rows_scalar<T>(a, (const void*)&cache_write_scalar_kernel<T>, a.x[1].p && a.x[2].p, *d, s);
}

template <typename T>
nrm_status cache_read(const HeadArgs& a, bool vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    (void)vec;
    return cache_rows_scalar<T>(a, (const void*)&cache_read_scalar_kernel<T>, a.y[0].p && a.y[1].p, *d, s);
}

}  // namespace nrm

// Instantiates the operators for one storage dtype.
#define NRM_INSTANTIATE_HEADS(T)                                                                       \
    namespace nrm {                                                                                    \
    template nrm_status head_fwd<T>(const HeadArgs&, bool, bool, bool, cudaStream_t);                  \
    template nrm_status head_bwd<T>(const HeadArgs&, bool, cudaStream_t);                              \
    template nrm_status cache_write<T>(const HeadArgs&, bool, cudaStream_t);                           \
    template nrm_status cache_read<T>(const HeadArgs&, bool, cudaStream_t);                            \
    }
