// heads.cuh -- kernels on attention heads: RMSNorm of each head with the
// position rotation in the same pass, forward and backward, the rotation alone,
// and the quantised key/value cache (written from given rows, from the key the
// norm and rotation just made, and read back).
//
// One row is one token's head of d <= 256 elements.  In the vector kernels a row
// belongs to the 4 to 32 lanes that hold one pair of vectors each: the two whose
// elements turn together, so a rotation needs no exchange between lanes.  A warp
// takes a token's heads a few rows at a time with the token's cosines and sines
// in registers; the lanes of a warp share the work of making them.  Layouts that
// fit no vector take a row per warp, element by element.
#pragma once

#include <type_traits>

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
// angle of a far position is as exact as that of a near one.  The float's 24
// bits times 2^66 / (2 pi), shifted by its exponent; whole turns fall off the top.
__device__ __forceinline__ uint64_t turn_step(float inv_freq) {
    constexpr uint64_t k = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi))
    const uint32_t bits = __float_as_uint(inv_freq);
    const int e = int(bits >> 23 & 0xffu);
    const uint64_t m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
    const uint64_t lo = m * k, hi = __umul64hi(m, k);
    const int s = 152 - max(e, 1);  // inv_freq == m * 2^(e - 150)
    uint64_t f = 0;
    if (s > 63) f = s < 128 ? hi >> (s - 64) : 0;
    else if (s > 0) f = lo >> s | hi << (64 - s);
    else if (s > -64) f = lo << -s;
    return bits >> 31 ? 0 - f : f;
}

__device__ __forceinline__ int pair_axis(const RopeDev& r, int p) {
    return int(r.axis[p >> 4] >> ((p & 15) * 2)) & 3;
}

// cos and sin of a pair that turns by `step` per position, at position pos.  The
// top 32 bits of the phase, read as signed, are the angle in 2^-31 half turns.
__device__ __forceinline__ float2 pair_turn(const RopeDev& r, uint64_t step, int64_t pos) {
    const uint64_t phase = uint64_t(pos) * step;
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
// magnitude (compared as integers, so a NaN is the largest of all).  Groups
// above 2^100 are divided by 2^32 and groups below 2^-36 multiplied by 2^64
// (exactly, where it matters), so that products stay finite and residuals
// representable.
struct GroupQ {
    float scale;
    float m, r;  // the scaled largest magnitude and its reciprocal; both 0 where every code is 0
    float q;     // the form's largest number, scaled like m
};
__device__ __forceinline__ GroupQ group_q(uint32_t m_bits, int kind) {
    GroupQ g{0.f, 0.f, 0.f, 0.f};
    const float m = __uint_as_float(m_bits);
    if (m_bits >= 0x7f800000u) {  // a NaN or an infinity: the group reads back as NaN
        g.scale = __uint_as_float(0x7fffffffu);
    } else if (m >= 0x1p-100f) {  // else nothing but (almost) zeros
        const float q = cache_qmax(kind);
        const float p = m > 0x1p100f ? 0x1p-32f : (m < 0x1p-36f ? 0x1p64f : 1.f);
        g.scale = __fdiv_rn(m, q);
        g.m = m * p;
        g.r = __frcp_rn(g.m);
        g.q = q * p;
    }
    return g;
}
// x*q/m, such that the code nearest to it is the one nearest to the real
// quotient, ties seen as ties: q0 = (x*q)*r is off by under 2 units in the last
// place, and one step with its residual (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990) mends it.
// 16-bit x: x*q is exact.  A quotient that is half way between codes has so few
// bits that the residual and the sum come out exact; any other is further from
// half way than the 2^-23 by which the result may be off (an 11-bit x and m and
// an 8-bit border keep at least 2^-20).
// float32 x: the result is rounded to odd, by the sign of a second residual
// (with what the rounded product lost): a quotient that is not exact then never
// lands on an even number, and so never half way between codes.
template <typename T>
__device__ __forceinline__ float group_scaled(float x, const GroupQ& g) {
    const float n = __fmul_rn(x, g.q);
    const float u0 = __fmul_rn(n, g.r);
    if constexpr (sizeof(T) == 2) {
        const float u = fmaf(fmaf(-u0, g.m, n), g.r, u0);
        return g.r == 0.f ? 0.f : u;  // (a NaN is no code)
    } else {
        const float lost = fmaf(x, g.q, -n);  // n + lost == x*q
        const float u = fmaf(fmaf(-u0, g.m, n) + lost, g.r, u0);
        const float left = fmaf(-u, g.m, n) + lost;
        const int bits = __float_as_int(u);
        const bool off = left != 0.f && (bits & 1) == 0 && fabsf(u) >= 0x1p-24f;
        const float odd = off ? __int_as_float(bits + ((left > 0.f) == (u > 0.f) ? 1 : -1)) : u;
        return g.r == 0.f ? 0.f : odd;
    }
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

__device__ __forceinline__ int64_t row_div(int64_t n, const RowDiv& d) {
    return d.small ? int64_t(fast_div(uint32_t(n), FastDiv{uint32_t(d.d), d.m})) : n / d.d;
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
    const int64_t page = row_div(slot, c.page), at = slot - page * c.page.d;
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
// vectors of VE elements (16 or 8 bytes)
// ---------------------------------------------------------------------------
template <int BYTES> struct RawBits;
template <> struct RawBits<16> { using type = uint4; };
template <> struct RawBits<8> { using type = uint2; };
template <typename T, int VE> using Raw = typename RawBits<VE * int(sizeof(T))>::type;

// Loads of rows that this kernel may write in place: not through the read-only
// path, and not kept in L1.
__device__ __forceinline__ void ld_row(const void* p, uint4& r) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_row(const void* p, uint2& r) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
}
__device__ __forceinline__ void st_row(void* p, uint4 v) { st_v4(p, v); }
__device__ __forceinline__ void st_row(void* p, uint2 v) {
    asm volatile("st.global.v2.u32 [%0], {%1,%2};" :: "l"(p), "r"(v.x), "r"(v.y) : "memory");
}

template <typename T, int VE>
__device__ __forceinline__ void raw_unpack(const Raw<T, VE>& r, float (&v)[VE]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VE * int(sizeof(T)) / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(w[i]);
        } else {
            const float2 f = cvt2<T>(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> raw_pack(const float (&v)[VE]) {
    Raw<T, VE> r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VE * int(sizeof(T)) / 4; ++i) {
        if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(v[i]);
        else w[i] = pack2<T>(make_float2(v[2 * i], v[2 * i + 1]));
    }
    return r;
}

// The largest magnitude's bits.
template <int VE>
__device__ __forceinline__ uint32_t abs_max_bits(const float (&v)[VE]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VE; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Codes of VE consecutive elements, stored at element e of the row.
template <typename T, int VE>
__device__ __forceinline__ void store_codes(uint8_t* row, int e, const float (&v)[VE], const GroupQ& q, int kind) {
    float u[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) u[i] = group_scaled<T>(v[i], q);
    if (kind == NRM_CACHE_INT4) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) w |= (uint32_t(__float2int_rn(u[i])) & 0xfu) << (4 * i);
        uint8_t* at = row + (e >> 1);
        if constexpr (VE == 8) *reinterpret_cast<uint32_t*>(at) = w;
        else if constexpr (VE == 4) *reinterpret_cast<uint16_t*>(at) = uint16_t(w);
        else *at = uint8_t(w);
        return;
    }
    uint32_t w[(VE + 3) / 4] = {};
    if (kind == NRM_CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < VE; i += 2) w[i / 4] |= e4m3x2(u[i], u[i + 1]) << (8 * (i % 4));
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) w[i / 4] |= (uint32_t(__float2int_rn(u[i])) & 0xffu) << (8 * (i % 4));
    }
    uint8_t* at = row + e;
    if constexpr (VE == 8) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    else if constexpr (VE == 4) *reinterpret_cast<uint32_t*>(at) = w[0];
    else *reinterpret_cast<uint16_t*>(at) = uint16_t(w[0]);
}

// A lane's place in the vector kernels: which row of the warp's, which pair of
// vectors of that row, and where they lie.  2^lg lanes hold a row.
template <int VE>
struct LaneAt {
    int sub, j;      // row of the warp's 32 >> lg rows, pair of vectors of the row
    int b0, b1;      // first elements of the two vectors
    bool on, turns;  // holds elements; they turn
    __device__ __forceinline__ LaneAt(int lane, int lg, int d, const RopeDev& r) {
        sub = lane >> lg;
        j = lane & ((1 << lg) - 1);
        on = 2 * VE * j < d;
        turns = 2 * VE * j < r.rot;
        const bool half = turns && !r.adjacent;
        b0 = half ? VE * j : 2 * VE * j;
        b1 = half ? VE * j + (r.rot >> 1) : b0 + VE;
    }
};

// The angles of a warp's tokens: lane l makes those of pairs l, l + 32, ..., and
// every lane then takes the VE pairs of its own vectors through shared memory.
struct WarpTurns {
    uint64_t step[kHeadMaxPairs / 32];
    int axis;
    __device__ __forceinline__ WarpTurns(const RopeDev& r, int lane) : axis(0) {
#pragma unroll
        for (int s = 0; s < kHeadMaxPairs / 32; ++s) {
            const int p = lane + 32 * s;
            step[s] = 0;
            if (2 * p < r.rot) {
                step[s] = turn_step(__ldg(r.inv_freq + p));
                axis |= pair_axis(r, p) << (2 * s);
            }
        }
    }
    // cos[p], sin[p] of token t, for every pair.  Called by the whole warp.
    __device__ __forceinline__ void make(const RopeDev& r, int lane, int64_t t, float* cos, float* sin) const {
        __syncwarp();
#pragma unroll
        for (int s = 0; s < kHeadMaxPairs / 32; ++s) {
            const int p = lane + 32 * s;
            if (2 * p < r.rot) {
                const int64_t pos = __ldg(r.pos + (axis >> (2 * s) & 3) * r.pos_stride + t);
                const float2 cs = pair_turn(r, step[s], pos);
                cos[p] = cs.x;
                sin[p] = cs.y;
            }
        }
        __syncwarp();
    }
};

// Turns a lane's two vectors by its VE pairs' angles.
template <int VE>
__device__ __forceinline__ void turn_vecs(float (&u)[VE], float (&v)[VE], const float (&c)[VE], const float (&s)[VE],
                                          bool adjacent) {
    if (!adjacent) {
#pragma unroll
        for (int i = 0; i < VE; ++i) turn(u[i], v[i], make_float2(c[i], s[i]));
    } else {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) turn(u[2 * i], u[2 * i + 1], make_float2(c[i], s[i]));
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            turn(v[2 * i], v[2 * i + 1], make_float2(c[VE / 2 + i], s[VE / 2 + i]));
    }
}

// Sum over the 2^lg lanes of a row; every lane of it gets the same bits.
__device__ __forceinline__ float row_sum(float v, int lg) {
    for (int o = 1 << lg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// ---------------------------------------------------------------------------
// forward on vectors: norm, rotation, cache
// ---------------------------------------------------------------------------
constexpr int kHeadRows = 2;  // rows of a lane in flight

// A warp takes (token, chunk) units; chunk c of 2^lchunk takes the token's row
// steps c, c + 2^lchunk, ...  (a step: kHeadRows * (32 >> lg) rows).
template <typename T, int VE, bool NORM, bool CACHE>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_fwd_vec_kernel(const __grid_constant__ HeadArgs a, int lg, int lchunk) {
    __shared__ __align__(16) float s_cos[kHeadWarps][kHeadMaxPairs], s_sin[kHeadWarps][kHeadMaxPairs];
    __shared__ uint32_t s_max[CACHE ? kHeadWarps : 1][CACHE ? 64 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const LaneAt<VE> at(lane, lg, a.d, a.rope);
    const WarpTurns turns(a.rope, lane);
    const int rows = 32 >> lg;
    const int heads = a.heads[0] + a.heads[1] + (CACHE ? a.heads[2] : 0);
    const int64_t units = a.tokens << lchunk;
    const float inv_d = 1.f / float(a.d);
    for (int64_t un = int64_t(blockIdx.x) * kHeadWarps + warp; un < units; un += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = un >> lchunk;
        int h0 = (int(un) & ((1 << lchunk) - 1)) * (rows * kHeadRows);
        const int64_t slot = CACHE ? cache_slot(a.cache, __ldg(a.slots + t), a.err) : -1;
        turns.make(a.rope, lane, t, s_cos[warp], s_sin[warp]);
        float c[VE], s[VE];
        if (at.turns) {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                c[i] = s_cos[warp][VE * at.j + i];
                s[i] = s_sin[warp][VE * at.j + i];
            }
        }
        for (; h0 < heads; h0 += (rows * kHeadRows) << lchunk) {
            Raw<T, VE> x0[kHeadRows], x1[kHeadRows];
            int which[kHeadRows], hd[kHeadRows];
#pragma unroll
            for (int k = 0; k < kHeadRows; ++k) {
                const int hh = h0 + k * rows + at.sub;
                which[k] = hh < a.heads[0] ? 0 : (hh < a.heads[0] + a.heads[1] ? 1 : 2);
                hd[k] = hh - (which[k] > 0 ? a.heads[0] : 0) - (which[k] > 1 ? a.heads[1] : 0);
                x0[k] = x1[k] = Raw<T, VE>{};
                if (hh >= heads) which[k] = 3;  // no row
                else if (at.on) {
                    const HeadView v = a.x[which[k]];
                    const T* x = reinterpret_cast<const T*>(v.p) + t * v.ts + hd[k] * v.hs;
                    ld_row(x + at.b0, x0[k]);
                    ld_row(x + at.b1, x1[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < kHeadRows; ++k) {
                float u[VE], v[VE];
                raw_unpack<T, VE>(x0[k], u);
                raw_unpack<T, VE>(x1[k], v);
                if (NORM) {
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < VE; ++i) sum = fmaf(u[i], u[i], fmaf(v[i], v[i], sum));
                    const float r = rsqrtf(fmaf(row_sum(sum, lg), inv_d, a.eps));
                    if (which[k] < 2) {
                        if (at.j == 0 && a.rstd[which[k]]) a.rstd[which[k]][t * a.heads[which[k]] + hd[k]] = r;
#pragma unroll
                        for (int i = 0; i < VE; ++i) {
                            u[i] = __fmul_rn(u[i], r);
                            v[i] = __fmul_rn(v[i], r);
                        }
                        const T* w = reinterpret_cast<const T*>(a.w[which[k]]);
                        if (w && at.on) {
                            float w0[VE], w1[VE];
                            raw_unpack<T, VE>(__ldg(reinterpret_cast<const Raw<T, VE>*>(w + at.b0)), w0);
                            raw_unpack<T, VE>(__ldg(reinterpret_cast<const Raw<T, VE>*>(w + at.b1)), w1);
#pragma unroll
                            for (int i = 0; i < VE; ++i) {
                                u[i] = __fmul_rn(u[i], w0[i]);
                                v[i] = __fmul_rn(v[i], w1[i]);
                            }
                        }
                    }
                }
                if (which[k] < 2) {
                    if (at.turns) turn_vecs<VE>(u, v, c, s, a.rope.adjacent);
                    x0[k] = raw_pack<T, VE>(u);
                    x1[k] = raw_pack<T, VE>(v);
                    const HeadView y = a.y[which[k]];
                    if (at.on && y.p) {
                        T* o = reinterpret_cast<T*>(y.p) + t * y.ts + hd[k] * y.hs;
                        st_row(o + at.b0, x0[k]);
                        st_row(o + at.b1, x1[k]);
                    }
                }
                if constexpr (CACHE) {
                    // uniform: the warp's rows of this step hold a key or a value, and the token has a slot
                    if (slot < 0 || h0 + (k + 1) * rows <= a.heads[0]) continue;
                    // the cache stores the key in the activations' type: what a separate write would read
                    raw_unpack<T, VE>(x0[k], u);
                    raw_unpack<T, VE>(x1[k], v);
                    uint32_t m0 = at.on ? abs_max_bits<VE>(u) : 0, m1 = at.on ? abs_max_bits<VE>(v) : 0;
                    const int group = a.cache.group;
                    if (group == a.d) {
                        m0 = max(m0, m1);
                        for (int o = 1 << lg >> 1; o > 0; o >>= 1) m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                        m1 = m0;
                    } else {
                        // groups of whole vectors, which other lanes may hold: through shared memory
                        uint32_t* sm = s_max[warp] + at.sub * (a.d / VE);
                        if (at.on) {
                            sm[at.b0 / VE] = m0;
                            sm[at.b1 / VE] = m1;
                        }
                        __syncwarp();
                        if (at.on) {
                            const int n = group / VE, g0 = at.b0 / group * n, g1 = at.b1 / group * n;
                            for (int i = 0; i < n; ++i) {
                                m0 = max(m0, sm[g0 + i]);
                                m1 = max(m1, sm[g1 + i]);
                            }
                        }
                        __syncwarp();
                    }
                    if (at.on && (which[k] == 1 || which[k] == 2)) {
                        const CacheRow cr = cache_row(a.cache, slot, hd[k]);
                        const GroupQ q0 = group_q(m0, a.cache.kind), q1 = group_q(m1, a.cache.kind);
                        float* scales = a.cache.scales[which[k] - 1] + cr.scale;
                        if (at.b0 % group == 0) scales[at.b0 / group] = q0.scale;
                        if (at.b1 % group == 0) scales[at.b1 / group] = q1.scale;
                        uint8_t* codes = a.cache.codes[which[k] - 1] + cr.code;
                        store_codes<T, VE>(codes, at.b0, u, q0, a.cache.kind);
                        store_codes<T, VE>(codes, at.b1, v, q1, a.cache.kind);
                    }
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// backward on vectors
// ---------------------------------------------------------------------------
template <typename T, int VE>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_bwd_vec_kernel(const __grid_constant__ HeadArgs a, int lg, int lchunk, int nq) {
    __shared__ __align__(16) float s_cos[kHeadWarps][kHeadMaxPairs], s_sin[kHeadWarps][kHeadMaxPairs];
    __shared__ float part[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = int(blockIdx.x) < nq ? 0 : 1;
    const int cta = int(blockIdx.x) - (which ? nq : 0);
    const int ctas = which ? int(gridDim.x) - nq : nq;
    const LaneAt<VE> at(lane, lg, a.d, a.rope);
    const WarpTurns turns(a.rope, lane);
    const int rows = 32 >> lg;
    const int heads = a.heads[which];
    const int64_t units = a.tokens << lchunk;
    const float inv_d = 1.f / float(a.d);
    const HeadView xv = a.x[which], gv = a.dy[which], dv = a.y[which];
    float w0[VE], w1[VE], acc0[VE], acc1[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        w0[i] = w1[i] = 1.f;
        acc0[i] = acc1[i] = 0.f;
    }
    if (at.on && a.w[which]) {
        const T* w = reinterpret_cast<const T*>(a.w[which]);
        raw_unpack<T, VE>(__ldg(reinterpret_cast<const Raw<T, VE>*>(w + at.b0)), w0);
        raw_unpack<T, VE>(__ldg(reinterpret_cast<const Raw<T, VE>*>(w + at.b1)), w1);
    }
    for (int64_t un = int64_t(cta) * kHeadWarps + warp; un < units; un += int64_t(ctas) * kHeadWarps) {
        const int64_t t = un >> lchunk;
        turns.make(a.rope, lane, t, s_cos[warp], s_sin[warp]);
        float c[VE], s[VE];
        if (at.turns) {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                c[i] = s_cos[warp][VE * at.j + i];
                s[i] = s_sin[warp][VE * at.j + i];
            }
        }
        for (int h = (int(un) & ((1 << lchunk) - 1)) * rows; h < heads; h += rows << lchunk) {
            const int hd = h + at.sub;
            const bool row = hd < heads, on = row && at.on;
            Raw<T, VE> x0{}, x1{}, y0{}, y1{};
            float r = 0.f;
            if (on) {
                const T* g = reinterpret_cast<const T*>(gv.p) + t * gv.ts + hd * gv.hs;
                const T* x = reinterpret_cast<const T*>(xv.p) + t * xv.ts + hd * xv.hs;
                ld_row(g + at.b0, y0);
                ld_row(g + at.b1, y1);
                ld_row(x + at.b0, x0);
                ld_row(x + at.b1, x1);
                r = __ldg(a.rstd[which] + t * heads + hd);
            }
            float u[VE], v[VE], gu[VE], gw[VE];
            raw_unpack<T, VE>(x0, u);
            raw_unpack<T, VE>(x1, v);
            raw_unpack<T, VE>(y0, gu);
            raw_unpack<T, VE>(y1, gw);
            if (at.turns) turn_vecs<VE>(gu, gw, c, s, a.rope.adjacent);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                acc0[i] = fmaf(gu[i], u[i] * r, acc0[i]);
                acc1[i] = fmaf(gw[i], v[i] * r, acc1[i]);
                gu[i] *= w0[i];
                gw[i] *= w1[i];
                sum = fmaf(gu[i], u[i], fmaf(gw[i], v[i], sum));
            }
            const float f = row_sum(sum, lg) * inv_d * r * r * r;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                gu[i] = fmaf(-u[i], f, gu[i] * r);
                gw[i] = fmaf(-v[i], f, gw[i] * r);
            }
            if (on) {
                T* o = reinterpret_cast<T*>(dv.p) + t * dv.ts + hd * dv.hs;
                st_row(o + at.b0, raw_pack<T, VE>(gu));
                st_row(o + at.b1, raw_pack<T, VE>(gw));
            }
        }
    }
    if (a.ws == nullptr) return;
    // the warp's rows, then the CTA's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        for (int o = 1 << lg; o < 32; o <<= 1) {
            acc0[i] += __shfl_xor_sync(0xffffffffu, acc0[i], o);
            acc1[i] += __shfl_xor_sync(0xffffffffu, acc1[i], o);
        }
        if (at.sub == 0 && at.on) {
            part[warp][at.b0 + i] = acc0[i];
            part[warp][at.b1 + i] = acc1[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kHeadWarps * 32) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kHeadWarps; ++w) sum += part[w][i];
        a.ws[int64_t(blockIdx.x) * a.d + i] = sum;
    }
}

// ---------------------------------------------------------------------------
// cache rows on vectors: 2^lg lanes a row, NV vectors of a row to a lane
// ---------------------------------------------------------------------------
constexpr int kCacheRows = 4;  // rows of a lane in flight

template <typename T, int VE, int NV>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_write_vec_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads, int lg) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> lg, j = lane & ((1 << lg) - 1), rows = 32 >> lg;
    const int which = a.x[1].p ? int(blockIdx.y) : 1;
    const HeadView xv = a.x[1 + which];
    const int64_t n = a.tokens * by_heads.d;
    const int group = a.cache.group, kind = a.cache.kind;
    const int gv = group / VE;                       // vectors of a group
    const bool whole = group == a.d, pow2 = (gv & (gv - 1)) == 0;
    const int64_t step = int64_t(rows) * kCacheRows;
    for (int64_t base = (int64_t(blockIdx.x) * kHeadWarps + warp) * step; base < n;
         base += int64_t(gridDim.x) * kHeadWarps * step) {
        Raw<T, VE> raw[kCacheRows][NV];
        int64_t slot[kCacheRows];
        int hd[kCacheRows];
#pragma unroll
        for (int k = 0; k < kCacheRows; ++k) {
            const int64_t i = base + k * rows + sub;
            slot[k] = -1;
            hd[k] = 0;
            if (i < n) {
                const int64_t t = row_div(i, by_heads);
                hd[k] = int(i - t * by_heads.d);
                slot[k] = __ldg(a.slots + t);
                const T* x = reinterpret_cast<const T*>(xv.p) + t * xv.ts + hd[k] * xv.hs;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    raw[k][v] = Raw<T, VE>{};
                    const int e = (j + 32 * v) * VE;
                    if (e < a.d) ld_row(x + e, raw[k][v]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kCacheRows; ++k) {
            slot[k] = cache_slot(a.cache, slot[k], a.err);
            float x[NV][VE];
            uint32_t m[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                raw_unpack<T, VE>(raw[k][v], x[v]);
                m[v] = (j + 32 * v) * VE < a.d && slot[k] >= 0 ? abs_max_bits<VE>(x[v]) : 0;
            }
            if (whole) {
                if constexpr (NV == 2) m[0] = max(m[0], m[1]);
                for (int o = 1 << lg >> 1; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
                if constexpr (NV == 2) m[1] = m[0];
            } else if (pow2) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    for (int o = gv >> 1; o > 0; o >>= 1) m[v] = max(m[v], __shfl_xor_sync(0xffffffffu, m[v], o));
            } else {  // NV == 1
                const int first = (sub << lg) + j / gv * gv;
                uint32_t all = 0;
                for (int i = 0; i < gv; ++i) all = max(all, __shfl_sync(0xffffffffu, m[0], (first + i) & 31));
                m[0] = all;
            }
            if (slot[k] < 0) continue;
            const CacheRow cr = cache_row(a.cache, slot[k], hd[k]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = (j + 32 * v) * VE;
                if (e >= a.d) continue;
                const GroupQ q = group_q(m[v], kind);
                if (e % group == 0) a.cache.scales[which][cr.scale + e / group] = q.scale;
                store_codes<T, VE>(a.cache.codes[which] + cr.code, e, x[v], q, kind);
            }
        }
    }
}

// The VE codes at element e of a row, as they lie in memory.
template <int VE>
__device__ __forceinline__ uint2 load_codes(const uint8_t* row, int e, int kind) {
    uint2 w{0u, 0u};
    if (kind == NRM_CACHE_INT4) {
        const uint8_t* at = row + (e >> 1);
        if constexpr (VE == 8) w.x = __ldg(reinterpret_cast<const uint32_t*>(at));
        else if constexpr (VE == 4) w.x = __ldg(reinterpret_cast<const uint16_t*>(at));
        else w.x = __ldg(at);
    } else {
        const uint8_t* at = row + e;
        if constexpr (VE == 8) w = __ldg(reinterpret_cast<const uint2*>(at));
        else if constexpr (VE == 4) w.x = __ldg(reinterpret_cast<const uint32_t*>(at));
        else w.x = __ldg(reinterpret_cast<const uint16_t*>(at));
    }
    return w;
}
// The numbers they are.  A whole number goes to float32 by way of its bits: with
// its sign bit flipped it is the low end of the mantissa of 2^23 + code + half.
template <int VE>
__device__ __forceinline__ void code_values(uint2 w, int kind, float (&v)[VE]) {
    if (kind == NRM_CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
            const float2 f = e4m3x2_values((i < 4 ? w.x : w.y) >> (8 * (i % 4)));
            v[i] = f.x;
            v[i + 1] = f.y;
        }
    } else if (kind == NRM_CACHE_INT8) {
        const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < VE; ++i)
            v[i] = __uint_as_float(__byte_perm(i < 4 ? x : y, 0x4B000000u, 0x7650 + i % 4)) - 8388736.f;
    } else {
        const uint32_t x = w.x ^ 0x88888888u;
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = __uint_as_float((x >> (4 * i) & 0xfu) | 0x4B000000u) - 8388616.f;
    }
}

template <typename T, int VE, int NV>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_read_vec_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads, int lg) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane >> lg, j = lane & ((1 << lg) - 1), rows = 32 >> lg;
    const int which = a.y[0].p ? int(blockIdx.y) : 1;
    const HeadView yv = a.y[which];
    const int64_t n = a.tokens * by_heads.d;
    const int group = a.cache.group, kind = a.cache.kind;
    const int64_t step = int64_t(rows) * kCacheRows;
    for (int64_t base = (int64_t(blockIdx.x) * kHeadWarps + warp) * step; base < n;
         base += int64_t(gridDim.x) * kHeadWarps * step) {
        int64_t tok[kCacheRows], slot[kCacheRows];
        int hd[kCacheRows];
#pragma unroll
        for (int k = 0; k < kCacheRows; ++k) {
            const int64_t i = base + k * rows + sub;
            slot[k] = -1;
            if (i < n) {
                tok[k] = row_div(i, by_heads);
                hd[k] = int(i - tok[k] * by_heads.d);
                slot[k] = __ldg(a.slots + tok[k]);
            }
        }
        uint2 w[kCacheRows][NV];
        float sc[kCacheRows][NV];
#pragma unroll
        for (int k = 0; k < kCacheRows; ++k) {
            slot[k] = cache_slot(a.cache, slot[k], a.err);
            if (slot[k] < 0) continue;
            const CacheRow cr = cache_row(a.cache, slot[k], hd[k]);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = (j + 32 * v) * VE;
                if (e >= a.d) continue;
                w[k][v] = load_codes<VE>(a.cache.codes[which] + cr.code, e, kind);
                sc[k][v] = __ldg(a.cache.scales[which] + cr.scale + e / group);
            }
        }
#pragma unroll
        for (int k = 0; k < kCacheRows; ++k) {
            if (slot[k] < 0) continue;
            T* y = reinterpret_cast<T*>(yv.p) + tok[k] * yv.ts + hd[k] * yv.hs;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int e = (j + 32 * v) * VE;
                if (e >= a.d) continue;
                float x[VE];
                code_values<VE>(w[k][v], kind, x);
#pragma unroll
                for (int i = 0; i < VE; ++i) x[i] *= sc[k][v];
                st_row(y + e, raw_pack<T, VE>(x));
            }
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
            if (2 * (lane + 32 * s) < a.rope.rot)
                cs[s] = pair_turn(a.rope, turn_step(__ldg(a.rope.inv_freq + lane + 32 * s)),
                                  __ldg(a.rope.pos + pair_axis(a.rope, lane + 32 * s) * a.rope.pos_stride + t));
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
            if (2 * (lane + 32 * s) < a.rope.rot)
                cs[s] = pair_turn(a.rope, turn_step(__ldg(a.rope.inv_freq + lane + 32 * s)),
                                  __ldg(a.rope.pos + pair_axis(a.rope, lane + 32 * s) * a.rope.pos_stride + t));
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
cache_write_scalar_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads, int) {
    __shared__ float stage[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.x[1].p ? int(blockIdx.y) : 1;
    const HeadView xv = a.x[1 + which];
    float* row = stage[warp];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = row_div(i, by_heads);
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
cache_read_scalar_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads, int) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.y[0].p ? int(blockIdx.y) : 1;
    const HeadView yv = a.y[which];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = row_div(i, by_heads);
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

// Lanes of a row that holds `n` vectors (or pairs of them): 2^lg >= n, at most 32.
inline int row_lanes_log2(int n) {
    int lg = 0;
    while ((1 << lg) < n && lg < 5) ++lg;
    return lg;
}

// Chunks (as a power of two) that a token's `steps` row steps are split into:
// one while tokens alone give every SM 16 warps, else as many as are needed.
inline int head_chunks_log2(int64_t tokens, int steps, const DevInfo& d) {
    int lc = 0;
    while ((1 << lc) < steps && (tokens << lc) < int64_t(16) * d.sms) ++lc;
    return lc;
}

template <typename T, int VE>
nrm_status head_fwd_vec(const HeadArgs& a, bool norm, bool cache, const DevInfo& d, cudaStream_t s) {
    const void* fn = norm ? (cache ? (const void*)&head_fwd_vec_kernel<T, VE, true, true>
                                   : (const void*)&head_fwd_vec_kernel<T, VE, true, false>)
                          : (cache ? (const void*)&head_fwd_vec_kernel<T, VE, false, true>
                                   : (const void*)&head_fwd_vec_kernel<T, VE, false, false>);
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head forward kernel cannot be resident");
    int lg = row_lanes_log2(a.d / (2 * VE));
    const int heads = a.heads[0] + a.heads[1] + (cache ? a.heads[2] : 0), per = (32 >> lg) * kHeadRows;
    int lc = head_chunks_log2(a.tokens, (heads + per - 1) / per, d);
    int64_t ctas = ((a.tokens << lc) + kHeadWarps - 1) / kHeadWarps;
    if (ctas > int64_t(occ) * d.sms) ctas = int64_t(occ) * d.sms;
    HeadArgs args = a;
    void* kargs[] = {&args, &lg, &lc};
    return cuda_status(cudaLaunchKernel(fn, dim3(unsigned(ctas)), dim3(kHeadWarps * 32), kargs, 0, s),
                       "head forward launch");
}
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
nrm_status head_fwd(const HeadArgs& a, bool norm, bool cache, int vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    HeadArgs args = a;
    args.err = d->err;
    if (vec == 16) return head_fwd_vec<T, 16 / int(sizeof(T))>(args, norm, cache, *d, s);
    if (vec == 8) return head_fwd_vec<T, 8 / int(sizeof(T))>(args, norm, cache, *d, s);
    return head_fwd_scalar<T>(args, norm, cache, *d, s);
}

template <typename T>
nrm_status head_bwd(const HeadArgs& a, int vec, cudaStream_t s) {
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
    const void* fn = vec == 16  ? (const void*)&head_bwd_vec_kernel<T, 16 / int(sizeof(T))>
                     : vec == 8 ? (const void*)&head_bwd_vec_kernel<T, 8 / int(sizeof(T))>
                                : (const void*)&head_bwd_scalar_kernel<T>;
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head backward kernel cannot be resident");
    int lg = vec ? row_lanes_log2(a.d * int(sizeof(T)) / (2 * vec)) : 5;
    const int per = vec ? 32 >> lg : kHeadWarps;
    const int steps[2] = {(a.heads[0] + per - 1) / per, (a.heads[1] + per - 1) / per};
    int lc = vec ? head_chunks_log2(a.tokens, steps[0] > steps[1] ? steps[0] : steps[1], *d) : 0;
    // CTAs go to q and k by what they cost: a token's row steps, and one more for its angles
    int64_t cap = int64_t(occ) * d->sms;
    if (cap > head_bwd_max_partials(*d)) cap = head_bwd_max_partials(*d);
    const int64_t units = vec ? ((a.tokens << lc) + kHeadWarps - 1) / kHeadWarps : a.tokens;
    int64_t cq = cap, ck = 0;
    if (a.heads[1]) {
        ck = cap * (steps[1] + 1) / (steps[0] + steps[1] + 2);
        if (ck < 1) ck = 1;
        cq = cap - ck;
    }
    int nq = int(cq < units ? cq : units), nk = int(ck < units ? ck : units);
    HeadArgs args = a;
    void* kargs_vec[] = {&args, &lg, &lc, &nq};
    void* kargs[] = {&args, &nq};
    nrm_status st = cuda_status(cudaLaunchKernel(fn, dim3(unsigned(nq + nk)), dim3(kHeadWarps * 32),
                                                 vec ? kargs_vec : kargs, 0, s),
                                "head backward launch");
    if (st != NRM_OK || a.ws == nullptr) return st;
    const float* ws = a.ws;
    int dd = a.d;
    T* dwq = reinterpret_cast<T*>(a.dw[0]);
    T* dwk = reinterpret_cast<T*>(a.dw[1]);
    void* sargs[] = {&ws, &dd, &nq, &nk, &dwq, &dwk};
    return launch_pdl((const void*)&head_dw_kernel<T>, dim3(unsigned(a.d + 31) / 32, 2), dim3(kHeadSumWarps * 32),
                      sargs, s);
}

// Launches a cache kernel over tokens * heads rows, `both`: of keys and of values.
inline nrm_status cache_launch(const HeadArgs& a, const void* fn, int rows_per_warp, int lg, bool both,
                               const DevInfo& d, cudaStream_t s) {
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "cache kernel cannot be resident");
    const int64_t rows = a.tokens * a.heads[1], per = int64_t(rows_per_warp) * kHeadWarps;
    int64_t ctas = (rows + per - 1) / per;
    const int64_t cap = int64_t(occ) * d.sms;
    if (ctas > cap) ctas = cap;
    HeadArgs args = a;
    args.err = d.err;
    RowDiv by_heads = make_row_div(a.heads[1], rows);
    void* kargs[] = {&args, &by_heads, &lg};
    return cuda_status(cudaLaunchKernel(fn, dim3(unsigned(ctas), both ? 2 : 1), dim3(kHeadWarps * 32), kargs, 0, s),
                       "cache launch");
}

// The vector kernel of a row of d elements: one vector to a lane, or two where a
// warp cannot hold the row else.  Two need groups that stay within 32 vectors.
template <typename T, typename F>
nrm_status cache_rows(const HeadArgs& a, int vec, F&& launch) {
    const int ve = vec / int(sizeof(T)), gv = ve ? a.cache.group / ve : 0;
    if (vec == 16 && a.d <= 32 * ve) return launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
    if (vec == 8 && a.d <= 32 * ve) return launch(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
    if (vec == 16 && (a.cache.group == a.d || (gv & (gv - 1)) == 0))
        return launch(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
    return launch(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{});
}

template <typename T>
nrm_status cache_write(const HeadArgs& a, int vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    const bool both = a.x[1].p && a.x[2].p;
    return cache_rows<T>(a, vec, [&](auto bytes, auto nv) {
        if constexpr (bytes.value == 0) {
            return cache_launch(a, (const void*)&cache_write_scalar_kernel<T>, 1, 5, both, *d, s);
        } else {
            constexpr int VE = bytes.value / int(sizeof(T));
            const int lg = row_lanes_log2(a.d / VE);
            return cache_launch(a, (const void*)&cache_write_vec_kernel<T, VE, nv.value>, (32 >> lg) * kCacheRows, lg,
                                both, *d, s);
        }
    });
}

template <typename T>
nrm_status cache_read(const HeadArgs& a, int vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    const bool both = a.y[0].p && a.y[1].p;
    return cache_rows<T>(a, vec, [&](auto bytes, auto nv) {
        if constexpr (bytes.value == 0) {
            return cache_launch(a, (const void*)&cache_read_scalar_kernel<T>, 1, 5, both, *d, s);
        } else {
            constexpr int VE = bytes.value / int(sizeof(T));
            const int lg = row_lanes_log2(a.d / VE);
            return cache_launch(a, (const void*)&cache_read_vec_kernel<T, VE, nv.value>, (32 >> lg) * kCacheRows, lg,
                                both, *d, s);
        }
    });
}

}  // namespace nrm

// Instantiates the operators for one storage dtype.
#define NRM_INSTANTIATE_HEADS(T)                                                                       \
    namespace nrm {                                                                                    \
    template nrm_status head_fwd<T>(const HeadArgs&, bool, bool, int, cudaStream_t);                  \
    template nrm_status head_bwd<T>(const HeadArgs&, int, cudaStream_t);                              \
    template nrm_status cache_write<T>(const HeadArgs&, int, cudaStream_t);                           \
    template nrm_status cache_read<T>(const HeadArgs&, int, cudaStream_t);                            \
    }
