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

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "heads.h"

namespace nrm {

constexpr int kHeadWarps = 8;                       // warps of a CTA

// Every kernel here is launched with its predecessor in the stream still running:
// it sets up its indices, then waits for that kernel's end before it touches
// memory, and lets its own successor be launched.
__device__ __forceinline__ void pdl_next() {
    pdl_wait();
    pdl_trigger();
}

// A load of what the predecessor may have written: weights, frequencies, positions,
// slots, codes, scales.  The read-only path (__ldg, const __restrict__) wants memory
// that nobody writes while the kernel lives, and here the predecessor still does;
// the compiler may also move such loads to before the wait.  It was no faster:
// a read of 131072 tokens from 4 bits takes 110 us either way.
template <typename R>
__device__ __forceinline__ R ld_after(const R* p) {
    R r;
    if constexpr (sizeof(R) == 1) {
        uint32_t v;
        asm volatile("ld.global.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
        r = R(v);
    } else if constexpr (sizeof(R) == 2) {
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(*reinterpret_cast<uint16_t*>(&r)) : "l"(p) : "memory");
    } else if constexpr (sizeof(R) == 4) {
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(*reinterpret_cast<uint32_t*>(&r)) : "l"(p) : "memory");
    } else if constexpr (std::is_integral_v<R>) {
        asm volatile("ld.global.u64 %0, [%1];" : "=l"(r) : "l"(p) : "memory");
    } else if constexpr (sizeof(R) == 8) {
        asm volatile("ld.global.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    } else {
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    }
    return r;
}

// Work in waves: as many CTAs as are resident at once, each warp taking `rounds`
// units that lie a wave's warps apart, then the next wave's CTAs.  CTAs that stay
// for all of a large problem drift apart, and what the GPU touches at one time
// spreads over more and more of memory: the rotation of 65536 tokens (bf16, 12 + 12
// heads of 128: 400 MB read and 400 written) takes 140 us that way, 117 in waves of
// four or six rounds (118 at the copy rate), 121 of eight and 127 of ten.  Where
// instructions bound (the norm of heads of 64), a new wave's start costs 1 to 2% at
// six rounds, 4% at four.
constexpr int kWaveRounds = 6;  // at most
struct Waves {
    int ctas, rounds;  // of a wave
};
template <int WARPS>
struct WaveUnits {
    int64_t first, end, stride;  // of this warp
    __device__ __forceinline__ WaveUnits(const Waves& w, int64_t units, int warp) {
        const int wave = int(blockIdx.x) < w.ctas ? 0 : int(blockIdx.x) / w.ctas;
        stride = int64_t(w.ctas) * WARPS;
        first = wave * w.rounds * stride;
        end = min(units, first + w.rounds * stride);
        first += (int(blockIdx.x) - wave * w.ctas) * WARPS + warp;
    }
};

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
// phase's top 32 bits, in 2^-32 turns, are taken off the nearest quarter turn before
// they become a float32, which so is off by at most 2^-28 turns (of a whole half turn
// it would be 2^-26: cosines off by 1.5 units in their last place more).  The quarter
// turns then exchange and negate the two.
__device__ __forceinline__ float2 pair_turn(const RopeDev& r, uint64_t step, int64_t pos) {
    const uint32_t phase = uint32_t((uint64_t(pos) * step) >> 32);
    const uint32_t quarters = (phase + 0x20000000u) >> 30;
    float s, c;
    sincospif(float(int32_t(phase - (quarters << 30))) * 0x1p-31f, &s, &c);
    const float cos = quarters & 1u ? s : c, sin = quarters & 1u ? c : s;
    const uint32_t neg_cos = (quarters + 1u) << 30, neg_sin = (quarters << 30) ^ (r.inverse ? 0x80000000u : 0u);
    return make_float2(__uint_as_float(__float_as_uint(cos) ^ (neg_cos & 0x80000000u)),
                       __uint_as_float(__float_as_uint(sin) ^ (neg_sin & 0x80000000u)));
}

// (u, v) turned by (cos, sin), rounded as on vectors (LaneMap, LaneTurns): the
// rotation's bits do not depend on how a row is accessed.
__device__ __forceinline__ void turn(float& u, float& v, float2 cs) {
    const float a = fmaf(-v, cs.y, __fmul_rn(u, cs.x));
    const float b = fmaf(u, cs.y, __fmul_rn(v, cs.x));
    u = a;
    v = b;
}

// ---------------------------------------------------------------------------
// quantising a group by its largest magnitude
// ---------------------------------------------------------------------------
// A stored form: its largest number, and one over it.
struct FormQ {
    int kind;
    float q, r;
    __device__ __forceinline__ constexpr explicit FormQ(int k) : kind(k), q(0.f), r(0.f) {
        q = k == NRM_CACHE_E4M3 ? 448.f : (k == NRM_CACHE_INT8 ? 127.f : 7.f);
        r = k == NRM_CACHE_E4M3 ? 1.f / 448.f : (k == NRM_CACHE_INT8 ? 1.f / 127.f : 1.f / 7.f);
    }
};

// A group's scale and what its codes need, from the bits of its largest
// magnitude (compared as integers, so a NaN is the largest of all).  Groups
// above 2^100 are divided by 2^32, and of float32 groups those below 2^-36
// multiplied by 2^64 (exactly, where it matters), so that products stay finite
// and residuals representable.
struct GroupQ {
    float scale;
    float n, r;  // minus the scaled largest magnitude, and about its reciprocal; both 0 where every code is 0
    float q;     // the form's largest number, scaled like m
};
// m/q rounded to nearest, for the forms' q: Markstein's division by a known number
// (checked against the division for every mantissa).
__device__ __forceinline__ float over_qmax(float m, const FormQ& f) {
    const float s = __fmul_rn(m, f.r);
    return fmaf(fmaf(-s, f.q, m), f.r, s);
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <typename T>
__device__ __forceinline__ GroupQ group_q(uint32_t m_bits, const FormQ& f) {
    const float m = __uint_as_float(m_bits);
    float p = 1.f;
    if constexpr (sizeof(T) == 4) p = m < 0x1p-36f ? 0x1p64f : p;
    if constexpr (!std::is_same_v<T, __half>) p = m > 0x1p100f ? 0x1p-32f : p;
    GroupQ g{over_qmax(m, f), -(m * p), rcp_approx(m * p), f.q * p};
    // a NaN or an infinity (the group reads back as NaN), or nothing but (almost) zeros
    const bool nan = m_bits >= 0x7f800000u;
    if (nan || m < 0x1p-100f) g = GroupQ{nan ? __uint_as_float(0x7fffffffu) : 0.f, 0.f, 0.f, 0.f};
    return g;
}
// x*q/m, such that the code nearest to it is the one nearest to the real
// quotient, ties seen as ties: u0 = (x*q)*r is off by a few units in the last
// place (r by one), and one step with its residual (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990) mends it.
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
        const float u = fmaf(fmaf(u0, g.n, n), g.r, u0);
        return g.r == 0.f ? 0.f : u;  // (a NaN is no code)
    } else {
        const float lost = fmaf(x, g.q, -n);  // n + lost == x*q
        const float u = fmaf(fmaf(u0, g.n, n) + lost, g.r, u0);
        const float left = fmaf(u, g.n, n) + lost;
        const int bits = __float_as_int(u);
        const bool off = left != 0.f && (bits & 1) == 0 && fabsf(u) >= 0x1p-24f;
        const float odd = off ? __int_as_float(bits + ((left > 0.f) == (u > 0.f) ? 1 : -1)) : u;
        return g.r == 0.f ? 0.f : odd;
    }
}
// Of two elements, neither a NaN.
template <typename T>
__device__ __forceinline__ float2 group_scaled2(float2 x, const GroupQ& g) {
    if constexpr (sizeof(T) == 2) {
        const float2 n = __fmul2_rn(x, f2(g.q)), u0 = __fmul2_rn(n, f2(g.r));
        return __ffma2_rn(__ffma2_rn(u0, f2(g.n), n), f2(g.r), u0);
    } else {
        return make_float2(group_scaled<T>(x.x, g), group_scaled<T>(x.y, g));
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
    CacheRow r{head * c.head_stride, head * c.scale_head_stride};
    if (!c.flat) {
        const int64_t page = row_div(slot, c.page);
        slot -= page * c.page.d;
        r.code += page * c.page_stride;
        r.scale += page * c.scale_page_stride;
    }
    r.code += slot * c.slot_stride;
    r.scale += slot * c.scale_slot_stride;
    return r;
}

// Quantises the d values of `row` (of T, as floats in shared memory, visible to
// the warp) into the cache's tensor `which` (0: keys, 1: values).
template <typename T>
__device__ __forceinline__ void quantise_row(const float* row, int d, const CacheDev& c, int which, int64_t slot,
                                             int head, int lane) {
    const CacheRow at = cache_row(c, slot, head);
    uint8_t* codes = c.codes[which] + at.code;
    float* scales = c.scales[which] + at.scale;
    const FormQ form(c.kind);
    for (int g0 = 0; g0 < d; g0 += c.group) {
        uint32_t m = 0;
        for (int i = lane; i < c.group; i += 32) m = max(m, __float_as_uint(row[g0 + i]) & 0x7fffffffu);
        const GroupQ q = group_q<T>(__reduce_max_sync(0xffffffffu, m), form);
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
// vectors of VE elements (16 or 8 bytes, or 4 bytes of a 16-bit type)
// ---------------------------------------------------------------------------
template <int BYTES> struct RawBits;
template <> struct RawBits<16> { using type = uint4; };
template <> struct RawBits<8> { using type = uint2; };
template <> struct RawBits<4> { using type = uint1; };
template <typename T, int VE> using Raw = typename RawBits<VE * int(sizeof(T))>::type;

// Loads of rows, which this kernel may write in place: not kept in L1.
__device__ __forceinline__ void ld_row(const void* p, uint4& r) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_row(const void* p, uint2& r) {
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld_row(const void* p, uint1& r) {
    asm volatile("ld.global.L1::no_allocate.u32 %0, [%1];" : "=r"(r.x) : "l"(p) : "memory");
}
__device__ __forceinline__ void st_row(void* p, uint4 v) { st_v4(p, v); }
__device__ __forceinline__ void st_row(void* p, uint2 v) {
    asm volatile("st.global.v2.u32 [%0], {%1,%2};" :: "l"(p), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void st_row(void* p, uint1 v) {
    asm volatile("st.global.u32 [%0], %1;" :: "l"(p), "r"(v.x) : "memory");
}

// The elements as pairs of floats, for the packed fp32 instructions (two elements
// each, rounded as the scalar instruction would).
template <typename T, int VE>
__device__ __forceinline__ void raw_unpack(const Raw<T, VE>& r, float2 (&v)[VE / 2]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else v[i] = cvt2<T>(w[i]);
    }
}
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> raw_pack(const float2 (&v)[VE / 2]) {
    Raw<T, VE> r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(v[i].x);
            w[2 * i + 1] = __float_as_uint(v[i].y);
        } else {
            w[i] = pack2<T>(v[i]);
        }
    }
    return r;
}

// A lane's two vectors as the first and the second elements of its VE pairs: the
// two vectors, or (ADJ) the even and the odd elements of both.
template <typename T, int VE, bool ADJ>
__device__ __forceinline__ void pair_unpack(const Raw<T, VE>& r0, const Raw<T, VE>& r1, float2 (&u)[VE / 2],
                                            float2 (&v)[VE / 2]) {
    float2 a[VE / 2], b[VE / 2];
    raw_unpack<T, VE>(r0, a);
    raw_unpack<T, VE>(r1, b);
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        if constexpr (!ADJ) {
            u[i] = a[i];
            v[i] = b[i];
        } else {
            const float2 x = 2 * i < VE / 2 ? a[2 * i % (VE / 2)] : b[2 * i % (VE / 2)];
            const float2 y = 2 * i + 1 < VE / 2 ? a[(2 * i + 1) % (VE / 2)] : b[(2 * i + 1) % (VE / 2)];
            u[i] = make_float2(x.x, y.x);
            v[i] = make_float2(x.y, y.y);
        }
    }
}
template <typename T, int VE, bool ADJ>
__device__ __forceinline__ void pair_pack(const float2 (&u)[VE / 2], const float2 (&v)[VE / 2], Raw<T, VE>& r0,
                                          Raw<T, VE>& r1) {
    if constexpr (!ADJ) {
        r0 = raw_pack<T, VE>(u);
        r1 = raw_pack<T, VE>(v);
    } else {
        float2 e[VE];  // the pairs in their order
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            e[2 * i] = make_float2(u[i].x, v[i].x);
            e[2 * i + 1] = make_float2(u[i].y, v[i].y);
        }
        float2 a[VE / 2], b[VE / 2];
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            a[i] = e[i];
            b[i] = e[VE / 2 + i];
        }
        r0 = raw_pack<T, VE>(a);
        r1 = raw_pack<T, VE>(b);
    }
}

// Largest magnitudes (a NaN is the largest of all): of float32 its bits, compared
// as integers; of 16-bit types two at once, in the halves of a word.
template <typename T>
__device__ __forceinline__ uint32_t mag_max(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) {
        return max(a, b & 0x7fffffffu);
    } else if constexpr (std::is_same_v<T, __half>) {
        const __half2 m = __hmax2_nan(*reinterpret_cast<__half2*>(&a), __habs2(*reinterpret_cast<__half2*>(&b)));
        return *reinterpret_cast<const uint32_t*>(&m);
    } else {
        const __nv_bfloat162 m =
            __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
}
template <typename T, int VE>
__device__ __forceinline__ uint32_t raw_mag(const Raw<T, VE>& r) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VE * int(sizeof(T)) / 4; ++i) m = mag_max<T>(m, w[i]);
    return m;
}
// The float32 bits of what such a word holds.
template <typename T>
__device__ __forceinline__ uint32_t mag_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    else return __float_as_uint(Io<T>::load(typename Io<T>::bits_t(max(m & 0xffffu, m >> 16))));
}

// Codes of VE consecutive elements, in the low bytes of two words.  A whole number
// comes out of the low bits of u + 1.5 * 2^23 (the sum rounds to nearest, ties to
// even).
template <typename T, int VE>
__device__ __forceinline__ uint2 make_codes(Raw<T, VE> x, const GroupQ& q, int kind) {
    if (q.r == 0.f) x = Raw<T, VE>{};  // no NaN reaches the arithmetic
    float2 u[VE / 2];
    raw_unpack<T, VE>(x, u);
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) u[i] = group_scaled2<T>(u[i], q);
    uint32_t w[2] = {0u, 0u};
    if (kind == NRM_CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < VE; i += 2) w[i / 4] |= e4m3x2(u[i / 2].x, u[i / 2].y) << (8 * (i % 4));
        return make_uint2(w[0], w[1]);
    }
    constexpr uint32_t magic = 0x4B400000u;  // 1.5 * 2^23
    uint32_t b[VE];
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) {
        const float2 f = __fadd2_rn(u[i], f2(__uint_as_float(magic)));
        b[2 * i] = __float_as_uint(f.x);
        b[2 * i + 1] = __float_as_uint(f.y);
    }
    if (kind == NRM_CACHE_INT8) {
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
            const uint32_t two = __byte_perm(b[i], b[i + 1], 0x0040);
            w[i / 4] = i % 4 ? __byte_perm(w[i / 4], two, 0x5410) : two;
        }
        if constexpr (VE == 2) w[0] &= 0xffffu;
    } else {
        // sum of code_i * 16^i: the constants come off at the end, and with 8 added to
        // each code no digit borrows from the next
        constexpr uint32_t ones = VE == 8 ? 0x11111111u : (VE == 4 ? 0x1111u : 0x11u);
        uint32_t d = b[VE - 1];
#pragma unroll
        for (int i = VE - 2; i >= 0; --i) d = d * 16 + b[i];
        w[0] = (d - magic * ones + 8 * ones) ^ (8 * ones);
    }
    return make_uint2(w[0], w[1]);
}
// Stores 1, 2, 4 or 8 bytes at an address aligned to them.
__device__ __forceinline__ void st_bytes(uint8_t* at, uint2 w, int bytes) {
    if (bytes == 8) *reinterpret_cast<uint2*>(at) = w;
    else if (bytes == 4) *reinterpret_cast<uint32_t*>(at) = w.x;
    else if (bytes == 2) *reinterpret_cast<uint16_t*>(at) = uint16_t(w.x);
    else *at = uint8_t(w.x);
}
template <typename T, int VE>
__device__ __forceinline__ void store_codes(uint8_t* at, Raw<T, VE> x, const GroupQ& q, int kind) {
    const uint2 w = make_codes<T, VE>(x, q, kind);
    if (kind == NRM_CACHE_INT4) st_bytes(at, w, VE / 2);
    else st_bytes(at, w, VE);
}
// The codes of two neighbouring vectors.
template <typename T, int VE>
__device__ __forceinline__ void store_codes_twice(uint8_t* at, const Raw<T, VE> (&x)[2], const GroupQ& q, int kind) {
    const uint2 a = make_codes<T, VE>(x[0], q, kind), b = make_codes<T, VE>(x[1], q, kind);
    if (kind == NRM_CACHE_INT4) {
        constexpr int bits = 4 * VE;
        if constexpr (VE == 8) st_bytes(at, make_uint2(a.x, b.x), 8);
        else st_bytes(at, make_uint2(a.x | b.x << (bits % 32), 0u), VE);
    } else if constexpr (VE == 8) {
        *reinterpret_cast<uint4*>(at) = make_uint4(a.x, a.y, b.x, b.y);
    } else if constexpr (VE == 4) {
        st_bytes(at, make_uint2(a.x, b.x), 8);
    } else {
        st_bytes(at, make_uint2(a.x | b.x << 16, 0u), 4);
    }
}

// A lane's place in the vector kernels: which row of the warp's, which pair of
// vectors of that row, and where they lie.  2^lg lanes hold a row.
template <int VE, bool ADJ>
struct LaneAt {
    int sub, j;      // row of the warp's 32 >> lg rows, pair of vectors of the row
    int b0, b1;      // first elements of the two vectors
    bool on, turns;  // holds elements; they turn
    __device__ __forceinline__ LaneAt(int lane, int lg, int d, const RopeDev& r) {
        sub = lane >> lg;
        j = lane & ((1 << lg) - 1);
        on = 2 * VE * j < d;
        turns = 2 * VE * j < r.rot;
        const bool half = turns && !ADJ;
        b0 = half ? VE * j : 2 * VE * j;
        b1 = half ? VE * j + (r.rot >> 1) : b0 + VE;
    }
};

// The turn of each pair per position, with the pair's axis in the low two bits
// (an angle loses less than |pos| * 2^-62 turns by that).  Filled by the CTA's
// threads; the caller's barrier makes them visible.
__device__ __forceinline__ void fill_steps(const RopeDev& r, uint64_t* steps, int tid, int threads) {
    for (int p = tid; 2 * p < r.rot; p += threads)
        steps[p] = (turn_step(ld_after(r.inv_freq + p)) & ~uint64_t(3)) | uint64_t(pair_axis(r, p));
}
// What a warp copies for the tokens of a unit: positions (one an axis), cache slot.
constexpr int kTokenSlot = kHeadMaxAxes;
struct TokenWords {
    int64_t w[kHeadMaxAxes + 1];
};
// cos[k * rot/2 + p], sin[...] of each token k at positions tok[k].w[axis], for
// every pair p: lane l makes those of pairs l, l + 32, ..., and every lane then
// takes the VE pairs of its own vectors from there.  Called by the whole warp.
template <typename W>
__device__ __forceinline__ void make_turns(const RopeDev& r, const uint64_t* steps, int lane, const W* tok, int tokens,
                                           float* cos, float* sin) {
    __syncwarp();
    const int pairs = r.rot >> 1;
    for (int p = lane; p < pairs; p += 32) {
        const uint64_t step = steps[p];
        for (int k = 0; k < tokens; ++k) {
            const float2 cs = pair_turn(r, step & ~uint64_t(3), tok[k].w[step & 3]);
            cos[k * pairs + p] = cs.x;
            sin[k * pairs + p] = cs.y;
        }
    }
    __syncwarp();
}

// A lane's VE angles.
template <int VE>
struct LaneTurns {
    float2 c[VE / 2], s[VE / 2];
    __device__ __forceinline__ void take(const float* cos, const float* sin) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            c[i] = *reinterpret_cast<const float2*>(cos + 2 * i);
            s[i] = *reinterpret_cast<const float2*>(sin + 2 * i);
        }
    }
    // Turns the lane's pairs.  (The packed instruction cannot negate: one product is scalar.)
    __device__ __forceinline__ void turn(float2 (&u)[VE / 2], float2 (&v)[VE / 2]) const {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const float2 a = __fmul2_rn(u[i], c[i]);
            const float2 b = __ffma2_rn(u[i], s[i], __fmul2_rn(v[i], c[i]));
            u[i] = make_float2(fmaf(-v[i].x, s[i].x, a.x), fmaf(-v[i].y, s[i].y, a.y));
            v[i] = b;
        }
    }
};

// The forward's row map of a lane: the weights w0, w1 of its pairs' two elements
// and their turn in one, (u, v) -> (uu u + uv v, vu u + vv v), uu = w0 cos, uv =
// -w1 sin, vu = w0 sin, vv = w1 cos.  Made once for a token's rows of a tensor,
// and fewer registers than weights and angles.
template <int VE>
struct LaneMap {
    float2 uu[VE / 2], uv[VE / 2], vu[VE / 2], vv[VE / 2];
    // w0, w1 on entry in uu, vv.
    __device__ __forceinline__ void turned(const float* cos, const float* sin) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const float2 c = *reinterpret_cast<const float2*>(cos + 2 * i);
            const float2 s = *reinterpret_cast<const float2*>(sin + 2 * i);
            uv[i] = __fmul2_rn(vv[i], f2neg(s));
            vu[i] = __fmul2_rn(uu[i], s);
            uu[i] = __fmul2_rn(uu[i], c);
            vv[i] = __fmul2_rn(vv[i], c);
        }
    }
    // (`turns`: elements past the rotated part are their own, whatever their partner holds)
    template <int R>
    __device__ __forceinline__ void apply(float2 (&u)[R][VE / 2], float2 (&v)[R][VE / 2], bool turns) const {
        if (turns) {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i)
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const float2 a = __ffma2_rn(v[k][i], uv[i], __fmul2_rn(u[k][i], uu[i]));
                    v[k][i] = __ffma2_rn(u[k][i], vu[i], __fmul2_rn(v[k][i], vv[i]));
                    u[k][i] = a;
                }
        } else {
#pragma unroll
            for (int i = 0; i < VE / 2; ++i)
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    u[k][i] = __fmul2_rn(u[k][i], uu[i]);
                    v[k][i] = __fmul2_rn(v[k][i], vv[i]);
                }
        }
    }
};

// Sum over the 2^lg lanes of a row; every lane of it gets the same bits.
__device__ __forceinline__ float row_sum(float v, int lg) {
#pragma unroll
    for (int i = 4; i >= 0; --i)
        if (i < lg) v += __shfl_xor_sync(0xffffffffu, v, 1 << i);
    return v;
}
template <typename T>
__device__ __forceinline__ uint32_t row_mag(uint32_t m, int lg) {
#pragma unroll
    for (int i = 4; i >= 0; --i)
        if (i < lg) m = mag_max<T>(m, __shfl_xor_sync(0xffffffffu, m, 1 << i));
    return m;
}

// ---------------------------------------------------------------------------
// asynchronous copies of a lane's own vectors
// ---------------------------------------------------------------------------
// A lane copies its vectors of the next steps to places in shared memory that no
// other lane reads, a step or more ahead, so the bytes in flight do not
// depend on registers or occupancy and no barrier is needed: the lane waits for
// its own copies.
constexpr int kHeadStages = 3;  // backward

template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_addr(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(smem_addr(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of copies of this thread have landed.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Copies the positions of 2^ltok tokens from t0 on (those below `tokens`).
template <bool MANY, typename W>
__device__ __forceinline__ void copy_positions(const RopeDev& r, W* tok, int64_t t0, int ltok, int64_t tokens, int lane) {
    static_assert(kHeadMaxAxes == 4, "four words a token");
    if constexpr (!MANY) {
        if (lane < r.axes) cp_async<8>(&tok[0].w[lane], r.pos + lane * r.pos_stride + t0);
    } else {
        for (int i = lane; i < 4 << ltok; i += 32)
            if ((i & 3) < r.axes && t0 + (i >> 2) < tokens)
                cp_async<8>(&tok[i >> 2].w[i & 3], r.pos + (i & 3) * r.pos_stride + t0 + (i >> 2));
    }
}

// ---------------------------------------------------------------------------
// forward on vectors: norm, rotation, cache
// ---------------------------------------------------------------------------

// A warp's way through its work: (2^ltok tokens, chunk) units, of each the tensors
// q, k (and v), of each the row steps chunk, chunk + 2^lchunk, ... of a token's
// steps counted through all tensors.  A step is kHeadRows rows of a lane; the
// common one, to the tensor's next step, adds to a head and (in the caller) to a
// pointer.
template <int TENSORS, bool MANY>
struct StepWalk {
    int64_t un;          // unit
    int which;           // tensor
    int h0, heads;       // the step's first head; the tensor's heads
    int first;           // steps of the token's earlier tensors
    bool fresh, turned;  // the first step of a unit; of a tensor (of a unit)
    int lper, lchunk, ltok;  // log2 of: heads of a step, chunks, tokens of a unit
    int64_t units, stride;

    __device__ __forceinline__ void start(const HeadArgs& a, int64_t unit) {
        un = unit;
        which = first = 0;
        fresh = true;
        settle(a);
    }
    __device__ __forceinline__ bool live() const { return un < units; }
    // The unit's first token.
    __device__ __forceinline__ int64_t token() const { return MANY ? un >> lchunk << ltok : un >> lchunk; }
    __device__ __forceinline__ int head_step() const { return 1 << (lper + lchunk); }
    // Moves to the next step; `turned` stays false where only the head moved, within the tensor.
    __device__ __forceinline__ void next(const HeadArgs& a) {
        h0 += head_step();
        fresh = turned = false;
        if (h0 < heads) return;
        leave(a);
        settle(a);
    }

private:
    __device__ __forceinline__ void leave(const HeadArgs& a) {
        first += (heads + (1 << lper) - 1) >> lper;
        if (++which == TENSORS) {
            un += stride;
            which = first = 0;
            fresh = true;
        }
    }
    __device__ __forceinline__ void settle(const HeadArgs& a) {
        turned = true;
        while (un < units) {
            heads = a.heads[which];
            h0 = ((int(un) - first) & ((1 << lchunk) - 1)) << lper;
            if (h0 < heads) return;
            leave(a);
        }
    }
};

// For each row x of q and k: r = (mean(x^2) + eps)^-1/2, y = R(x r w) as one map of
// pairs times r (without the norm r = 1 and the map is the rotation); rows of k and
// v also go to the cache (below).
//
// Bound by bytes (a row is read and written once), and close behind by issue
// slots: with the row arithmetic left out the kernel's copies alone take 50 us of
// its 53 at bf16 16384 tokens of 32 + 8 heads of 128 (338 MB, 50 us at the copy
// rate of 6.8 TB/s; 6.3 TB/s reached).  What was measured there, in us:
//   one row a warp, scalar 259; vectors, a lane's rows loaded as they are needed 85;
//   fp32 pairs and uniform steps 69; copies ahead, one row a step 72 (the rotation
//   of 32760 tokens 77 -> 64); two rows a step 58; weights and angles in one map,
//   57, with 40 registers fewer; the turns per position in shared memory and three
//   stages 56; work in waves, weights in shared memory and the norm a template
//   parameter 53 (the rotation of video tokens 66 -> 61, of 25216 image tokens of 12
//   + 12 heads of 64 30 -> 26.5, at 116 registers in four CTAs an SM).
// Three CTAs of four warps an SM at up to 168 registers (the rotation alone needs
// fewer, and four fit).  Before the waves, the norm took 61 in four CTAs of 128
// registers and 57 in two of eight warps; a serving chunk 42 and 44 against 41.  A
// fourth stage 55; steps of four rows, two at a time, 57 to 58.
constexpr int kHeadRows = 2;      // rows of a lane in a step
constexpr int kHeadFwdWarps = 4;  // warps of a CTA
constexpr int kHeadFwdStages = 3;

template <typename T, int VE>
constexpr size_t head_fwd_smem() {
    return size_t(kHeadFwdStages) * 2 * kHeadRows * kHeadFwdWarps * 32 * VE * sizeof(T);
}

template <typename T, int VE, bool ADJ, bool CACHE, bool MANY, bool norm>
__global__ void __launch_bounds__(kHeadFwdWarps * 32, 3)
head_fwd_vec_kernel(const __grid_constant__ HeadArgs a, int lg, int ltokens, int lchunk, Waves waves) {
    constexpr int H = VE / 2, D = kHeadFwdStages, R = kHeadRows, N = kHeadFwdWarps * 32, BYTES = VE * int(sizeof(T));
    extern __shared__ __align__(16) unsigned char dyn[];
    // (a warp's rows hold 32 * VE pairs, so its tokens have no more)
    __shared__ __align__(16) float s_cos[kHeadFwdWarps][MANY ? 32 * VE : kHeadMaxPairs];
    __shared__ __align__(16) float s_sin[kHeadFwdWarps][MANY ? 32 * VE : kHeadMaxPairs];
    __shared__ TokenWords s_tok[kHeadFwdWarps][D][MANY ? 32 : 1];
    __shared__ uint64_t s_step[kHeadMaxPairs];
    __shared__ Raw<T, VE> s_w[2][norm ? kHeadMaxD / VE : 1];  // the weights
    __shared__ uint32_t s_max[CACHE ? kHeadFwdWarps : 1][CACHE ? 64 : 1];
    Raw<T, VE>* ring = reinterpret_cast<Raw<T, VE>*>(dyn) + threadIdx.x;  // [stage][row][vector], N apart
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
    const LaneAt<VE, ADJ> at(lane, lg, a.d, a.rope);
    // the warp's rows are `rows` heads of each of its tokens
    const int ltok = MANY ? ltokens : 0, lhp = 5 - lg - ltok, rows = 1 << lhp;
    const int hsub = MANY ? at.sub & (rows - 1) : at.sub, tsub = MANY ? at.sub >> lhp : 0;
    const int b01 = at.b1 - at.b0;
    const float inv_d = 1.f / float(a.d);
    const int g0 = CACHE ? at.b0 / a.cache.group : 0, g1 = CACHE ? at.b1 / a.cache.group : 0;
    const FormQ form(CACHE ? a.cache.kind : 0);
    const int packed = form.kind == NRM_CACHE_INT4;  // two elements to a byte
    int meet_lanes = 0;  // lanes whose vectors are a group, where these are neighbours and a power of two
    if (CACHE) {
        const int gv = a.cache.group / VE, n = ADJ ? gv / 2 : gv;
        const bool order = ADJ ? gv % 2 == 0 : (a.rope.rot == a.d && a.d / (2 * VE) % gv == 0);
        if (order && (n & (n - 1)) == 0) meet_lanes = n;
    }

    // lanes past the row copy nothing, and read zeros
    if (!at.on)
#pragma unroll
        for (int i = 0; i < 2 * D * R; ++i) ring[i * N] = Raw<T, VE>{};
    StepWalk<CACHE ? 3 : 2, MANY> in;
    in.lper = lhp + (R == 2 ? 1 : 0);
    in.lchunk = lchunk;
    in.ltok = ltok;
    const WaveUnits<kHeadFwdWarps> own(waves, (a.tokens + (1 << ltok) - 1) >> ltok << lchunk, warp);
    in.units = own.end;
    in.stride = own.stride;
    in.start(a, own.first);
    StepWalk<CACHE ? 3 : 2, MANY> cur = in;

    const T* px = nullptr;  // this lane's first vector of the step to copy
    int64_t row_x = 0;      // from one of a lane's rows to its next
    auto issue = [&](int stage) {
        if (in.live()) {
            const int64_t t0 = in.token();
            if (in.turned) {
                const HeadView v = a.x[in.which];
                px = reinterpret_cast<const T*>(v.p) + (t0 + tsub) * v.ts + (in.h0 + hsub) * v.hs + at.b0;
                row_x = rows * v.hs;
            }
            const int first = at.on && (!MANY || t0 + tsub < a.tokens) ? in.h0 + hsub : in.heads;  // this lane's first head
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (first + k * rows < in.heads) {
                    const T* p = px + k * row_x;
                    cp_async<BYTES>(ring + ((stage * R + k) * 2) * N, p);
                    cp_async<BYTES>(ring + ((stage * R + k) * 2 + 1) * N, p + b01);
                }
            }
            if (in.fresh) {
                copy_positions<MANY>(a.rope, s_tok[warp][stage], t0, ltok, a.tokens, lane);
                if (CACHE && lane < 1 << ltok && (!MANY || t0 + lane < a.tokens))
                    cp_async<8>(&s_tok[warp][stage][lane].w[kTokenSlot], a.slots + t0 + lane);
            }
            px += (R * row_x) << lchunk;
            in.next(a);
        }
        cp_async_commit();
    };
    pdl_next();
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i);
    // (both loads are under way before either is waited for)
    constexpr int W = 2 * kHeadMaxD / VE, PER = (W + N - 1) / N;
    Raw<T, VE> wt[norm ? PER : 1];
    if (norm) {
        float2 ones[H];
#pragma unroll
        for (int i = 0; i < H; ++i) ones[i] = f2(1.f);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = threadIdx.x + k * N, which = i / (W / 2), e = i % (W / 2) * VE;
            const T* w = i < W ? reinterpret_cast<const T*>(a.w[which]) : nullptr;
            wt[k] = w && e < a.d ? ld_after(reinterpret_cast<const Raw<T, VE>*>(w + e)) : raw_pack<T, VE>(ones);
        }
    }
    fill_steps(a.rope, s_step, threadIdx.x, N);
    if (norm) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = threadIdx.x + k * N;
            if (i < W) s_w[i / (W / 2)][i % (W / 2)] = wt[k];
        }
    }
    __syncthreads();

    const int w0 = at.on ? at.b0 / VE : 0, w1 = at.on ? at.b1 / VE : 0;
    LaneMap<VE> map;
    T* py = nullptr;
    float* pr = nullptr;
    int64_t row_y = 0, slot = -1;
    CacheRow cr{0, 0};
    bool out = false;
    for (int stage = 0; cur.live(); stage = stage + 1 == D ? 0 : stage + 1) {
        cp_async_wait<D - 2>();
        const int which = cur.which, heads = cur.heads, h = cur.h0 + hsub;
        const int64_t t = cur.token() + tsub;
        Raw<T, VE> x0[R], x1[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            // (of a row past the tensor's heads: what an earlier step left, used by no one)
            x0[k] = ring[((stage * R + k) * 2) * N];
            x1[k] = ring[((stage * R + k) * 2 + 1) * N];
        }
        if (cur.fresh) {
            make_turns(a.rope, s_step, lane, s_tok[warp][stage], MANY ? 1 << ltok : 1, s_cos[warp], s_sin[warp]);
            if (CACHE) {
                slot = !MANY || t < a.tokens ? cache_slot(a.cache, s_tok[warp][stage][tsub].w[kTokenSlot], a.err) : -1;
                if (slot >= 0) cr = cache_row(a.cache, slot, 0);
            }
            __syncwarp();
        }
        issue(stage == 0 ? D - 1 : stage - 1);
        if (cur.turned && which < 2) {
            const HeadView v = a.y[which];
            py = reinterpret_cast<T*>(v.p) + t * v.ts + h * v.hs + at.b0;
            row_y = rows * v.hs;
            out = v.p && at.on && (!MANY || t < a.tokens);
            if (norm) pr = at.j == 0 && (!MANY || t < a.tokens) && a.rstd[which] ? a.rstd[which] + t * heads + h : nullptr;
            if (norm || cur.fresh) {  // (without weights q and k share the map)
                if (norm) {
                    pair_unpack<T, VE, ADJ>(s_w[which][w0], s_w[which][w1], map.uu, map.vv);
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) map.uu[i] = map.vv[i] = f2(1.f);
                }
                const int p = (MANY ? tsub * (a.rope.rot >> 1) : 0) + VE * at.j;
                if (at.turns) map.turned(&s_cos[warp][p], &s_sin[warp][p]);
            }
        }
        if (which < 2) {
            float2 u[R][H], v[R][H];
#pragma unroll
            for (int k = 0; k < R; ++k) pair_unpack<T, VE, ADJ>(x0[k], x1[k], u[k], v[k]);
            float r[R];
#pragma unroll
            for (int k = 0; k < R; ++k) r[k] = 1.f;
            if (norm) {
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    float2 sq = f2(0.f);
#pragma unroll
                    for (int i = 0; i < H; ++i) sq = __ffma2_rn(u[k][i], u[k][i], __ffma2_rn(v[k][i], v[k][i], sq));
                    r[k] = sq.x + sq.y;
                }
#pragma unroll
                for (int k = 0; k < R; ++k) r[k] = rsqrtf(fmaf(row_sum(r[k], lg), inv_d, a.eps));
#pragma unroll
                for (int k = 0; k < R; ++k)
                    if (pr && h + k * rows < heads) pr[k * rows] = r[k];
            }
            map.apply(u, v, at.turns);
            if (norm) {
#pragma unroll
                for (int i = 0; i < H; ++i)
#pragma unroll
                    for (int k = 0; k < R; ++k) {
                        u[k][i] = __fmul2_rn(u[k][i], f2(r[k]));
                        v[k][i] = __fmul2_rn(v[k][i], f2(r[k]));
                    }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                pair_pack<T, VE, ADJ>(u[k], v[k], x0[k], x1[k]);
                if (out && h + k * rows < heads) {
                    T* p = py + k * row_y;
                    st_row(p, x0[k]);
                    st_row(p + b01, x1[k]);
                }
            }
            py += (R * row_y) << lchunk;
            if (pr) pr += cur.head_step();
        }
        if constexpr (CACHE) {
            // (the warp's condition.)  The cache stores the key in the activations' type: what a
            // separate write would read.
            if (which > 0) {
                const int group = a.cache.group;
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    uint32_t m0 = raw_mag<T, VE>(x0[k]), m1 = raw_mag<T, VE>(x1[k]);
                    if (group == a.d) {
                        m0 = m1 = row_mag<T>(at.on ? mag_max<T>(m0, m1) : 0u, lg);
                    } else if (meet_lanes > 0) {
                        // a group is one vector each of so many neighbouring lanes, or (ADJ) two
                        if (ADJ) m0 = m1 = mag_max<T>(m0, m1);
#pragma unroll
                        for (int i = 4; i >= 0; --i)
                            if (1 << i < meet_lanes) {
                                m0 = mag_max<T>(m0, __shfl_xor_sync(0xffffffffu, m0, 1 << i));
                                if (!ADJ) m1 = mag_max<T>(m1, __shfl_xor_sync(0xffffffffu, m1, 1 << i));
                            }
                        if (ADJ) m1 = m0;
                    } else {
                        // groups of whole vectors, which other lanes may hold: through shared memory
                        uint32_t* sm = s_max[warp] + at.sub * (a.d / VE);
                        const int n = group / VE;
                        if (at.on) {
                            sm[at.b0 / VE] = m0;
                            sm[at.b1 / VE] = m1;
                        }
                        __syncwarp();
                        if (at.on) {
                            for (int i = 0; i < n; ++i) {
                                m0 = mag_max<T>(m0, sm[g0 * n + i]);
                                m1 = mag_max<T>(m1, sm[g1 * n + i]);
                            }
                        }
                        __syncwarp();
                    }
                    if (slot >= 0 && at.on && h + k * rows < heads) {
                        const int hk = h + k * rows;
                        const GroupQ q0 = group_q<T>(mag_bits<T>(m0), form);
                        const GroupQ q1 = group == a.d ? q0 : group_q<T>(mag_bits<T>(m1), form);
                        float* scales = a.cache.scales[which - 1] + cr.scale + hk * a.cache.scale_head_stride;
                        if (at.b0 == g0 * group) scales[g0] = q0.scale;
                        if (at.b1 == g1 * group) scales[g1] = q1.scale;
                        uint8_t* codes = a.cache.codes[which - 1] + cr.code + hk * a.cache.head_stride;
                        store_codes<T, VE>(codes + (at.b0 >> packed), x0[k], q0, form.kind);
                        store_codes<T, VE>(codes + (at.b1 >> packed), x1[k], q1, form.kind);
                    }
                }
            }
        }
        cur.next(a);
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// backward on vectors
// ---------------------------------------------------------------------------
// For each row: g' = R^T dy, g = g' w, dx = r g - x r^2 sum(r g x)/d; dw_i sums
// g'_i x_i r over tokens and heads.  A lane keeps the sums of its columns in
// registers over all its rows, in float32; the CTA's rows then meet in a fixed
// order and head_dw_kernel adds the CTAs' partial rows.  So that a lane's sums
// belong to one weight, CTAs take q or k; a token's angles are made twice for that.
//
// Bound by bytes: bf16 16384 tokens of 32 + 8 heads of 128, 506 MB, 75 us at the
// copy rate, 80 measured with the column sums (6.3 TB/s).  Loads as they were needed
// 109, copies three steps ahead 84, two steps ahead 79 to 81, one 92 (all two CTAs of
// eight warps; CTAs of four warps, three or four an SM, 81 and 80).  CTAs that stay:
// two waves, as many as the partial rows allow, gain 6% at 400 MB of inputs and lose
// 2 to 8% between 60 and 100 MB.
//
// A lane's copies of a step: two vectors each of dy and x, and the row's r.
template <typename T, int VE>
constexpr size_t head_bwd_smem() {
    return size_t(kHeadStages) * kHeadWarps * 32 * (4 * VE * sizeof(T) + 4);
}

// How the backward's work is laid out: CTAs [0, nq) take q, the others k.
struct BwdPlan {
    int lg, lchunk, nq;
    int ltok[2];  // tokens of a warp's step, of q and of k
};
struct Positions {
    int64_t w[kHeadMaxAxes];
};

template <typename T, int VE, bool ADJ, bool MANY>
__global__ void __launch_bounds__(kHeadWarps * 32, 2)
head_bwd_vec_kernel(const __grid_constant__ HeadArgs a, const __grid_constant__ BwdPlan plan) {
    constexpr int H = VE / 2, D = kHeadStages, BYTES = VE * int(sizeof(T)), N = kHeadWarps * 32;
    extern __shared__ __align__(16) unsigned char dyn[];
    // (a warp's rows hold 32 * VE pairs, so its tokens have no more)
    __shared__ __align__(16) float s_cos[kHeadWarps][kHeadMaxD], s_sin[kHeadWarps][MANY ? 32 * VE : kHeadMaxPairs];
    __shared__ Positions s_tok[kHeadWarps][D][MANY ? 32 : 1];
    float(*part)[kHeadMaxD] = s_cos;  // at the end: a warp's sums, over its own cosines
    __shared__ uint64_t s_step[kHeadMaxPairs];
    Raw<T, VE>* ring = reinterpret_cast<Raw<T, VE>*>(dyn) + threadIdx.x;  // [stage][vector], N apart
    float* ring_r = reinterpret_cast<float*>(dyn + size_t(D) * 4 * N * BYTES) + threadIdx.x;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
    const int which = int(blockIdx.x) < plan.nq ? 0 : 1;
    const int cta = int(blockIdx.x) - (which ? plan.nq : 0);
    const int ctas = which ? int(gridDim.x) - plan.nq : plan.nq;
    const int lg = plan.lg, lchunk = plan.lchunk, ltok = MANY ? plan.ltok[which] : 0;
    const LaneAt<VE, ADJ> at(lane, lg, a.d, a.rope);
    const int heads = a.heads[which], mask = (1 << lchunk) - 1;
    // the warp's rows are 2^lhp heads of each of its tokens
    const int lhp = 5 - lg - ltok;
    const int hsub = MANY ? at.sub & ((1 << lhp) - 1) : at.sub, tsub = MANY ? at.sub >> lhp : 0;
    const int hstep = 1 << (lhp + lchunk);  // heads from one of a unit's steps to its next
    const int64_t units = (a.tokens + (1 << ltok) - 1) >> ltok << lchunk, stride = int64_t(ctas) * kHeadWarps;
    const float inv_d = 1.f / float(a.d);
    const HeadView xv = a.x[which], gv = a.dy[which], dv = a.y[which];
    const int b01 = at.b1 - at.b0;
    const int64_t step_x = hstep * xv.hs, step_g = hstep * gv.hs, step_o = hstep * dv.hs;
    float2 w0[H], w1[H], acc0[H], acc1[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        w0[i] = w1[i] = f2(1.f);
        acc0[i] = acc1[i] = f2(0.f);
    }
    // lanes past the row copy nothing, and read zeros
    if (!at.on)
#pragma unroll
        for (int i = 0; i < 4 * D; ++i) ring[i * N] = Raw<T, VE>{};
    // the first head of unit un's first step; a unit without one is passed over
    auto first_head = [&](int64_t un) { return (int(un) & mask) << lhp; };
    auto enter = [&](int64_t& un, int& h0) {
        h0 = first_head(un);
        while (un < units && h0 >= heads) {
            un += stride;
            h0 = first_head(un);
        }
    };
    int64_t in_un = int64_t(cta) * kHeadWarps + warp;
    int in_h;
    enter(in_un, in_h);
    int64_t un = in_un;
    int h0 = in_h;
    bool in_fresh = true, fresh = true;
    const T *pg = nullptr, *px = nullptr;
    const float* pr = nullptr;
    T* po = nullptr;
    auto issue = [&](int stage) {
        if (in_un < units) {
            const int64_t t0 = in_un >> lchunk << ltok;
            if (in_fresh) {
                const int64_t t = t0 + tsub;
                const int h = in_h + hsub;
                pg = reinterpret_cast<const T*>(gv.p) + t * gv.ts + h * gv.hs + at.b0;
                px = reinterpret_cast<const T*>(xv.p) + t * xv.ts + h * xv.hs + at.b0;
                pr = a.rstd[which] + t * heads + h;
                copy_positions<MANY>(a.rope, s_tok[warp][stage], t0, ltok, a.tokens, lane);
            }
            if (at.on && in_h + hsub < heads && (!MANY || t0 + tsub < a.tokens)) {
                Raw<T, VE>* to = ring + stage * 4 * N;
                cp_async<BYTES>(to, pg);
                cp_async<BYTES>(to + N, pg + b01);
                cp_async<BYTES>(to + 2 * N, px);
                cp_async<BYTES>(to + 3 * N, px + b01);
                cp_async<4>(ring_r + stage * N, pr);
            }
            pg += step_g;
            px += step_x;
            pr += hstep;
            in_h += hstep;
            in_fresh = in_h >= heads;
            if (in_fresh) {
                in_un += stride;
                enter(in_un, in_h);
            }
        }
        cp_async_commit();
    };
    pdl_next();
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i);
    if (at.on && a.w[which]) {
        const T* w = reinterpret_cast<const T*>(a.w[which]);
        pair_unpack<T, VE, ADJ>(ld_after(reinterpret_cast<const Raw<T, VE>*>(w + at.b0)),
                                ld_after(reinterpret_cast<const Raw<T, VE>*>(w + at.b1)), w0, w1);
    }
    fill_steps(a.rope, s_step, threadIdx.x, N);
    __syncthreads();

    LaneTurns<VE> tn;
    for (int stage = 0; un < units; stage = stage + 1 == D ? 0 : stage + 1) {
        cp_async_wait<D - 2>();
        const int64_t t = (un >> lchunk << ltok) + tsub;
        const bool row = h0 + hsub < heads && (!MANY || t < a.tokens), on = row && at.on;
        const Raw<T, VE>* from = ring + stage * 4 * N;
        const Raw<T, VE> y0 = from[0], y1 = from[N], x0 = from[2 * N], x1 = from[3 * N];
        const float r = on ? ring_r[stage * N] : 0.f;
        if (fresh) {
            make_turns(a.rope, s_step, lane, s_tok[warp][stage], MANY ? 1 << ltok : 1, s_cos[warp], s_sin[warp]);
            const int p = (MANY ? tsub * (a.rope.rot >> 1) : 0) + VE * at.j;
            if (at.turns) tn.take(&s_cos[warp][p], &s_sin[warp][p]);
            po = reinterpret_cast<T*>(dv.p) + t * dv.ts + (h0 + hsub) * dv.hs + at.b0;
        }
        issue(stage == 0 ? D - 1 : stage - 1);
        float2 u[H], v[H], gu[H], gw[H];
        pair_unpack<T, VE, ADJ>(y0, y1, gu, gw);
        if (at.turns) tn.turn(gu, gw);
        pair_unpack<T, VE, ADJ>(x0, x1, u, v);
        float2 sum = f2(0.f);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            gu[i] = __fmul2_rn(gu[i], f2(r));
            gw[i] = __fmul2_rn(gw[i], f2(r));
            if (row) {  // (what a row past the heads reads is an earlier step's)
                acc0[i] = __ffma2_rn(gu[i], u[i], acc0[i]);
                acc1[i] = __ffma2_rn(gw[i], v[i], acc1[i]);
            }
            gu[i] = __fmul2_rn(gu[i], w0[i]);
            gw[i] = __fmul2_rn(gw[i], w1[i]);
            sum = __ffma2_rn(gu[i], u[i], __ffma2_rn(gw[i], v[i], sum));
        }
        // dx = r g - x r^2 sum(r g x) / d, the terms r g at hand
        const float f = -(row_sum(sum.x + sum.y, lg) * inv_d * r * r);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            gu[i] = __ffma2_rn(u[i], f2(f), gu[i]);
            gw[i] = __ffma2_rn(v[i], f2(f), gw[i]);
        }
        if (on) {
            Raw<T, VE> o0, o1;
            pair_pack<T, VE, ADJ>(gu, gw, o0, o1);
            st_row(po, o0);
            st_row(po + b01, o1);
        }
        po += step_o;
        h0 += hstep;
        fresh = h0 >= heads;
        if (fresh) {
            un += stride;
            enter(un, h0);
        }
    }
    cp_async_wait<0>();
    if (a.ws == nullptr) return;
    __syncwarp();
    // the warp's rows, then the CTA's warps, in a fixed order
#pragma unroll
    for (int i = 0; i < H; ++i) {
        for (int o = 1 << lg; o < 32; o <<= 1) {
            acc0[i].x += __shfl_xor_sync(0xffffffffu, acc0[i].x, o);
            acc0[i].y += __shfl_xor_sync(0xffffffffu, acc0[i].y, o);
            acc1[i].x += __shfl_xor_sync(0xffffffffu, acc1[i].x, o);
            acc1[i].y += __shfl_xor_sync(0xffffffffu, acc1[i].y, o);
        }
        if (at.sub == 0 && at.on) {
            const int e = ADJ ? at.b0 + 4 * i : at.b0 + 2 * i, f = ADJ ? e + 1 : at.b1 + 2 * i, n = ADJ ? 2 : 1;
            part[warp][e] = acc0[i].x;
            part[warp][e + n] = acc0[i].y;
            part[warp][f] = acc1[i].x;
            part[warp][f + n] = acc1[i].y;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += N) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kHeadWarps; ++w) sum += part[w][i];
        a.ws[int64_t(blockIdx.x) * a.d + i] = sum;
    }
}

// ---------------------------------------------------------------------------
// cache rows on vectors
// ---------------------------------------------------------------------------
// 2^lg lanes hold a row, one or two vectors each.  A warp's 32 >> lg row
// places are 2^lhp heads of each of its tokens; every lane goes over its heads,
// 2^lhp apart, a key and a value at a time.
struct CacheLanes {
    int lg;      // lanes of a row
    int per;     // lanes of them that hold vectors
    int lhp;     // heads of a token that the warp holds at once
    int lchunk;  // a token's heads are split over 2^lchunk warps
    int gl;      // writing: lanes of a group
    int wide;    // writing: a lane's 32 bytes are aligned to them
};

// 32 bytes at once, where they are aligned (every lane then fills whole sectors).
__device__ __forceinline__ void ld_row_wide(const void* p, uint4 (&r)[2]) {
    asm volatile("ld.global.L1::no_allocate.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0].x), "=r"(r[0].y), "=r"(r[0].z), "=r"(r[0].w), "=r"(r[1].x), "=r"(r[1].y), "=r"(r[1].z),
                   "=r"(r[1].w)
                 : "l"(p) : "memory");
}
// Writing.  A lane's vectors are neighbours: a group is then fewer lanes, and a
// lane makes one scale for both.  The group's largest magnitude meets by shuffles.
//
// Bound by issue slots (227 instructions for four rows of 128: magnitudes,
// a scale, four packed operations a pair of elements for codes that round like
// the real quotient) and by bytes: 131072 tokens of 8 + 8 heads of 128, bf16 to
// four bits in groups of 32, 706 MB, 104 us at the copy rate, 124 measured (5.7
// TB/s; CTAs that stay 129); to 8 bits, a scale a row, 815 MB, 120 and 124 to 127.
// One vector a lane, or two that are not neighbours, 160 to 215; copies ahead as in
// the forward 186 (more instructions); the form at run time 141.
template <typename T, int VE, int NV, int KIND>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_write_vec_kernel(const __grid_constant__ HeadArgs a, CacheLanes cl, Waves waves) {
    constexpr int E = NV * VE;  // elements of a lane
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
    const int sub = lane >> cl.lg, j = lane & ((1 << cl.lg) - 1), hp = 1 << cl.lhp, hsub = sub & (hp - 1);
    const bool on = j < cl.per;
    const int heads = a.heads[1], group = a.cache.group;
    constexpr FormQ form(KIND);
    constexpr int packed = KIND == NRM_CACHE_INT4;  // two elements to a byte
    const bool whole = group == a.d, pow2 = (cl.gl & (cl.gl - 1)) == 0;
    const int source = (sub << cl.lg) + (whole ? 0 : j / cl.gl * cl.gl);  // first lane of this lane's group
    const int gi = j * E / group;
    const bool leads = j * E == gi * group;
    const int ltok = 5 - cl.lg - cl.lhp;  // tokens of a warp
    const WaveUnits<kHeadWarps> own(waves, (a.tokens + (1 << ltok) - 1) >> ltok << cl.lchunk, warp);
    // neither a token's slot nor its rows wait for one another: the slot was asked for a unit ago
    auto ask = [&](int64_t un) {
        const int64_t t = (un >> cl.lchunk << ltok) + (sub >> cl.lhp);
        return un < own.end && t < a.tokens ? ld_after(a.slots + t) : int64_t(-1);
    };
    int64_t un = own.first;
    pdl_next();
    int64_t asked = ask(un);
    for (; un < own.end; un += own.stride) {
        const int64_t t = (un >> cl.lchunk << ltok) + (sub >> cl.lhp);
        const int64_t slot = cache_slot(a.cache, asked, a.err);
        asked = ask(un + own.stride);
        const bool live = t < a.tokens && on;
        int h0 = (int(un) & ((1 << cl.lchunk) - 1)) << cl.lhp;
        const CacheRow cr = cache_row(a.cache, slot < 0 ? 0 : slot, h0 + hsub);
        const T* px[2];
        uint8_t* pc[2];
        float* ps[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            px[w] = reinterpret_cast<const T*>(a.x[1 + w].p) + t * a.x[1 + w].ts + (h0 + hsub) * a.x[1 + w].hs + j * E;
            pc[w] = a.cache.codes[w] + cr.code + ((j * E) >> packed);
            ps[w] = a.cache.scales[w] + cr.scale + gi;
        }
#pragma unroll 1
        for (; h0 < heads; h0 += hp << cl.lchunk) {
            Raw<T, VE> raw[2][NV];
            const bool here = live && h0 + hsub < heads;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
#pragma unroll
                for (int v = 0; v < NV; ++v) raw[w][v] = Raw<T, VE>{};
                if (a.x[1 + w].p && here) {
                    if constexpr (NV * VE * sizeof(T) == 32) {
                        if (cl.wide) {
                            ld_row_wide(px[w], raw[w]);
                            continue;
                        }
                    }
#pragma unroll
                    for (int v = 0; v < NV; ++v) ld_row(px[w] + v * VE, raw[w][v]);
                }
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (a.x[1 + w].p) {
                    uint32_t m = raw_mag<T, VE>(raw[w][0]);
                    if constexpr (NV == 2) m = mag_max<T>(m, raw_mag<T, VE>(raw[w][1]));
                    if (whole) {
                        m = row_mag<T>(m, cl.lg);
                    } else if (pow2) {
#pragma unroll
                        for (int i = 4; i >= 0; --i)
                            if (1 << i < cl.gl) m = mag_max<T>(m, __shfl_xor_sync(0xffffffffu, m, 1 << i));
                    } else {
                        uint32_t all = 0;
                        for (int i = 0; i < cl.gl; ++i)
                            all = mag_max<T>(all, __shfl_sync(0xffffffffu, m, (source + i) & 31));
                        m = all;
                    }
                    if (here && slot >= 0) {
                        const GroupQ q = group_q<T>(mag_bits<T>(m), form);
                        if (leads) *ps[w] = q.scale;
                        if constexpr (NV == 2) store_codes_twice<T, VE>(pc[w], raw[w], q, form.kind);
                        else store_codes<T, VE>(pc[w], raw[w][0], q, form.kind);
                    }
                }
                px[w] += (hp * a.x[1 + w].hs) << cl.lchunk;
                pc[w] += (hp * a.cache.head_stride) << cl.lchunk;
                ps[w] += (hp * a.cache.scale_head_stride) << cl.lchunk;
            }
        }
    }
}

// VE codes, as they lie in memory.
template <int VE>
__device__ __forceinline__ uint2 load_codes(const uint8_t* at, int kind) {
    uint2 w{0u, 0u};
    if (kind == NRM_CACHE_INT4) {
        if constexpr (VE == 8) w.x = ld_after(reinterpret_cast<const uint32_t*>(at));
        else if constexpr (VE == 4) w.x = ld_after(reinterpret_cast<const uint16_t*>(at));
        else w.x = ld_after(at);
    } else {
        if constexpr (VE == 8) w = ld_after(reinterpret_cast<const uint2*>(at));
        else if constexpr (VE == 4) w.x = ld_after(reinterpret_cast<const uint32_t*>(at));
        else w.x = ld_after(reinterpret_cast<const uint16_t*>(at));
    }
    return w;
}
// The values they stand for, code * scale.  A whole number goes to float32 by way
// of its bits: with its sign bit flipped it takes a place in the mantissa of 2^23,
// where it reads 2^23 + (code + half) * 16^i; the power goes into the scale.
template <int VE>
__device__ __forceinline__ void code_values(uint2 w, int kind, float scale, float2 (&v)[VE / 2]) {
    if (kind == NRM_CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i)
            v[i] = __fmul2_rn(e4m3x2_values((i < 2 ? w.x : w.y) >> (16 * (i % 2))), f2(scale));
    } else if (kind == NRM_CACHE_INT8) {
        const uint32_t x = w.x ^ 0x80808080u, y = w.y ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
            const float2 f = make_float2(__uint_as_float(__byte_perm(i < 4 ? x : y, 0x4B000000u, 0x7650 + i % 4)),
                                         __uint_as_float(__byte_perm(i < 4 ? x : y, 0x4B000000u, 0x7651 + i % 4)));
            v[i / 2] = __fmul2_rn(__fadd2_rn(f, f2(-8388736.f)), f2(scale));  // - (2^23 + 128)
        }
    } else {
        const uint32_t x = w.x ^ 0x88888888u;
        const float2 down[2] = {make_float2(scale, scale * 0x1p-4f), make_float2(scale * 0x1p-8f, scale * 0x1p-12f)};
#pragma unroll
        for (int i = 0; i < VE; i += 2) {
            const uint32_t y = i < 4 ? x : x >> 16;
            const int p = 4 * (i % 4);
            const float2 f = make_float2(__uint_as_float((y & (0xfu << p)) | 0x4B000000u),
                                         __uint_as_float((y & (0xf0u << p)) | 0x4B000000u));
            const float2 off = i % 4 ? make_float2(-8390656.f, -8421376.f)   // - (2^23 + 8 * 16^2), 16^3
                                     : make_float2(-8388616.f, -8388736.f);  // - (2^23 + 8), 16
            v[i / 2] = __fmul2_rn(__fadd2_rn(f, off), down[i % 4 / 2]);
        }
    }
}

// Reading: bound by bytes, 706 MB for the same 131072 tokens, 104 us at the copy
// rate, 110 measured (6.4 TB/s; CTAs that stay 114).  A lane's two vectors are here
// those at j and j + per: each store of a warp then covers whole lines (two
// neighbouring vectors a lane, stored 32 bytes at once, took 122 against 116).  Five
// CTAs an SM; four and six 113 and 125 here, 11.4 and 12.1 against 10.7 for 15250
// tokens of 4 heads.
template <typename T, int VE, int KIND>
__global__ void __launch_bounds__(kHeadWarps * 32, 5)
cache_read_vec_kernel(const __grid_constant__ HeadArgs a, CacheLanes cl, Waves waves) {
    constexpr int NV = 2;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0);
    const int sub = lane >> cl.lg, j = lane & ((1 << cl.lg) - 1), hp = 1 << cl.lhp, hsub = sub & (hp - 1);
    const bool on = j < cl.per;
    const int heads = a.heads[1];
    constexpr int kind = KIND, packed = kind == NRM_CACHE_INT4;  // two elements to a byte
    const int ltok = 5 - cl.lg - cl.lhp;  // tokens of a warp
    const int v_next = (cl.per * VE) >> packed;
    int gi[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) gi[v] = (j + v * cl.per) * VE / a.cache.group;
    const WaveUnits<kHeadWarps> own(waves, (a.tokens + (1 << ltok) - 1) >> ltok << cl.lchunk, warp);
    auto ask = [&](int64_t un) {  // a token's slot, asked for a unit ahead
        const int64_t t = (un >> cl.lchunk << ltok) + (sub >> cl.lhp);
        return un < own.end && t < a.tokens ? ld_after(a.slots + t) : int64_t(-1);
    };
    int64_t un = own.first;
    pdl_next();
    int64_t asked = ask(un);
    for (; un < own.end; un += own.stride) {
        const int64_t t = (un >> cl.lchunk << ltok) + (sub >> cl.lhp);
        const int64_t slot = cache_slot(a.cache, asked, a.err);
        asked = ask(un + own.stride);
        if (slot < 0 || !on) continue;
        int h = ((int(un) & ((1 << cl.lchunk) - 1)) << cl.lhp) + hsub;
        const CacheRow cr = cache_row(a.cache, slot, h);
        const uint8_t* pc[2];
        const float* ps[2];
        T* py[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pc[i] = a.cache.codes[i] + cr.code + ((j * VE) >> packed);
            ps[i] = a.cache.scales[i] + cr.scale;
            py[i] = reinterpret_cast<T*>(a.y[i].p) + t * a.y[i].ts + h * a.y[i].hs + j * VE;
        }
#pragma unroll 1
        for (; h < heads; h += hp << cl.lchunk) {
            uint2 w[2][NV];
            float sc[2][NV];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.y[i].p) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        w[i][v] = load_codes<VE>(pc[i] + v * v_next, kind);
                        sc[i][v] = ld_after(ps[i] + gi[v]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.y[i].p) {
#pragma unroll
                    for (int v = 0; v < NV; ++v) {
                        float2 x[VE / 2];
                        code_values<VE>(w[i][v], kind, sc[i][v], x);
                        st_row(py[i] + v * cl.per * VE, raw_pack<T, VE>(x));
                    }
                }
                pc[i] += (hp * a.cache.head_stride) << cl.lchunk;
                ps[i] += (hp * a.cache.scale_head_stride) << cl.lchunk;
                py[i] += (hp * a.y[i].hs) << cl.lchunk;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// any layout: a row per warp, two elements per slot
// ---------------------------------------------------------------------------
// Rows whose rotated halves start between vectors (rot/2 odd), unaligned views, odd
// d.  Bound by latency and issue slots; a warp has 4 / S rows of S slots a lane
// under way.  bf16, 6653 tokens of 24 + 12 heads of 40 with 10 rotated (38 MB, 5.8 us
// at the copy rate): 55 us, one row at a time 64; backward 143.  About 250
// instructions a row.

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

// The turns per position of a lane's slots, and the axes.
template <int S>
struct SlotSteps {
    uint64_t step[S];
    int axis;
    __device__ __forceinline__ SlotSteps(const RopeDev& r, int lane) : axis(0) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
            step[s] = 0;
            if (2 * (lane + 32 * s) < r.rot) {
                step[s] = turn_step(ld_after(r.inv_freq + lane + 32 * s));
                axis |= pair_axis(r, lane + 32 * s) << (2 * s);
            }
        }
    }
    __device__ __forceinline__ void make(const RopeDev& r, int lane, int64_t t, float2 (&cs)[S]) const {
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (2 * (lane + 32 * s) < r.rot)
                cs[s] = pair_turn(r, step[s], ld_after(r.pos + (axis >> (2 * s) & 3) * r.pos_stride + t));
    }
};

template <typename T, int S, bool CACHE>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_fwd_scalar_kernel(const __grid_constant__ HeadArgs a, int norm) {
    constexpr int R = 4 / S;  // rows of a warp under way
    __shared__ float stage[CACHE ? kHeadWarps : 1][CACHE ? kHeadMaxD : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = a.heads[0] + a.heads[1] + (CACHE ? a.heads[2] : 0);
    const int slots = (a.d + 1) >> 1;
    pdl_next();
    const SlotSteps<S> steps(a.rope, lane);
    SlotAt e[S];
#pragma unroll
    for (int s = 0; s < S; ++s) e[s] = slot_at(lane + 32 * s, a.d, a.rope);
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        float2 cs[S];
        steps.make(a.rope, lane, t, cs);
        const int64_t slot = CACHE ? cache_slot(a.cache, ld_after(a.slots + t), a.err) : -1;
        const int apart = int(gridDim.y) * kHeadWarps;  // heads of a warp
        for (int h0 = warp + int(blockIdx.y) * kHeadWarps; h0 < heads; h0 += apart * R) {
            int which[R], hd[R];
            float u[R][S], v[R][S];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int hh = h0 + k * apart;
                which[k] = hh < a.heads[0] ? 0 : (hh < a.heads[0] + a.heads[1] ? 1 : (hh < heads ? 2 : 3));
                hd[k] = hh - (which[k] > 0 ? a.heads[0] : 0) - (which[k] > 1 ? a.heads[1] : 0);
                const HeadView xv = a.x[which[k] < 3 ? which[k] : 0];
                const T* x = reinterpret_cast<const T*>(xv.p) + t * xv.ts + hd[k] * xv.hs;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    u[k][s] = v[k][s] = 0.f;
                    if (which[k] < 3 && lane + 32 * s < slots) {
                        u[k][s] = ld_elem<T>(x, e[s].e0);
                        if (e[s].e1 < a.d) v[k][s] = ld_elem<T>(x, e[s].e1);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (which[k] < 2) {
                    float r = 1.f;
                    if (norm) {
                        float sum = 0.f;
#pragma unroll
                        for (int s = 0; s < S; ++s) sum = fmaf(u[k][s], u[k][s], fmaf(v[k][s], v[k][s], sum));
                        r = rsqrtf(warp_sum(sum) / float(a.d) + a.eps);
                        float* rstd = a.rstd[which[k]];
                        if (lane == 0 && rstd) rstd[t * a.heads[which[k]] + hd[k]] = r;
                    }
                    const HeadView yv = a.y[which[k]];
                    T* y = reinterpret_cast<T*>(yv.p) + t * yv.ts + hd[k] * yv.hs;
                    const void* w = a.w[which[k]];
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        if (lane + 32 * s < slots) {
                            const bool two = e[s].e1 < a.d;
                            if (norm) {
                                u[k][s] = __fmul_rn(u[k][s], r);
                                v[k][s] = __fmul_rn(v[k][s], r);
                                if (w) {
                                    u[k][s] = __fmul_rn(u[k][s], ld_elem<T>(w, e[s].e0));
                                    if (two) v[k][s] = __fmul_rn(v[k][s], ld_elem<T>(w, e[s].e1));
                                }
                            }
                            if (e[s].turns) turn(u[k][s], v[k][s], cs[s]);
                            if (yv.p) {
                                st_elem<T>(y, e[s].e0, u[k][s]);
                                if (two) st_elem<T>(y, e[s].e1, v[k][s]);
                            }
                        }
                    }
                }
                if (CACHE && which[k] > 0 && which[k] < 3 && slot >= 0) {
                    // the cache stores the key in the activations' type: what a separate write would read
                    float* row = stage[warp];
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        if (lane + 32 * s < slots) {
                            row[e[s].e0] = round_to<T>(u[k][s]);
                            if (e[s].e1 < a.d) row[e[s].e1] = round_to<T>(v[k][s]);
                        }
                    }
                    __syncwarp();
                    quantise_row<T>(row, a.d, a.cache, which[k] - 1, slot, hd[k], lane);
                    __syncwarp();
                }
            }
        }
    }
}

// Backward.  CTAs [0, nq) take q, the others k, so that a thread's sums for dw
// belong to one weight; each CTA writes its partial row [d].
template <typename T, int S>
__global__ void __launch_bounds__(kHeadWarps * 32)
head_bwd_scalar_kernel(const __grid_constant__ HeadArgs a, int nq) {
    constexpr int R = 4 / S;  // rows of a warp under way
    __shared__ float part[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = int(blockIdx.x) < nq ? 0 : 1;
    const int cta = int(blockIdx.x) - (which ? nq : 0);
    const int ctas = which ? int(gridDim.x) - nq : nq;
    const int slots = (a.d + 1) >> 1, heads = a.heads[which];
    pdl_next();
    const SlotSteps<S> steps(a.rope, lane);
    SlotAt e[S];
    float w0[S], w1[S], acc_u[S], acc_v[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        e[s] = slot_at(lane + 32 * s, a.d, a.rope);
        w0[s] = w1[s] = 1.f;
        acc_u[s] = acc_v[s] = 0.f;
        if (a.w[which] && lane + 32 * s < slots) {
            w0[s] = ld_elem<T>(a.w[which], e[s].e0);
            if (e[s].e1 < a.d) w1[s] = ld_elem<T>(a.w[which], e[s].e1);
        }
    }
    for (int64_t t = cta; t < a.tokens; t += ctas) {
        float2 cs[S];
        steps.make(a.rope, lane, t, cs);
        for (int h0 = warp; h0 < heads; h0 += kHeadWarps * R) {
            float u[R][S], v[R][S], gu[R][S], gv[R][S], r[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const int h = h0 + k * kHeadWarps;
                const T* x = reinterpret_cast<const T*>(a.x[which].p) + t * a.x[which].ts + h * a.x[which].hs;
                const T* dy = reinterpret_cast<const T*>(a.dy[which].p) + t * a.dy[which].ts + h * a.dy[which].hs;
                r[k] = h < heads ? a.rstd[which][t * heads + h] : 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    u[k][s] = v[k][s] = gu[k][s] = gv[k][s] = 0.f;
                    if (h < heads && lane + 32 * s < slots) {
                        u[k][s] = ld_elem<T>(x, e[s].e0);
                        gu[k][s] = ld_elem<T>(dy, e[s].e0);
                        if (e[s].e1 < a.d) {
                            v[k][s] = ld_elem<T>(x, e[s].e1);
                            gv[k][s] = ld_elem<T>(dy, e[s].e1);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float sum = 0.f;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (e[s].turns) turn(gu[k][s], gv[k][s], cs[s]);
                    acc_u[s] = fmaf(gu[k][s], u[k][s] * r[k], acc_u[s]);
                    acc_v[s] = fmaf(gv[k][s], v[k][s] * r[k], acc_v[s]);
                    gu[k][s] *= w0[s];
                    gv[k][s] *= w1[s];
                    sum = fmaf(gu[k][s], u[k][s], fmaf(gv[k][s], v[k][s], sum));
                }
                const float f = warp_sum(sum) / float(a.d) * r[k] * r[k] * r[k];
                const int h = h0 + k * kHeadWarps;
                T* dx = reinterpret_cast<T*>(a.y[which].p) + t * a.y[which].ts + h * a.y[which].hs;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    if (h < heads && lane + 32 * s < slots) {
                        st_elem<T>(dx, e[s].e0, fmaf(-u[k][s], f, gu[k][s] * r[k]));
                        if (e[s].e1 < a.d) st_elem<T>(dx, e[s].e1, fmaf(-v[k][s], f, gv[k][s] * r[k]));
                    }
                }
            }
        }
    }
    if (a.ws == nullptr) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (lane + 32 * s < slots) {
            part[warp][e[s].e0] = acc_u[s];
            if (e[s].e1 < a.d) part[warp][e[s].e1] = acc_v[s];
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
// rounding error along (Neumaier's sum).  2.5 us after the backward, most of it
// launch and the first loads; a tree of float pairs over the warps was no faster.
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
head_dw_kernel(const float* ws, int d, int nq, int nk, T* dwq, T* dwk) {
    pdl_next();
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
            tot.c += part[w][1][lane];
        }
        st_elem<T>(out, col, tot.s + tot.c);
    }
}

// ---------------------------------------------------------------------------
// cache rows: one row per warp
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kHeadWarps * 32)
cache_write_scalar_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads) {
    __shared__ float stage[kHeadWarps][kHeadMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.x[1].p ? int(blockIdx.y) : 1;
    const HeadView xv = a.x[1 + which];
    float* row = stage[warp];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    pdl_next();
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = row_div(i, by_heads);
        const int h = int(i - t * heads);
        const int64_t slot = cache_slot(a.cache, ld_after(a.slots + t), a.err);
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
cache_read_scalar_kernel(const __grid_constant__ HeadArgs a, RowDiv by_heads) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = a.y[0].p ? int(blockIdx.y) : 1;
    const HeadView yv = a.y[which];
    const int heads = a.heads[1];
    const int64_t rows = a.tokens * heads;
    pdl_next();
    for (int64_t i = int64_t(blockIdx.x) * kHeadWarps + warp; i < rows; i += int64_t(gridDim.x) * kHeadWarps) {
        const int64_t t = row_div(i, by_heads);
        const int h = int(i - t * heads);
        const int64_t slot = cache_slot(a.cache, ld_after(a.slots + t), a.err);
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

// Chunks (as a power of two) that a token's `steps` row steps are split into: one
// while tokens alone give every SM `warps` warps, else as many as that takes.
inline int head_chunks_log2(int64_t tokens, int steps, int warps, const DevInfo& d) {
    int lc = 0;
    while ((1 << lc) < steps && (tokens << lc) < int64_t(warps) * d.sms) ++lc;
    return lc;
}

// The grid for `work` CTAs' worth of single units, of which `resident` run at once.
inline int64_t make_waves(int64_t work, int64_t resident, Waves* w) {
    w->ctas = int(std::min(work, resident));
    const int64_t all = (work + w->ctas - 1) / w->ctas;  // rounds
    const int64_t waves = std::min((all + kWaveRounds - 1) / kWaveRounds, int64_t(1) << 16);
    w->rounds = int((all + waves - 1) / waves);
    const int64_t full = work / (int64_t(w->ctas) * w->rounds);
    return full * w->ctas + std::min(work - full * w->ctas * w->rounds, int64_t(w->ctas));
}

// Tokens (as a power of two) that share a warp's rows where a token's `heads` heads
// leave some of the 32 >> lg free, and tokens are many enough to fill the SMs so
// (f16, 21209 tokens of 1 + 1 heads of 64: 31 us with a token a warp, 9 so).
inline int head_tokens_log2(int64_t tokens, int heads, int lg, const DevInfo& d) {
    int lt = 0;
    while (lt < 5 - lg && heads <= (32 >> lg) >> (lt + 1) && tokens >> (lt + 1) >= int64_t(8) * d.sms) ++lt;
    return lt;
}

// f of the conditions as constants.
template <typename F>
const void* pick(F&& f) {
    return f();
}
template <typename F, typename... More>
const void* pick(F&& f, bool first, More... more) {
    return first ? pick([&](auto... rest) { return f(std::true_type{}, rest...); }, more...)
                 : pick([&](auto... rest) { return f(std::false_type{}, rest...); }, more...);
}

template <typename T, int VE>
nrm_status head_fwd_vec(const HeadArgs& a, bool norm, bool cache, const DevInfo& d, cudaStream_t s) {
    int lg = row_lanes_log2(a.d / (2 * VE));
    int lt = head_tokens_log2(a.tokens, (std::max(a.heads[0], a.heads[1]) + kHeadRows - 1) / kHeadRows, lg, d);
    const void* fn = pick([](auto adj, auto with_cache, auto many, auto with_norm) {
        return (const void*)&head_fwd_vec_kernel<T, VE, adj.value, with_cache.value, many.value, with_norm.value>;
    }, bool(a.rope.adjacent), cache, lt > 0, norm);
    const size_t smem = head_fwd_smem<T, VE>();
    if (nrm_status st = prepare_kernel(fn, smem, false); st != NRM_OK) return st;
    const int occ = cached_occupancy(fn, kHeadFwdWarps * 32, smem);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head forward kernel cannot be resident");
    const int per = (32 >> lg >> lt) * kHeadRows;
    int steps = 0;
    for (int i = 0; i < (cache ? 3 : 2); ++i) steps += (a.heads[i] + per - 1) / per;
    const int64_t blocks = (a.tokens + (1 << lt) - 1) >> lt;
    int lc = head_chunks_log2(blocks, steps, 16, d);
    Waves waves{};
    const int64_t ctas = make_waves(((blocks << lc) + kHeadFwdWarps - 1) / kHeadFwdWarps, int64_t(occ) * d.sms, &waves);
    HeadArgs args = a;
    void* kargs[] = {&args, &lg, &lt, &lc, &waves};
    return launch_pdl(fn, dim3(unsigned(ctas)), dim3(kHeadFwdWarps * 32), kargs, s, smem);
}

// f of the slots that a lane of a scalar kernel holds: 1, 2 or 4 for d up to 64, 128, 256.
template <typename F>
const void* pick_slots(int d, F&& f) {
    if (d <= 64) return f(std::integral_constant<int, 1>{});
    if (d <= 128) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 4>{});
}

template <typename T>
nrm_status head_fwd_scalar(const HeadArgs& a, bool norm, bool cache, const DevInfo& d, cudaStream_t s) {
    int rows = 0;
    const void* fn = pick_slots(a.d, [&](auto n) {
        rows = 4 / n.value * kHeadWarps;
        return cache ? (const void*)&head_fwd_scalar_kernel<T, n.value, true>
                     : (const void*)&head_fwd_scalar_kernel<T, n.value, false>;
    });
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head forward kernel cannot be resident");
    const int64_t cap = int64_t(occ) * d.sms;
    const int heads = a.heads[0] + a.heads[1] + (cache ? a.heads[2] : 0);
    // few tokens: their heads are split over CTAs
    const int64_t gx = a.tokens < cap ? a.tokens : cap;
    int64_t gy = (heads + rows - 1) / rows;
    if (gy > (cap + gx - 1) / gx) gy = (cap + gx - 1) / gx;
    HeadArgs args = a;
    int with_norm = norm;
    void* kargs[] = {&args, &with_norm};
    return launch_pdl(fn, dim3(unsigned(gx), unsigned(gy)), dim3(kHeadWarps * 32), kargs, s);
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
    if constexpr (sizeof(T) == 2)
        if (vec == 4) return head_fwd_vec<T, 2>(args, norm, cache, *d, s);
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
    BwdPlan plan{};
    plan.lg = vec ? row_lanes_log2(a.d * int(sizeof(T)) / (2 * vec)) : 5;
    // CTAs go to q and k by what they cost: a token's row steps, and one more for its angles
    int steps[2];
    int64_t blocks[2], units[2];
    for (int i = 0; i < 2; ++i) {
        plan.ltok[i] = vec ? head_tokens_log2(a.tokens, a.heads[i], plan.lg, *d) : 0;
        const int per = vec ? 32 >> plan.lg >> plan.ltok[i] : kHeadWarps;
        steps[i] = (a.heads[i] + per - 1) / per;
        blocks[i] = (a.tokens + (1 << plan.ltok[i]) - 1) >> plan.ltok[i];
    }
    plan.lchunk = vec ? head_chunks_log2(a.tokens, std::max(steps[0], steps[1]), 8, *d) : 0;
    for (int i = 0; i < 2; ++i)
        units[i] = a.heads[i] == 0 ? 0 : (vec ? ((blocks[i] << plan.lchunk) + kHeadWarps - 1) / kHeadWarps : blocks[i]);
    const void* fn = pick_slots(a.d, [](auto n) { return (const void*)&head_bwd_scalar_kernel<T, n.value>; });
    size_t smem = 0;
    auto take = [&](auto ve) {
        constexpr int VE = decltype(ve)::value;
        fn = pick([](auto adj, auto many) {
            return (const void*)&head_bwd_vec_kernel<T, VE, adj.value, many.value>;
        }, bool(a.rope.adjacent), plan.ltok[0] > 0 || plan.ltok[1] > 0);
        smem = head_bwd_smem<T, VE>();
    };
    if (vec == 16) take(std::integral_constant<int, 16 / int(sizeof(T))>{});
    if (vec == 8) take(std::integral_constant<int, 8 / int(sizeof(T))>{});
    if constexpr (sizeof(T) == 2)
        if (vec == 4) take(std::integral_constant<int, 2>{});
    if (smem)
        if (nrm_status st = prepare_kernel(fn, smem, false); st != NRM_OK) return st;
    const int occ = cached_occupancy(fn, kHeadWarps * 32, smem);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "head backward kernel cannot be resident");
    int64_t cap = int64_t(occ) * d->sms;
    if (cap > head_bwd_max_partials(*d)) cap = head_bwd_max_partials(*d);
    int64_t cq = cap, ck = 0;
    if (a.heads[1]) {
        const double cost[2] = {double(blocks[0]) * (steps[0] + 1), double(blocks[1]) * (steps[1] + 1)};
        ck = std::min(std::max(int64_t(double(cap) * (cost[1] / (cost[0] + cost[1]))), int64_t(1)), cap - 1);
        cq = cap - ck;
    }
    plan.nq = int(std::min(cq, units[0]));
    int nq = plan.nq, nk = int(std::min(ck, units[1]));
    HeadArgs args = a;
    void* kargs_vec[] = {&args, &plan};
    void* kargs[] = {&args, &nq};
    nrm_status st = launch_pdl(fn, dim3(unsigned(nq + nk)), dim3(kHeadWarps * 32), vec ? kargs_vec : kargs, s, smem);
    if (st != NRM_OK || a.ws == nullptr) return st;
    const float* ws = a.ws;
    int dd = a.d;
    T* dwq = reinterpret_cast<T*>(a.dw[0]);
    T* dwk = reinterpret_cast<T*>(a.dw[1]);
    void* sargs[] = {&ws, &dd, &nq, &nk, &dwq, &dwk};
    return launch_pdl((const void*)&head_dw_kernel<T>, dim3(unsigned(a.d + 31) / 32, 2), dim3(kHeadSumWarps * 32),
                      sargs, s);
}

// A row to each warp: any layout.
template <typename T>
nrm_status cache_launch_scalar(const HeadArgs& a, const void* fn, bool both, const DevInfo& d, cudaStream_t s) {
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "cache kernel cannot be resident");
    const int64_t rows = a.tokens * a.heads[1];
    int64_t ctas = (rows + kHeadWarps - 1) / kHeadWarps;
    if (ctas > int64_t(occ) * d.sms) ctas = int64_t(occ) * d.sms;
    HeadArgs args = a;
    RowDiv by_heads = make_row_div(a.heads[1], rows);
    void* kargs[] = {&args, &by_heads};
    return launch_pdl(fn, dim3(unsigned(ctas), both ? 2 : 1), dim3(kHeadWarps * 32), kargs, s);
}

// `lanes` lanes of a row hold vectors, `gl` of them a group.
inline nrm_status cache_launch_vec(const HeadArgs& a, const void* fn, int lanes, int gl, bool wide, const DevInfo& d,
                                   cudaStream_t s) {
    const int occ = cached_occupancy(fn, kHeadWarps * 32, 0);
    if (occ <= 0) return fail(NRM_ERR_CUDA, "cache kernel cannot be resident");
    CacheLanes cl{};
    cl.lg = row_lanes_log2(lanes);
    cl.per = lanes;
    cl.gl = gl;
    cl.wide = wide;
    while (cl.lhp < 5 - cl.lg && (1 << cl.lhp) < a.heads[1]) ++cl.lhp;
    const int ltok = 5 - cl.lg - cl.lhp;
    const int64_t blocks = (a.tokens + (1 << ltok) - 1) >> ltok;
    cl.lchunk = head_chunks_log2(blocks, (a.heads[1] + (1 << cl.lhp) - 1) >> cl.lhp, 16, d);
    Waves waves{};
    const int64_t ctas = make_waves(((blocks << cl.lchunk) + kHeadWarps - 1) / kHeadWarps, int64_t(occ) * d.sms, &waves);
    HeadArgs args = a;
    void* kargs[] = {&args, &cl, &waves};
    return launch_pdl(fn, dim3(unsigned(ctas)), dim3(kHeadWarps * 32), kargs, s);
}

// Whether rows start on 32 bytes in every given view.
template <typename T>
bool rows_on_32(const HeadView (&views)[2], int64_t tokens, int heads) {
    constexpr int64_t n = 32 / int64_t(sizeof(T));
    for (const HeadView& v : views)
        if (v.p && (reinterpret_cast<uintptr_t>(v.p) % 32 || (tokens > 1 && v.ts % n) || (heads > 1 && v.hs % n)))
            return false;
    return true;
}

// The kernel of a stored form: f of the form as a constant.
template <typename F>
const void* cache_kind(int kind, F&& f) {
    if (kind == NRM_CACHE_E4M3) return f(std::integral_constant<int, NRM_CACHE_E4M3>{});
    if (kind == NRM_CACHE_INT8) return f(std::integral_constant<int, NRM_CACHE_INT8>{});
    return f(std::integral_constant<int, NRM_CACHE_INT4>{});
}

// Two vectors of a row to a lane, where every group is whole lanes; else one,
// where a warp holds the row.
template <typename T, int BYTES>
nrm_status cache_write_vec(const HeadArgs& a, const DevInfo& d, cudaStream_t s) {
    constexpr int VE = BYTES / int(sizeof(T));
    const int nvec = a.d / VE, gv = a.cache.group / VE;
    auto by_kind = [&](auto f) { return cache_kind(a.cache.kind, f); };
    const HeadView views[2] = {a.x[1], a.x[2]};
    if (gv % 2 == 0)
        return cache_launch_vec(a, by_kind([](auto kind) {
                                    return (const void*)&cache_write_vec_kernel<T, VE, 2, decltype(kind)::value>;
                                }), nvec / 2, gv / 2,
                                rows_on_32<T>(views, a.tokens, a.heads[1]), d, s);
    if (nvec <= 32)
        return cache_launch_vec(a, by_kind([](auto kind) {
                                    return (const void*)&cache_write_vec_kernel<T, VE, 1, decltype(kind)::value>;
                                }), nvec, gv, false, d, s);
    return cache_launch_scalar<T>(a, (const void*)&cache_write_scalar_kernel<T>, a.x[1].p && a.x[2].p, d, s);
}

template <typename T>
nrm_status cache_write(const HeadArgs& a, int vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    HeadArgs args = a;
    args.err = d->err;
    if (vec == 16) return cache_write_vec<T, 16>(args, *d, s);
    if (vec == 8) return cache_write_vec<T, 8>(args, *d, s);
    if constexpr (sizeof(T) == 2)
        if (vec == 4) return cache_write_vec<T, 4>(args, *d, s);
    return cache_launch_scalar<T>(args, (const void*)&cache_write_scalar_kernel<T>, a.x[1].p && a.x[2].p, *d, s);
}

template <typename T>
nrm_status cache_read(const HeadArgs& a, int vec, cudaStream_t s) {
    const DevInfo* d = dev_info();
    if (!d) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    if (a.tokens == 0) return NRM_OK;
    HeadArgs args = a;
    args.err = d->err;
    const void* fn = nullptr;
    auto take = [&](auto ve) {
        fn = cache_kind(a.cache.kind, [](auto kind) {
            return (const void*)&cache_read_vec_kernel<T, decltype(ve)::value, decltype(kind)::value>;
        });
    };
    if (vec == 16) take(std::integral_constant<int, 16 / int(sizeof(T))>{});
    if (vec == 8) take(std::integral_constant<int, 8 / int(sizeof(T))>{});
    if constexpr (sizeof(T) == 2)
        if (vec == 4) take(std::integral_constant<int, 2>{});
    if (fn) return cache_launch_vec(args, fn, a.d * int(sizeof(T)) / (2 * vec), 0, false, *d, s);
    return cache_launch_scalar<T>(args, (const void*)&cache_read_scalar_kernel<T>, a.y[0].p && a.y[1].p, *d, s);
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
