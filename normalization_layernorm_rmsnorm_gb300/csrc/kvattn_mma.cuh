// kvattn_mma.cuh -- the attention over the cache on matrix instructions.
//
// Both products are m16n8k16 with fp16 factors and fp32 sums, the query heads of
// a pair as the eight columns: logits = codes of 16 keys [16 x d] * queries [d x
// 8], and out^T = codes of 16 values [d x 16] * weights [16 x 8].  A code is
// exact in fp16 in every stored form; the keys' scales multiply the logits, the
// values' the weights.  Queries are scaled by a power of two to at most 2^15: those
// of 16 bits then are exact, of float32 ones the rest is a second factor (22 bits).
//
// (An integer could be taken as it lies, as one of fp16's smallest numbers, with a
// bias that one more product takes off again, which saves its conversion: 131072
// positions in 4 bits 58 us instead of 60.  But an instruction lines its terms up
// by the exponents that their factors are stored with and cuts them off at 2^-25 of
// the largest, and the smallest numbers are stored with 2^-14: terms then end at
// 2^-15 of a code's step times the largest weight, so that where the position that
// draws the weight has a code of 0, what the others give is off.)
//
// A weight is p times its value's scale, multiplied in float32 with the largest
// scale seen brought below 2^15 and rounded to fp16: 11 bits down to 2^-28 of the
// largest p times the largest scale, nothing below 2^-39.  (The bounds are the
// product's alone: a p or a scale far below the largest keeps its bits as long as
// the product does.)  bfloat16 outputs, whose significand has 8 bits, take that;
// where the output has more (fp16, float32), what the rounding left off is a
// second factor, 2^11 times as large, with a sum of its own in each tile: 22 bits
// down to 2^-28, nothing below 2^-50.  (Two factors of one size end at one
// place: below 2^-20 the second is 0.)
//
// The order of the d elements in a product is free, so a lane takes its keys'
// elements as they lie in 8 (or 4) neighbours, and its values' in 4 (or 2).
//
// The columns' heads are the lanes' pairs in both results, so the running
// maximum, the rescaling and the sum need nothing from other lanes but the
// maximum over the positions; weights change from rows to columns by a
// transposing exchange of 8x8 matrices.
//
// Codes and scales are copied asynchronously into the warp's own ring in shared
// memory, a tile of 32 positions at a time: its keys while the values before them are
// worked on, and its values while the keys are; warps share nothing and the loop
// holds no barrier of the CTA.  (Two whole stages leave room for 10 warps, whose
// waits then show.)  The row of a page is found by the lane of its position, a tile
// ahead.  Rows are padded so that the fragments' reads have no conflicts.
// (Bulk copies of single rows are no way to move them: one takes an SM about ten
// cycles, 1.8 TB/s with rows of 64 bytes and 3.7 with 128, against 3.5 and 6.2 by
// 16-byte copies that eight lanes make of a row.)
#pragma once

#include "kvattn.cuh"

namespace nrm {

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// n bytes, and zeros for the rest.
__device__ __forceinline__ void cp_async_8_or_0(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_16_or_0(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_4_or_0(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8x8 matrix of 16-bit elements spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Shared memory at byte `at` of the CTA's ring.
template <typename R>
__device__ __forceinline__ R& in_ring(uint32_t at) {
    extern __shared__ __align__(128) unsigned char attn_ring[];
    return *reinterpret_cast<R*>(attn_ring + at);
}
template <int BYTES>
__device__ __forceinline__ uint32_t lds(uint32_t at) {
    if constexpr (BYTES == 4) return in_ring<const uint32_t>(at);
    else if constexpr (BYTES == 2) return in_ring<const uint16_t>(at);
    else return in_ring<const uint8_t>(at);
}

// Codes as pairs of fp16.
__device__ __forceinline__ uint32_t e4m3x2_halves(uint32_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
    return h;
}
// Integers as fp16: behind the upper byte of 1024 a code (plus 2^7 or 2^3, so that it is not negative) adds its own
// value, and a subtraction takes off what was added.
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr uint32_t kHalf1024 = 0x64006400u, kHalf1032 = 0x64086408u, kHalf1152 = 0x64806480u;  // twice each
// Four 8-bit codes: bytes (0, 1) and (2, 3).
template <int KIND>
__device__ __forceinline__ void codes8(uint32_t v, uint32_t& lo, uint32_t& hi) {
    if constexpr (KIND == NRM_CACHE_E4M3) {
        lo = e4m3x2_halves(v);
        hi = e4m3x2_halves(v >> 16);
    } else {
        v ^= 0x80808080u;
        lo = sub_half2(__byte_perm(v, kHalf1024, 0x7170), kHalf1152);
        hi = sub_half2(__byte_perm(v, kHalf1024, 0x7372), kHalf1152);
    }
}
// The 4-bit codes (plus 8) at the low ends of both halves, and those above, 16 times as large.
__device__ __forceinline__ uint32_t codes4(uint32_t v) { return sub_half2((v & 0x000f000fu) | kHalf1024, kHalf1032); }
__device__ __forceinline__ uint32_t codes4_next(uint32_t v) { return sub_half2((v & 0x00f000f0u) | kHalf1024, kHalf1152); }

// What a kernel is made for: the stored form, rows of UNITS units of 128, 64, 32 or 16 elements (every group is whole
// units; EXACT: of no fewer), and eights of heads.  With the count known the products of a tile are one block of
// instructions, which the loops' ends would cut in pieces too short to fill the waits.
template <int KIND_, int UNIT_, int UNITS_, int NT_, bool EXACT_ = true>
struct AttnForm {
    static constexpr int KIND = KIND_, UNIT = UNIT_, UNITS = UNITS_, NT = NT_, DMAX = UNIT * UNITS;
    static constexpr bool EXACT = EXACT_;
    // keys are read in units of 32 at most, of which a lane has KP elements; values in whole units, VP elements a lane
    static constexpr int SUB = UNIT < 32 ? UNIT : 32, SUBS = UNIT / SUB, STEPS = SUB / 16, TILES = UNIT / 16;
    static constexpr int KP = SUB / 4, VP = UNIT / 8;
    static constexpr int BITS = KIND == NRM_CACHE_INT4 ? 4 : 8;
    static constexpr int ROW = DMAX * BITS / 8;
    static constexpr int CHUNKS = ROW % 16 == 0 ? ROW / 16 : 0;  // 16-byte vectors of a row
    // rows in shared memory: an odd number of 32 bytes (a key's fragment of 8 bytes a lane, 4 rows at a time) or of 16
    // (else) apart, the fragments' reads meet no bank twice
    static constexpr int K_UNIT = BITS == 8 && SUB == 32 ? 32 : 16;
    static constexpr int K_PITCH = ((ROW + K_UNIT - 1) / K_UNIT | 1) * K_UNIT, V_PITCH = ((ROW + 15) / 16 | 1) * 16;
    static constexpr uint32_t V_AT = 32 * K_PITCH, S_AT = V_AT + 32 * V_PITCH;
};

// A warp's shared memory: a tile's keys, values and scales of both, the places of a tile's rows, and its scales of each
// unit.
struct AttnSmem {
    uint32_t codes;            // keys, values
    uint32_t scales;           // [keys, values][32][groups]
    uint32_t places;           // [32] code offsets
    uint32_t k_scales;         // [units][32]
    uint32_t v_scales;         // [units][32], the largest brought below 2^15
};
constexpr uint32_t kAttnPlaces = 32 * 8;
// Warps of a CTA, by the registers that a thread needs.  (12: 131072 positions in 4 bits take 60 us; 10: 68; 14, with
// 144 registers: 70; 16, with 128: 66.)
template <typename F>
constexpr int kAttnFormWarps = F::DMAX > 128 || F::NT > 1 ? 8 : kAttnWarps;
template <typename T>
constexpr int kAttnFactors = std::is_same_v<T, __nv_bfloat16> ? 1 : 2;  // of a weight
template <typename F>
__host__ __device__ constexpr uint32_t attn_warp_bytes(int groups) {
    return F::S_AT + 2 * 32 * groups * 4 + kAttnPlaces + 2 * F::UNITS * 128;
}

template <typename T, typename F>
__device__ __forceinline__ void attn_mma_piece(const AttnArgs& a, const AttnPiece& p, const AttnSmem& sm, int groups) {
    using bits = typename Io<T>::bits_t;
    constexpr int NT = F::NT, QT = sizeof(T) == 4 ? 2 : 1, WT = kAttnFactors<T>;
    constexpr int KSTEPS = F::DMAX / 16;
    const int lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
    const int units = F::EXACT ? F::UNITS : a.d / F::UNIT;
    int of_unit[F::UNITS];  // a unit's scale in its row's, in bytes
#pragma unroll
    for (int u = 0; u < F::UNITS; ++u) of_unit[u] = u * F::UNIT / a.cache.group * 4;

    // ---- the copies ----
    const int64_t j0 = p.lo + int64_t(p.tile0) * kAttnTile;
    const int64_t j1 = min(p.n, p.lo + int64_t(p.tile1) * kAttnTile);
    const int tiles = p.tile1 - p.tile0;
    const uint32_t ring = smem_addr(&in_ring<unsigned char>(0));
    const int64_t* const table = a.table + p.s * a.table_stride;
    int64_t page = 0, in_page = 0;
    auto look_up = [&](int64_t j) {  // this lane's position of a tile (in_page -1: there is none)
        j += lane;
        in_page = -1;
        if (j < j1) {
            const int64_t entry = row_div(j, a.cache.page);
            in_page = j - entry * a.cache.page.d;
            page = ld_after(table + entry);
        }
    };
    // the rows of keys (0) or values (1) at the places in shared memory; one that is not there becomes zeros
    auto copy_rows = [&](auto which, uint32_t m) {
        constexpr int W = decltype(which)::value, PITCH = W ? F::V_PITCH : F::K_PITCH;
        const uint32_t to = ring + sm.codes + (W ? F::V_AT : 0);
        const uint8_t* codes = a.cache.codes[W];
        if (F::EXACT && F::CHUNKS > 0 && a.near) {
            // places in 16 bytes; neighbouring lanes copy neighbouring vectors of a row
            constexpr int C = F::CHUNKS > 0 ? F::CHUNKS : 1;
            auto from = [&](int r, int c) { return codes + uint64_t(in_ring<const uint32_t>(sm.places + r * 4)) * 16 + c * 16; };
            if (m == 0xffffffffu) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    const int r = (i * 32 + lane) / C, c = (i * 32 + lane) % C;
                    cp_async_16(to + r * PITCH + c * 16, from(r, c));
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < C; ++i) {
                    const int r = (i * 32 + lane) / C, c = (i * 32 + lane) % C;
                    cp_async_16_or_0(to + r * PITCH + c * 16, from(r, c), int(m >> r << 4) & 16);
                }
            }
        } else {
            const int chunks = a.row_bytes / a.vec, row_step = 32 / chunks, chunk_step = 32 - row_step * chunks;
            int row = lane / chunks, chunk = lane - row * chunks;
#pragma unroll 1
            for (int i = 0; i < chunks; ++i) {
                const int64_t at = in_ring<const int64_t>(sm.places + row * 8) + chunk * a.vec;
                const int n = m >> row & 1 ? a.vec : 0;
                if (a.vec == 16) cp_async_16_or_0(to + row * PITCH + chunk * 16, codes + at, n);
                else cp_async_8_or_0(to + row * PITCH + chunk * 8, codes + at, n);
                row += row_step;
                chunk += chunk_step;
                if (chunk >= chunks) {
                    chunk -= chunks;
                    ++row;
                }
            }
        }
    };
    // the places of the tile that was looked up, its keys and the scales of both; which positions are there
    auto issue_keys = [&]() -> uint32_t {
        const bool ok = in_page >= 0 && uint64_t(page) < uint64_t(a.pages);
        if (in_page >= 0 && !ok) atomicOr(a.err, kErrCacheSlot);
        const uint32_t m = __ballot_sync(0xffffffffu, ok);
        int64_t code = 0, scale = 0;
        if (ok) {
            code = page * a.cache.page_stride + in_page * a.cache.slot_stride + p.head * a.cache.head_stride;
            scale = page * a.cache.scale_page_stride + in_page * a.cache.scale_slot_stride + p.head * a.cache.scale_head_stride;
        }
        if (F::EXACT && F::CHUNKS > 0 && a.near) in_ring<uint32_t>(sm.places + lane * 4) = uint32_t(code >> 4);
        else in_ring<int64_t>(sm.places + lane * 8) = code;
        __syncwarp();
        copy_rows(std::integral_constant<int, 0>{}, m);
        const uint32_t ks = ring + sm.scales + lane * groups * 4, vs = ks + 32 * groups * 4;
        const float *kf = a.cache.scales[0] + scale, *vf = a.cache.scales[1] + scale;
        if (a.scale_vec) {
#pragma unroll 1
            for (int g = 0; g < groups; g += 4) {
                cp_async_16_or_0(ks + g * 4, kf + g, ok ? 16 : 0);
                cp_async_16_or_0(vs + g * 4, vf + g, ok ? 16 : 0);
            }
        } else {
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                cp_async_4_or_0(ks + g * 4, kf + g, ok ? 4 : 0);
                cp_async_4_or_0(vs + g * 4, vf + g, ok ? 4 : 0);
            }
        }
        return m;
    };
    look_up(j0);
    uint32_t there = issue_keys(), next_there = 0;
    cp_async_commit();
    copy_rows(std::integral_constant<int, 1>{}, there);
    cp_async_commit();
    look_up(j0 + kAttnTile);

    // ---- the queries, while the first copies are under way ----
    uint32_t q[KSTEPS][NT][QT][2];
    float factor[NT][2];  // of the logits of this lane's two heads
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + gid;
        const bits* row = static_cast<const bits*>(a.q.p) + p.s * a.q.ts + (p.q0 + h) * a.q.hs;
        float x[F::DMAX / F::SUB][F::KP], most = 0.f;
#pragma unroll
        for (int u = 0; u < F::DMAX / F::SUB; ++u) {
            const int at = u * F::SUB + tid * F::KP;
            const bool there = h < p.heads && (F::EXACT || u < units);
            if (there && a.q_vec) {
                constexpr int B = F::KP * int(sizeof(T));  // 8, 16 or 32 bytes
                uint32_t w[B / 4];
#pragma unroll
                for (int b = 0; b < B; b += 16) {
                    if constexpr (B >= 16) {
                        const uint4 v = ld_after(reinterpret_cast<const uint4*>(row + at) + b / 16);
                        w[b / 4] = v.x, w[b / 4 + 1] = v.y, w[b / 4 + 2] = v.z, w[b / 4 + 3] = v.w;
                    } else {
                        const uint2 v = ld_after(reinterpret_cast<const uint2*>(row + at));
                        w[0] = v.x, w[1] = v.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < F::KP; ++i)
                    x[u][i] = sizeof(T) == 4 ? __uint_as_float(w[i % (B / 4)])
                                             : Io<T>::load(typename Io<T>::bits_t(w[i / 2 % (B / 4)] >> (16 * (i & 1))));
            } else {
#pragma unroll
                for (int i = 0; i < F::KP; ++i) x[u][i] = there ? Io<T>::load(ld_after(row + at + i)) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < F::KP; ++i) most = fmaxf(most, fabsf(x[u][i]));
        }
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // 2^e > most (an infinity stays one); float32's smallest number times `up` is 2^-23, which fp16 holds
        const int e = max(-111, min(128, int(__float_as_uint(most) >> 23) - 126));
        const float up = __uint_as_float(uint32_t(127 + 15 - e) << 23);
        const float down = __uint_as_float(uint32_t(127 - 15 + e) << 23) * a.scale_log2;
        factor[nt][0] = __shfl_sync(0xffffffffu, down, tid * 8);
        factor[nt][1] = __shfl_sync(0xffffffffu, down, tid * 8 + 4);
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ++ks) {
            const int u = ks / F::STEPS, part = ks % F::STEPS;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                // the elements that a fragment of codes pairs
                const int i0 = F::BITS == 8 ? part * 4 + b * 2 : part * 2 + b;
                const int i1 = F::BITS == 8 ? i0 + 1 : i0 + F::KP / 2;
                // the codes of the second pair of four lie 16 times as large
                const float by = F::BITS == 4 && b == 1 ? up * 0x1p-4f : up;
                const float lo = x[u][i0] * by, hi = x[u][i1] * by;
                q[ks][nt][0][b] = half2_bits(lo, hi);
                if constexpr (QT == 2) {
                    const float2 r = half2_floats(q[ks][nt][0][b]);
                    q[ks][nt][QT - 1][b] = half2_bits(lo - r.x, hi - r.y);
                }
            }
        }
    }

    // ---- the running softmax ----
    float acc[F::UNITS][F::TILES][NT][4], m[NT][2], sum[NT][2];
    int top[F::UNITS];  // the values' largest scale so far (its size: one may be negative) is below 2^top
#pragma unroll
    for (int u = 0; u < F::UNITS; ++u) {
        top[u] = -1000;
#pragma unroll
        for (int t = 0; t < F::TILES; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[u][t][nt][i] = 0.f;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, sum[nt][0] = sum[nt][1] = 0.f;

    for (int tile = 0; tile < tiles; ++tile) {
        cp_async_wait<1>();  // the keys and the scales
        __syncwarp();

        // the scales of this lane's position, of each unit; seldom a value's is larger than all before it, or a key's
        // so large that its product with the codes' sum, which is below 2^32, might leave float32 although the logit
        // does not
        constexpr float kHuge = 0x1p90f, kLess = 0x1p-64f;
        bool huge = false;
        {
            const uint32_t mine = sm.scales + (32 + lane) * groups * 4;
            float mine_of[F::UNITS], k_of[F::UNITS], k_by = 1.f;
            bool larger = false;
#pragma unroll
            for (int u = 0; u < F::UNITS; ++u) {
                if (!F::EXACT && u >= units) break;
                mine_of[u] = in_ring<const float>(mine + of_unit[u]);
                k_of[u] = in_ring<const float>(mine - 32 * groups * 4 + of_unit[u]);
                huge |= fabsf(k_of[u]) >= kHuge;
                larger |= fabsf(mine_of[u]) >= (top[u] < -126 ? -1.f : __uint_as_float(uint32_t(127 + top[u]) << 23));
            }
            larger |= huge;
            if (__any_sync(0xffffffffu, larger)) {
                huge = __any_sync(0xffffffffu, huge);
                if (huge) k_by = kLess;
#pragma unroll
                for (int u = 0; u < F::UNITS; ++u) {
                    if (!F::EXACT && u >= units) break;
                    const uint32_t b = __float_as_uint(mine_of[u]) & 0x7fffffffu;
                    const uint32_t most = __reduce_max_sync(0xffffffffu, b < 0x7f800000u ? b : 0u);
                    const int now = max(max(top[u], -100), int(most >> 23) - 126);
                    const float raise = exp2f(float(max(top[u] - now, -126)));
                    top[u] = now;
#pragma unroll
                    for (int t = 0; t < F::TILES; ++t)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[u][t][nt][i] *= raise;
                }
            }
#pragma unroll
            for (int u = 0; u < F::UNITS; ++u) {
                if (!F::EXACT && u >= units) break;
                in_ring<float>(sm.v_scales + (u * 32 + lane) * 4) = mine_of[u] * __uint_as_float(uint32_t(127 + 15 - top[u]) << 23);
                in_ring<float>(sm.k_scales + (u * 32 + lane) * 4) = k_of[u] * k_by;
            }
            __syncwarp();
        }

        // logits of positions gid, gid + 8, gid + 16 and gid + 24: [half of the tile][head, head + 1, 8 further]
        float l[2][NT][4];
#pragma unroll
        for (int u = 0; u < F::UNITS; ++u) {
            if (!F::EXACT && u >= units) break;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
                for (int sub = 0; sub < F::SUBS; ++sub) {
                    uint32_t f[F::STEPS][4];
                    const uint32_t from = sm.codes + (16 * half + gid) * F::K_PITCH + tid * (F::KP * F::BITS / 8) +
                                          (u * F::SUBS + sub) * (F::SUB * F::BITS / 8);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const uint32_t row = from + r * 8 * F::K_PITCH;
                        if constexpr (F::BITS == 8 && F::STEPS == 2) {
                            const uint2 w = in_ring<const uint2>(row);
                            codes8<F::KIND>(w.x, f[0][r], f[0][2 + r]);
                            codes8<F::KIND>(w.y, f[F::STEPS - 1][r], f[F::STEPS - 1][2 + r]);
                        } else if constexpr (F::BITS == 8) {
                            codes8<F::KIND>(lds<4>(row), f[0][r], f[0][2 + r]);
                        } else if constexpr (F::STEPS == 2) {
                            const uint32_t w = lds<4>(row) ^ 0x88888888u;  // elements (0, 4), (1, 5), (2, 6), (3, 7)
                            f[0][r] = codes4(w);
                            f[0][2 + r] = codes4_next(w);
                            f[F::STEPS - 1][r] = codes4(w >> 8);
                            f[F::STEPS - 1][2 + r] = codes4_next(w >> 8);
                        } else {
                            uint32_t w = lds<2>(row) ^ 0x8888u;  // elements (0, 2), (1, 3)
                            w |= w << 8;
                            f[0][r] = codes4(w);
                            f[0][2 + r] = codes4_next(w);
                        }
                    }
#pragma unroll
                    for (int st = 0; st < F::STEPS; ++st)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int t = 0; t < QT; ++t) {
                                const auto& qf = q[(u * F::SUBS + sub) * F::STEPS + st][nt][t];
                                mma16816(c[nt], f[st], qf[0], qf[1]);
                            }
                }
                const uint32_t scales = sm.k_scales + (u * 32 + 16 * half + gid) * 4;
                const float s0 = in_ring<const float>(scales), s1 = in_ring<const float>(scales + 32);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        l[half][nt][i] = u == 0 ? c[nt][i] * (i < 2 ? s0 : s1) : fmaf(c[nt][i], i < 2 ? s0 : s1, l[half][nt][i]);
            }
        }
        __syncwarp();
        if (tile + 1 < tiles) next_there = issue_keys();
        cp_async_commit();

        float grow[NT][2];
        bool grows = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < 4; ++i) l[half][nt][i] *= factor[nt][i & 1];
            if (huge) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i) l[half][nt][i] *= 1.f / kLess;
            }
            if (there != 0xffffffffu) {
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (!(there >> (16 * half + 8 * (i >> 1) + gid) & 1)) l[half][nt][i] = -INFINITY;
            }
            if (a.logits) {
                const int h = nt * 8 + tid * 2;
                const int64_t j = j0 + int64_t(tile) * kAttnTile + gid;
                float* to = attn_logits(a, p.s, p.pair, j) + h;
                if (h < a.logit_heads) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (j + 8 * k < j1)
                            *reinterpret_cast<float2*>(to + 8 * k * a.logit_heads) =
                                make_float2(l[k >> 1][nt][(k & 1) * 2], l[k >> 1][nt][(k & 1) * 2 + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float most = fmaxf(fmaxf(l[0][nt][i], l[0][nt][2 + i]), fmaxf(l[1][nt][i], l[1][nt][2 + i]));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 4));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 8));
                most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 16));
                most = fmaxf(m[nt][i], most);
                const float base = finite_max(most);
                grow[nt][i] = exp2_approx(m[nt][i] - base);  // (1 where they are equal: of both sums or neither)
                grows |= most > m[nt][i];
                m[nt][i] = most;
                float add = 0.f;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    l[half][nt][i] = exp2_approx(l[half][nt][i] - base);
                    l[half][nt][2 + i] = exp2_approx(l[half][nt][2 + i] - base);
                    add += l[half][nt][i] + l[half][nt][2 + i];
                }
                sum[nt][i] = fmaf(sum[nt][i], grow[nt][i], add);
            }
        }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int u = 0; u < F::UNITS; ++u)
#pragma unroll
                for (int t = 0; t < F::TILES; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[u][t][nt][i] *= grow[nt][i & 1];
        }

        // the values, half a tile after the other
        cp_async_wait<1>();
        __syncwarp();
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t v_from = sm.codes + F::V_AT + (16 * half + tid * 2) * F::V_PITCH + gid * F::VP * F::BITS / 8;
#pragma unroll
            for (int u = 0; u < F::UNITS; ++u) {
                if (!F::EXACT && u >= units) break;
                // the weights of positions gid and gid + 8, as columns those of 2 tid and 2 tid + 1, and of 8 further
                uint32_t b[NT][WT][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float s = in_ring<const float>(sm.v_scales + (u * 32 + 16 * half + 8 * r + gid) * 4);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float x = l[half][nt][2 * r] * s, y = l[half][nt][2 * r + 1] * s;
                        const uint32_t hi = half2_bits(x, y);
                        b[nt][0][r] = transpose8(hi);
                        if constexpr (WT == 2) {
                            const float2 f = half2_floats(hi);
                            b[nt][WT - 1][r] = transpose8(half2_bits((x - f.x) * 0x1p11f, (y - f.y) * 0x1p11f));
                        }
                    }
                }
                // elements of this lane's piece as pairs of positions (2 tid, 2 tid + 1) and 8 further
                uint32_t f[F::TILES][4];
                const uint32_t from = v_from + u * (F::UNIT * F::BITS / 8);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t row = from + r * 8 * F::V_PITCH;
                    constexpr int B = F::VP * F::BITS / 8;  // bytes of the piece: 16 to 1
                    uint32_t x[(B + 3) / 4], y[(B + 3) / 4];
                    if constexpr (B == 16) {
                        const uint4 v = in_ring<const uint4>(row), v2 = in_ring<const uint4>(row + F::V_PITCH);
                        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                        y[0] = v2.x, y[1] = v2.y, y[2] = v2.z, y[3] = v2.w;
                    } else if constexpr (B == 8) {
                        const uint2 v = in_ring<const uint2>(row), v2 = in_ring<const uint2>(row + F::V_PITCH);
                        x[0] = v.x, x[1] = v.y;
                        y[0] = v2.x, y[1] = v2.y;
                    } else {
                        x[0] = lds<B>(row);
                        y[0] = lds<B>(row + F::V_PITCH);
                    }
                    if constexpr (F::BITS == 8) {
#pragma unroll
                        for (int w4 = 0; w4 < (B + 3) / 4; ++w4) {
                            codes8<F::KIND>(__byte_perm(x[w4], y[w4], 0x5140), f[2 * w4][2 * r], f[2 * w4][2 * r + 1]);
                            if constexpr (B >= 4)
                                codes8<F::KIND>(__byte_perm(x[w4], y[w4], 0x7362), f[(2 * w4 + 1) % F::TILES][2 * r],
                                                f[(2 * w4 + 1) % F::TILES][2 * r + 1]);
                        }
                    } else {
#pragma unroll
                        for (int h2 = 0; h2 < (B + 1) / 2; ++h2) {  // two bytes of both rows: 4 elements
                            const uint32_t v = __byte_perm(x[h2 / 2], y[h2 / 2], h2 % 2 ? 0x7632 : 0x5410) ^ (B == 1 ? 0x00880088u : 0x88888888u);
                            f[(2 * h2) % F::TILES][2 * r] = codes4(v);
                            f[(2 * h2) % F::TILES][2 * r + 1] = codes4_next(v);
                            if constexpr (B > 1) {
                                f[(2 * h2 + 1) % F::TILES][2 * r] = codes4(v >> 8);
                                f[(2 * h2 + 1) % F::TILES][2 * r + 1] = codes4_next(v >> 8);
                            }
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < F::TILES; ++t)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < WT; ++k) {
                            float second[4] = {};
                            float(&to)[4] = k == 0 ? acc[u][t][nt] : second;
                            mma16816(to, f[t], b[nt][k][0], b[nt][k][1]);
                            if (k == 1) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) acc[u][t][nt][i] = fmaf(second[i], 0x1p-11f, acc[u][t][nt][i]);
                            }
                        }
            }
        }
        __syncwarp();
        there = next_there;
        if (tile + 1 < tiles) {
            copy_rows(std::integral_constant<int, 1>{}, there);
            look_up(j0 + int64_t(tile + 2) * kAttnTile);
        }
        cp_async_commit();
    }
    // ---- what the piece comes to ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float s = sum[nt][i];
            s += __shfl_xor_sync(0xffffffffu, s, 4);
            s += __shfl_xor_sync(0xffffffffu, s, 8);
            s += __shfl_xor_sync(0xffffffffu, s, 16);
            const int h = nt * 8 + tid * 2 + i;
            if (h >= p.heads) continue;
            const float scale = p.whole ? (s == 0.f ? 0.f : 1.f / s) : 1.f;
            bits* row = static_cast<bits*>(a.out.p) + p.s * a.out.ts + (p.q0 + h) * a.out.hs;
            float* part = a.part + p.part + h * attn_part_row(a.d);
#pragma unroll
            for (int u = 0; u < F::UNITS; ++u) {
                if (!F::EXACT && u >= units) break;
                const float unit = __uint_as_float(uint32_t(127 + top[u] - 15) << 23);
                const int at = u * F::UNIT + gid * F::VP;
                float v[F::VP];
#pragma unroll
                for (int t = 0; t < F::TILES; ++t) {
                    v[2 * t] = acc[u][t][nt][i] * scale * unit;
                    v[2 * t + 1] = acc[u][t][nt][2 + i] * (F::BITS == 4 ? scale * 0x1p-4f : scale) * unit;
                }
                // in fours, or the last two
#pragma unroll
                for (int k = 0; k < F::VP; k += 4) {
                    constexpr bool FOUR = F::VP >= 4;
                    const float v2 = FOUR ? v[(k + 2) % F::VP] : 0.f, v3 = FOUR ? v[(k + 3) % F::VP] : 0.f;
                    if (!p.whole || (a.out_vec && sizeof(T) == 4)) {
                        float* to = (p.whole ? reinterpret_cast<float*>(row) : part) + at + k;
                        if constexpr (FOUR) *reinterpret_cast<float4*>(to) = make_float4(v[k], v[k + 1], v2, v3);
                        else *reinterpret_cast<float2*>(to) = make_float2(v[k], v[k + 1]);
                    } else if (a.out_vec) {
                        if constexpr (sizeof(T) == 2) {
                            const uint32_t w0 = pack2<T>(make_float2(v[k], v[k + 1]));
                            if constexpr (FOUR) *reinterpret_cast<uint2*>(row + at + k) = make_uint2(w0, pack2<T>(make_float2(v2, v3)));
                            else *reinterpret_cast<uint32_t*>(row + at + k) = w0;
                        }
                    } else {
#pragma unroll
                        for (int e = k; e < F::VP && e < k + 4; ++e) row[at + e] = Io<T>::store(v[e]);
                    }
                }
            }
            if (gid == 0) {
                if (p.whole) {
                    attn_write_lse(a, p.s, p.q0 + h, m[nt][i], s);
                } else {
                    part[a.d] = m[nt][i];
                    part[a.d + 1] = s;
                }
            }
        }
    cp_async_wait<0>();
    __syncwarp();
}

template <typename T, typename F>
__global__ void __launch_bounds__(32 * kAttnFormWarps<F>, 1) attn_mma_kernel(const AttnArgs a) {
    __shared__ AttnTable table;
    pdl_next();
    attn_table(a, table);
    attn_empty<T>(a, table);
    const int groups = a.d / a.cache.group, warp = threadIdx.x >> 5;
    AttnSmem sm;
    sm.codes = uint32_t(warp) * attn_warp_bytes<F>(groups);
    sm.scales = sm.codes + F::S_AT;
    sm.places = sm.scales + 2 * 32 * groups * 4;
    sm.k_scales = sm.places + kAttnPlaces;
    sm.v_scales = sm.k_scales + F::UNITS * 128;
    attn_pieces(a, table, [&](const AttnPiece& p) { attn_mma_piece<T, F>(a, p, sm, groups); });
}

template <typename T, typename F>
nrm_status attn_mma_launch(AttnArgs& a, const DevInfo* dev, cudaStream_t s) {
    const void* fn = reinterpret_cast<const void*>(&attn_mma_kernel<T, F>);
    const int groups = a.d / a.cache.group;
    const size_t warp = attn_warp_bytes<F>(groups);
    // as many workers to an SM as have room for their rings beside the table
    const size_t room = size_t(dev->max_smem_optin) - sizeof(AttnTable) - 256;
    const int warps = int(std::min<size_t>(kAttnFormWarps<F>, room / warp));
    a.workers = dev->sms * warps;
    attn_snap(a);
    const size_t smem = warps * warp;
    nrm_status st = prepare_kernel(fn, smem, false);
    if (st != NRM_OK) return st;
    void* p[] = {&a};
    return launch_pdl(fn, dim3(unsigned(dev->sms)), dim3(unsigned(32 * warps)), p, s, smem);
}

// One translation unit for each storage type and stored form.
template <typename T, int KIND>
nrm_status attn_mma(AttnArgs& a, const DevInfo* dev, cudaStream_t s) {
    a.row_bytes = KIND == NRM_CACHE_INT4 ? a.d / 2 : a.d;
    const int nt = a.d <= 128 && a.shared > 8 ? 2 : 1;
    attn_chunks(a, 8 * nt);
    a.pages = a.cache.slots / a.cache.page.d;
    // the usual rows and groups have kernels of their own: units as long as the groups allow
    int unit = 16;
    for (int u : {32, 64, 128})
        if (a.d % u == 0 && a.cache.group % u == 0) unit = u;
    if (unit == 64 && a.d % 64 == 0 && a.d / 64 != 1 && a.d / 64 != 2 && a.d / 64 != 4) unit = 32;
#define NRM_ATTN_FORM(U, N) \
    if (unit == U && a.d == U * N) return attn_mma_launch<T, AttnForm<KIND, U, N, 1>>(a, dev, s)
#define NRM_ATTN_FORM2(U, N)                                                                        \
    if (unit == U && a.d == U * N)                                                                  \
    return nt == 2 ? attn_mma_launch<T, AttnForm<KIND, U, N, 2>>(a, dev, s) : attn_mma_launch<T, AttnForm<KIND, U, N, 1>>(a, dev, s)
    NRM_ATTN_FORM2(128, 1);
    NRM_ATTN_FORM2(64, 2);
    NRM_ATTN_FORM2(32, 4);
    NRM_ATTN_FORM2(64, 1);
    attn_chunks(a, 8);
    NRM_ATTN_FORM(32, 2);
    NRM_ATTN_FORM(16, 4);
    NRM_ATTN_FORM(16, 5);
    NRM_ATTN_FORM(32, 3);
    NRM_ATTN_FORM(16, 6);
    NRM_ATTN_FORM(32, 5);
    NRM_ATTN_FORM(16, 10);
    NRM_ATTN_FORM(128, 2);
    NRM_ATTN_FORM(64, 4);
#undef NRM_ATTN_FORM
#undef NRM_ATTN_FORM2
    return attn_mma_launch<T, AttnForm<KIND, 16, 16, 1, false>>(a, dev, s);
}

}  // namespace nrm
