// blocknorm.cuh -- the RMSNorm after a block, its gate and residual scale, the
// residual add and the RMSNorm before the next block in one pass, and its
// backward.
//
// Rows are cut into chunks, the chunks' column sums (the gradients of the
// weights and of the gate) go to the workspace in partial rows and are added in
// a fixed order.  A row of the gate that lies in one chunk is written at once;
// of the others each chunk holds at most two pieces (the end of its first and
// the beginning of its last).
#pragma once

#include "blocknorm.h"
#include "heads.cuh"

namespace nrm {

constexpr int kBlockThreads = 256;
constexpr int kBlockSumWarps = 32;

__device__ __forceinline__ float cta_sum(float v, float* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < int(blockDim.x >> 5); ++w) t += sums[w];
    return t;
}

// Sum of the warps' numbers in `sums` (at most 16), the same bits in every lane of every warp.
__device__ __forceinline__ float warps_sum(const float* sums, int warps) {
    const int lane = threadIdx.x & 31;
    float v = (lane & 15) < warps ? sums[lane & 15] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// r^3 v.  One factor at a time: the mean of a gradient times a row is about 1/r, so that no step is far from the
// result, while r^3 alone leaves float32 where a row and eps are tiny (r above 7e12).
__device__ __forceinline__ float cubed(float r, float v) { return r * (r * (r * v)); }

// Element i of a weight (1 where there is none).
template <typename T>
__device__ __forceinline__ float weight_at(const void* w, int64_t i) {
    using bits = typename Io<T>::bits_t;
    return w ? Io<T>::load(ld_after(static_cast<const bits*>(w) + i)) : 1.f;
}
template <typename T>
__device__ __forceinline__ float element(const void* p, int64_t i) {
    using bits = typename Io<T>::bits_t;
    return Io<T>::load(ld_after(static_cast<const bits*>(p) + i));
}
template <typename T>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<typename Io<T>::bits_t*>(p)[i] = Io<T>::store(v);
}

// The chunks of rows: as many as rows at most; chunk c's first row.
__device__ __forceinline__ int64_t chunk_begin(const BlockArgs& a, int64_t c) { return a.rows * c / a.chunks; }
__device__ __forceinline__ int64_t chunk_owner(const BlockArgs& a, int64_t row) {
    return ((row + 1) * a.chunks - 1) / a.rows;
}
// The partial row `kind` (0: dw_post, 1: dw_pre, 2: the end of a gate row that began in an earlier chunk, 3: the
// beginning of one that goes on in the next) of chunk c.
__device__ __forceinline__ float* part_row(const BlockArgs& a, int kind, int64_t c) {
    return a.part + (kind * a.chunks + c) * a.cols;
}

// ---------------------------------------------------------------------------
// rows too long for the kernels below, and the backward of inputs that do not begin
// at 16 bytes: a CTA for each row
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kBlockThreads) block_fwd_scalar_kernel(const BlockArgs a) {
    __shared__ float sums[32];
    pdl_next();
    const float cols = float(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t at = r * a.cols, gate_at = a.gates ? row_div(r, a.per_gate) * a.cols : 0;
        float r1 = 1.f;
        if (a.post) {
            float s = 0.f;
            for (int i = threadIdx.x; i < a.cols; i += kBlockThreads) {
                const float f = element<T>(a.f, at + i);
                s = fmaf(f, f, s);
            }
            r1 = rsqrtf(cta_sum(s, sums) / cols + a.eps);
            if (a.rstd_post && threadIdx.x == 0) a.rstd_post[r] = r1;
        }
        float s = 0.f;
        for (int i = threadIdx.x; i < a.cols; i += kBlockThreads) {
            float n = element<T>(a.f, at + i);
            if (a.post) n = n * r1 * weight_at<T>(a.w_post, i);
            const float g = a.alpha * (a.gates ? element<T>(a.gate, gate_at + i) : 1.f);
            const auto y = Io<T>::store(fmaf(g, n, element<T>(a.x, at + i)));
            static_cast<typename Io<T>::bits_t*>(a.y)[at + i] = y;
            const float z = Io<T>::load(y);
            s = fmaf(z, z, s);
        }
        if (!a.h) continue;
        const float r2 = rsqrtf(cta_sum(s, sums) / cols + a.eps);
        if (a.rstd_pre && threadIdx.x == 0) a.rstd_pre[r] = r2;
        for (int i = threadIdx.x; i < a.cols; i += kBlockThreads)
            put<T>(a.h, at + i, element<T>(a.y, at + i) * r2 * weight_at<T>(a.w_pre, i));
    }
}

// The gradient of y at element i of row r, from the row's c2 = r2^3 sum(G*y)/cols.
template <typename T>
__device__ __forceinline__ float grad_y(const BlockArgs& a, int64_t e, int i, float r2, float c2) {
    float d = a.dy ? element<T>(a.dy, e) : 0.f;
    if (a.dh) d = d + fmaf(r2, element<T>(a.dh, e) * weight_at<T>(a.w_pre, i), -element<T>(a.y, e) * c2);
    return d;
}

template <typename T>
__global__ void __launch_bounds__(kBlockThreads) block_bwd_scalar_kernel(const BlockArgs a) {
    __shared__ float sums[32];
    pdl_next();
    const float cols = float(a.cols);
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const int64_t at = r * a.cols, gate_at = a.gates ? row_div(r, a.per_gate) * a.cols : 0;
        const float r1 = a.post ? ld_after(a.rstd_post + r) : 1.f, r2 = a.dh ? ld_after(a.rstd_pre + r) : 0.f;
        float c2 = 0.f;
        if (a.dh) {
            float s = 0.f;
            for (int i = threadIdx.x; i < a.cols; i += kBlockThreads)
                s = fmaf(element<T>(a.dh, at + i) * weight_at<T>(a.w_pre, i), element<T>(a.y, at + i), s);
            c2 = cubed(r2, cta_sum(s, sums) / cols);
        }
        if (a.c2 && threadIdx.x == 0) a.c2[r] = c2;
        float s = 0.f;
        for (int i = threadIdx.x; i < a.cols; i += kBlockThreads) {
            const float d = grad_y<T>(a, at + i, i, r2, c2);
            put<T>(a.dx, at + i, d);
            const float dn = a.alpha * (a.gates ? element<T>(a.gate, gate_at + i) : 1.f) * d;
            if (a.post) s = fmaf(dn * weight_at<T>(a.w_post, i), element<T>(a.f, at + i), s);
            else put<T>(a.df, at + i, dn);
        }
        if (!a.post) continue;
        const float c1 = cubed(r1, cta_sum(s, sums) / cols);
        for (int i = threadIdx.x; i < a.cols; i += kBlockThreads) {
            const float d = grad_y<T>(a, at + i, i, r2, c2);
            const float dn = a.alpha * (a.gates ? element<T>(a.gate, gate_at + i) : 1.f) * d;
            put<T>(a.df, at + i, fmaf(r1, dn * weight_at<T>(a.w_post, i), -element<T>(a.f, at + i) * c1));
        }
    }
}

// The chunks' column sums: a thread for each column (blockIdx.x) of a chunk (blockIdx.y).
template <typename T>
__global__ void __launch_bounds__(kBlockThreads) block_cols_kernel(const BlockArgs a) {
    pdl_next();
    const int i = int(blockIdx.x) * kBlockThreads + threadIdx.x;
    if (i >= a.cols) return;
    const int64_t c = blockIdx.y, end = chunk_begin(a, c + 1);
    int64_t r = chunk_begin(a, c);
    const float w_pre = weight_at<T>(a.w_pre, i), w_post = a.post ? weight_at<T>(a.w_post, i) : 1.f;
    float sum_post = 0.f, sum_pre = 0.f;
    while (r < end) {
        // the rows of one gate row
        const int64_t g = a.gates ? row_div(r, a.per_gate) : 0, first = a.gates ? g * a.per_gate.d : r;
        const int64_t last = a.gates ? min(end, first + a.per_gate.d) : end;
        const bool begins = r == first, ends = !a.gates || last == first + a.per_gate.d;
        const float gate = a.gates ? element<T>(a.gate, g * a.cols + i) : 1.f;
        float sum = 0.f;
        for (; r < last; ++r) {
            const int64_t e = r * a.cols + i;
            float d = a.dy ? element<T>(a.dy, e) : 0.f;
            if (a.dh) {
                const float dh = element<T>(a.dh, e), y = element<T>(a.y, e), r2 = ld_after(a.rstd_pre + r);
                d = d + fmaf(r2, dh * w_pre, -y * ld_after(a.c2 + r));
                sum_pre = fmaf(dh, y * r2, sum_pre);
            }
            const float unit = element<T>(a.f, e) * (a.post ? ld_after(a.rstd_post + r) : 1.f);
            sum = fmaf(a.alpha * d, unit * w_post, sum);
            sum_post = fmaf(a.alpha * gate * d, unit, sum_post);
        }
        if (a.dgate) {
            if (begins && ends) put<T>(a.dgate, g * a.cols + i, sum);
            else part_row(a, begins ? 3 : 2, c)[i] = sum;
        }
    }
    if (a.dw_post) part_row(a, 0, c)[i] = sum_post;
    if (a.dw_pre) part_row(a, 1, c)[i] = sum_pre;
}

// ---------------------------------------------------------------------------
// whole 16-byte vectors, forward: a row in the registers of a CTA
// ---------------------------------------------------------------------------
// Every input is read once and every output written once; the stored stream is
// kept as its rounded bits for the second norm.  A CTA takes `per` neighbouring
// rows, one at a time, so that its columns of the weights and the gate stay in
// registers, and asks for a row DEPTH rows before it is needed.  Bound by bytes
// (16384 rows of 4096: 85 us, 0.93 of the copy rate; as many bytes in float32,
// 16384 rows of 2048: 83).
// FAST: both norms, and rows of whole vectors for every thread: nothing then parts the loops' instructions.
template <typename T, int VPT, int DEPTH, int MOST, int CTAS, bool FAST>
__global__ void __launch_bounds__(MOST, CTAS) block_fwd_vec_kernel(const BlockArgs a, int per) {
    constexpr int VE = kVec<T>, H = VE / 2;
    __shared__ float sums[2][2][16];
    pdl_next();
    const int threads = int(blockDim.x), t = threadIdx.x, warps = threads >> 5;
    const int64_t first = int64_t(blockIdx.x) * per, end = min(a.rows, first + per);
    const int nvec = a.cols / VE;
    const float inv = 1.f / float(a.cols);
    int phase = 0;
    auto row_sum = [&](float v, int which) {
        v = warp_sum(v);
        if (warps == 1) return v;
        if ((t & 31) == 0) sums[which][phase][t >> 5] = v;
        __syncthreads();
        return warps_sum(sums[which][phase], warps);
    };
    auto vec = [&](const void* p, int64_t i) { return ld_after(static_cast<const uint4*>(p) + i); };
    auto in_row = [&](int j) { return FAST || j * threads + t < nvec; };
    const bool post = FAST || a.post, pre = FAST || a.h;
    uint4 fr[DEPTH][VPT], xr[DEPTH][VPT];
    auto load_row = [&](int d, int64_t row) {
        if (row >= end) return;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (in_row(j)) fr[d][j] = vec(a.f, row * nvec + j * threads + t);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
            if (in_row(j)) xr[d][j] = vec(a.x, row * nvec + j * threads + t);
    };
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) load_row(d, first + d);
    // this thread's columns of alpha * gate * w_post and of w_pre
    float2 scale[VPT][H], w_pre[VPT][H];
    auto load_scale = [&](int64_t gate_row) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float2 v[H];
#pragma unroll
            for (int h = 0; h < H; ++h) scale[j][h] = f2(a.alpha);
            if (!in_row(j)) continue;
            if (a.gates) {
                unpack2<T>(vec(a.gate, gate_row * nvec + j * threads + t), v);
#pragma unroll
                for (int h = 0; h < H; ++h) scale[j][h] = __fmul2_rn(scale[j][h], v[h]);
            }
            if (a.w_post) {
                unpack2<T>(vec(a.w_post, j * threads + t), v);
#pragma unroll
                for (int h = 0; h < H; ++h) scale[j][h] = __fmul2_rn(scale[j][h], v[h]);
            }
        }
    };
    int64_t gate_row = a.gates ? row_div(first, a.per_gate) : 0, gate_end = a.gates ? (gate_row + 1) * a.per_gate.d : end;
    load_scale(gate_row);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
#pragma unroll
        for (int h = 0; h < H; ++h) w_pre[j][h] = f2(1.f);
        if (pre && a.w_pre && in_row(j)) unpack2<T>(vec(a.w_pre, j * threads + t), w_pre[j]);
    }
    for (int64_t r0 = first; r0 < end; r0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int64_t r = r0 + d;
            if (r >= end) break;
            if (r == gate_end) {
                gate_end += a.per_gate.d;
                load_scale(++gate_row);
            }
            const int64_t at = r * nvec + t;
            float r1 = 1.f;
            if (post) {
                float2 s = f2(0.f);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    if (!in_row(j)) break;
                    float2 f[H];
                    unpack2<T>(fr[d][j], f);
#pragma unroll
                    for (int h = 0; h < H; ++h) s = __ffma2_rn(f[h], f[h], s);
                }
                r1 = rsqrtf(row_sum(s.x + s.y, 0) * inv + a.eps);
                if (a.rstd_post && t == 0) a.rstd_post[r] = r1;
            }
            float2 s = f2(0.f);
            uint4 yr[VPT];
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                if (!in_row(j)) break;
                float2 f[H], x[H];
                unpack2<T>(fr[d][j], f);
                unpack2<T>(xr[d][j], x);
#pragma unroll
                for (int h = 0; h < H; ++h) x[h] = __ffma2_rn(__fmul2_rn(f[h], f2(r1)), scale[j][h], x[h]);
                yr[j] = pack2x<T>(x);
                st_v4(static_cast<uint4*>(a.y) + at + j * threads, yr[j]);
                if constexpr (sizeof(T) == 2) unpack2<T>(yr[j], x);
#pragma unroll
                for (int h = 0; h < H; ++h) s = __ffma2_rn(x[h], x[h], s);
            }
            load_row(d, r + DEPTH);
            if (pre) {
                const float r2 = rsqrtf(row_sum(s.x + s.y, 1) * inv + a.eps);
                if (a.rstd_pre && t == 0) a.rstd_pre[r] = r2;
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    if (!in_row(j)) break;
                    float2 y[H];
                    unpack2<T>(yr[j], y);
#pragma unroll
                    for (int h = 0; h < H; ++h) y[h] = __fmul2_rn(__fmul2_rn(y[h], f2(r2)), w_pre[j][h]);
                    st_v4(static_cast<uint4*>(a.h) + at + j * threads, pack2x<T>(y));
                }
            }
            phase ^= 1;
        }
    }
}

// ---------------------------------------------------------------------------
// rows of any length and alignment, forward: the same, element by element
// ---------------------------------------------------------------------------
// Thread t has the elements t, t + THREADS, ... (a known number apart: an access is then one instruction); what hides
// the loads' latency is the CTAs of an SM and the next row, which is asked for before the second norm.  Bound by
// instructions (8192 rows of 4095: 74 us, 0.53 of the copy rate; in three passes over a row 139).
constexpr int kBlockElems = 8;  // of a thread
template <typename T, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) block_fwd_elem_kernel(const BlockArgs a, int per) {
    using bits = typename Io<T>::bits_t;
    constexpr int E = kBlockElems, threads = THREADS, warps = THREADS / 32;
    __shared__ float sums[2][2][32];
    pdl_next();
    const int t = threadIdx.x, lane = t & 31, left = a.cols - t;
    const int64_t first = int64_t(blockIdx.x) * per, end = min(a.rows, first + per);
    const float inv = 1.f / float(a.cols);
    int phase = 0;
    auto row_sum = [&](float v, int which) {
        v = warp_sum(v);
        if (warps == 1) return v;
        if (lane == 0) sums[which][phase][t >> 5] = v;
        __syncthreads();
        return warp_sum(lane < warps ? sums[which][phase][lane] : 0.f);
    };
    auto there = [&](int e) { return left > e * threads; };
    bits fr[E], xr[E];
    auto load_row = [&](int64_t row) {
        if (row >= end) return;
        const bits *f = static_cast<const bits*>(a.f) + row * a.cols + t, *x = static_cast<const bits*>(a.x) + row * a.cols + t;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (there(e)) fr[e] = ld_after(f + e * threads);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (there(e)) xr[e] = ld_after(x + e * threads);
    };
    load_row(first);
    float scale[E], w_pre[E];  // alpha * gate * w_post
    auto load_scale = [&](int64_t gate_row) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int i = e * threads + t;
            scale[e] = a.alpha;
            if (!there(e)) continue;
            if (a.gates) scale[e] *= element<T>(a.gate, gate_row * a.cols + i);
            if (a.w_post) scale[e] *= element<T>(a.w_post, i);
        }
    };
    int64_t gate_row = a.gates ? row_div(first, a.per_gate) : 0, gate_end = a.gates ? (gate_row + 1) * a.per_gate.d : end;
    load_scale(gate_row);
#pragma unroll
    for (int e = 0; e < E; ++e) w_pre[e] = a.h && there(e) ? weight_at<T>(a.w_pre, e * threads + t) : 1.f;
    for (int64_t r = first; r < end; ++r) {
        if (r == gate_end) {
            gate_end += a.per_gate.d;
            load_scale(++gate_row);
        }
        float r1 = 1.f;
        if (a.post) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (there(e)) s = fmaf(Io<T>::load(fr[e]), Io<T>::load(fr[e]), s);
            r1 = rsqrtf(row_sum(s, 0) * inv + a.eps);
            if (a.rstd_post && t == 0) a.rstd_post[r] = r1;
        }
        float s = 0.f, y[E];
        bits* to = static_cast<bits*>(a.y) + r * a.cols + t;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (!there(e)) continue;
            const bits b = Io<T>::store(fmaf(Io<T>::load(fr[e]) * r1, scale[e], Io<T>::load(xr[e])));
            to[e * threads] = b;
            y[e] = Io<T>::load(b);
            s = fmaf(y[e], y[e], s);
        }
        load_row(r + 1);
        if (a.h) {
            const float r2 = rsqrtf(row_sum(s, 1) * inv + a.eps);
            if (a.rstd_pre && t == 0) a.rstd_pre[r] = r2;
            to = static_cast<bits*>(a.h) + r * a.cols + t;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (there(e)) to[e * threads] = Io<T>::store(y[e] * r2 * w_pre[e]);
        }
        phase ^= 1;
    }
}

// ---------------------------------------------------------------------------
// backward: rows through a ring in shared memory
// ---------------------------------------------------------------------------
// A CTA stays for its chunk of rows.  One bulk copy for each of dh, dy, f and y
// brings the next rows into a slot of the ring (a few slots ahead: enough bytes in
// flight for the memory without a register each), and groups of threads take a
// row of the slot each, a thread the same VPT vectors of every row, so that the
// columns' sums stay in its registers.  A row's elements are read from the slot
// once and kept as their bits through its two sums (sum(G*y), then sum(g*f),
// which needs the first); after the first the slot is free.  A slot does not
// reach over the end of a gate's row; there the groups' sums of its gradient are
// added, in their order.
//
// Rows of whole 16-byte vectors are taken so.  Of others (ELEMS, the threads of a
// group) a thread takes 16 bytes' worth of elements, ELEMS apart, one by one; the copies are rounded
// outwards to 16 bytes, which stays within the tensor, but for its last bytes,
// which thread 0 brings itself.
constexpr int kBlockConsumers = 512;
constexpr int kBlockSlots = 8;                       // at most
constexpr uint64_t kBlockWaitNs = 2000000000ull;     // bounded waits: 2 s
constexpr int kBlockBar = 1;                         // the groups' named barriers

struct BlockRing {
    int groups, threads;     // groups of threads to a CTA; threads of a group, whole warps
    int rows;                // of a slot: groups times the rows that a group takes at once
    int slots;               // two at least: rows are asked for a slot ahead of those that are worked on
    int places;              // for the groups' sums
    uint32_t tensor_bytes;   // of a tensor's rows in a slot
    uint32_t slot_bytes;
    uint32_t ring_at;        // after the weights
};

// The chunk's rows, slot by slot: f(first row, rows, whether a gate's row ends with them).
struct BlockWalk {
    int64_t r, end, gate_end;
    int count;
    __device__ __forceinline__ BlockWalk(const BlockArgs& a, bool by_gate) : r(chunk_begin(a, blockIdx.x)), end(chunk_begin(a, blockIdx.x + 1)) {
        gate_end = by_gate ? (row_div(r, a.per_gate) + 1) * a.per_gate.d : end;
        count = 0;
    }
    __device__ __forceinline__ bool next(const BlockArgs& a, const BlockRing& g) {
        r += count;
        if (r >= end) return false;
        if (r == gate_end) gate_end += a.per_gate.d;
        count = int(min(int64_t(g.rows), min(end, gate_end) - r));
        return true;
    }
};

// What thread 0 asks for, slot by slot: the next rows of up to four tensors.
struct BlockAsk {
    BlockWalk walk;
    const void* from[4];
    int asked = 0, slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ BlockAsk(const BlockArgs& a, bool by_gate, const void* t0, const void* t1, const void* t2, const void* t3)
        : walk(a, by_gate), from{t0, t1, t2, t3} {}
    // false: the slot's last rows were not done with in time
    __device__ __forceinline__ bool next(const BlockArgs& a, const BlockRing& g, unsigned char* smem, uint64_t* full, uint64_t* empty,
                                         int64_t row_bytes, uint64_t pol, bool elem) {
        if (!walk.next(a, g)) return true;
        if (round > 0 && !mbar_wait_bounded(&empty[slot], (round - 1) & 1u, kBlockWaitNs)) {
            walk.r = walk.end;  // no more copies
            walk.count = 0;
            return false;
        }
        int64_t begin = walk.r * row_bytes, end = begin + walk.count * row_bytes;
        unsigned char* to = smem + g.ring_at + size_t(slot) * g.slot_bytes;
        if (elem) {
            const int64_t last = end;
            begin &= ~int64_t(15);
            end = min((end + 15) & ~int64_t(15), (a.rows * row_bytes) & ~int64_t(15));
            if (end < last) {  // the tensors' last bytes
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (from[k])
                        for (int64_t i = end; i < last; i += 2)
                            *reinterpret_cast<uint16_t*>(to + k * g.tensor_bytes + (i - begin)) =
                                ld_after(reinterpret_cast<const uint16_t*>(static_cast<const unsigned char*>(from[k]) + i));
            }
        }
        const uint32_t bytes = uint32_t(end - begin);
        mbar_arrive_expect_tx(&full[slot], bytes * ((from[0] != nullptr) + (from[1] != nullptr) + (from[2] != nullptr) + (from[3] != nullptr)));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (from[k] && bytes)
                bulk_g2s(to + k * g.tensor_bytes, static_cast<const unsigned char*>(from[k]) + begin, bytes, &full[slot], pol);
        ++asked;
        if (++slot == g.slots) {
            slot = 0;
            ++round;
        }
        return true;
    }
    // no copy may be under way when the CTA ends
    __device__ __forceinline__ void settle(const BlockRing& g, uint64_t* full) const {
        for (int i = 0; i < g.slots && i < asked; ++i)
            (void)mbar_wait_bounded(&full[i], uint32_t((asked - 1 - i) / g.slots) & 1u, kBlockWaitNs);
    }
};

// The sums of R numbers each over a group's threads.
template <int R>
__device__ __forceinline__ void group_sums(float (&v)[R], float* place, int group, int warps, int threads) {
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] = warp_sum(v[k]);
    if (warps == 1) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < R; ++k) place[k * 16 + warp] = v[k];
    }
    named_barrier(kBlockBar + group, threads);
#pragma unroll
    for (int k = 0; k < R; ++k) v[k] = warps_sum(place + k * 16 + group * warps, warps);
}

// FAST: everything is there, with one gate for many rows or none, and rows of whole vectors for every thread.
template <typename T, int VPT, int ROWS, bool FAST, int ELEMS = 0>
__global__ void __launch_bounds__(kBlockConsumers, 1) block_bwd_ring_kernel(const BlockArgs a, const BlockRing g) {
    using bits = typename Io<T>::bits_t;
    constexpr int VE = kVec<T>, H = VE / 2;
    constexpr bool ELEM = ELEMS != 0;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t full[kBlockSlots], empty[kBlockSlots];
    __shared__ float sums[2][2][ROWS * 16];
    __shared__ int s_bad;
    const int threads = ELEM ? ELEMS : g.threads;  // of a group
    const int group = int(threadIdx.x) / threads, t = int(threadIdx.x) - group * threads, warps = threads >> 5;
    const int nvec = ELEM ? VPT * threads : a.cols / VE;  // vectors of a row, or threads' shares of one
    // Shares of elements: share j of thread t has the elements t + (j*VE + e)*ELEMS.  From a row (0 behind its end), and
    // into one.
    auto gather = [&](auto&& load, int j, int t) {
        const int left = a.cols - t;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) {
                const int at = (j * VE + k) * ELEMS;
                w[k] = left > at ? uint32_t(load(t + at)) : 0u;
            } else {
                const int at = (j * VE + 2 * k) * ELEMS, next = at + ELEMS;
                const uint32_t lo = left > at ? uint32_t(load(t + at)) : 0u, hi = left > next ? uint32_t(load(t + next)) : 0u;
                w[k] = __byte_perm(lo, hi, 0x5410);
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    auto scatter = [&](bits* row, int j, int t, uint4 v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        const int left = a.cols - t;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const int at = (j * VE + e) * ELEMS;
            if (left > at) row[t + at] = sizeof(T) == 4 ? bits(w[e % 4]) : bits(w[e / 2 % 4] >> (16 * (e & 1)));
        }
    };
    // vector or share j of thread t of row r of a tensor
    auto from_global = [&](const void* p, int64_t r, int j, int t) {
        if constexpr (ELEM) {
            const bits* row = static_cast<const bits*>(p) + r * a.cols;
            return gather([&](int at) { return ld_after(row + at); }, j, t);
        } else {
            return ld_after(static_cast<const uint4*>(p) + r * nvec + (j * threads + t));
        }
    };
    auto to_global = [&](void* p, int64_t r, int j, int t, uint4 v) {
        if constexpr (ELEM) scatter(static_cast<bits*>(p) + r * a.cols, j, t, v);
        else st_v4(static_cast<uint4*>(p) + r * nvec + (j * threads + t), v);
    };
    if (threadIdx.x == 0) {
        s_bad = 0;
        for (int i = 0; i < g.slots; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], g.groups);
        }
        mbar_init_fence();
    }
    pdl_next();
    uint4* const weights = reinterpret_cast<uint4*>(smem);  // w_pre, w_post
    for (int i = int(threadIdx.x); i < 2 * nvec; i += int(blockDim.x)) {
        const void* w = i < nvec ? a.w_pre : a.w_post;
        float2 one[H];
#pragma unroll
        for (int h = 0; h < H; ++h) one[h] = f2(1.f);
        const int k = i < nvec ? i : i - nvec;
        weights[i] = w ? from_global(w, 0, k / threads, k % threads) : pack2x<T>(one);
    }
    __syncthreads();

    const bool has_dh = FAST || a.dh, has_dy = FAST || a.dy, post = FAST || a.post;
    const bool by_row = !FAST && a.gates > 0 && a.per_gate.d == 1;  // a gate of its own for every row: its gradient is written as it is made
    const bool by_gate = a.gates > 0 && !by_row && (a.gates > 1 || a.dgate);
    const int64_t row_bytes = int64_t(a.cols) * int64_t(sizeof(T));
    const uint64_t pol = l2_evict_first();
    bool bad = false;
    BlockAsk ask(a, by_gate, a.dh, a.dy, a.f, a.dh ? a.y : nullptr);
    if (threadIdx.x == 0)
        for (int i = 0; i < g.slots; ++i) ask.next(a, g, smem, full, empty, row_bytes, pol, ELEM);

    // Over rows with one gate (and over all without), the sums of dgate and dw_post are this one's, times alpha*w_post
    // and alpha*gate: sum_unit = sum of dx*f*r1.
    float2 sum_pre[VPT][H], sum_post[VPT][H], sum_unit[VPT][H];
    float2 scale[VPT][H];  // alpha * gate * w_post
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int h = 0; h < H; ++h) sum_pre[j][h] = sum_post[j][h] = sum_unit[j][h] = f2(0.f);
    auto load_scale = [&](int64_t gate_row, bool with_weight, float2 (&to)[VPT][H]) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = j * threads + t;
#pragma unroll
            for (int h = 0; h < H; ++h) to[j][h] = f2(a.alpha);
            if (i >= nvec) break;
            float2 v[H];
            if (with_weight) {
                unpack2<T>(weights[nvec + i], v);
#pragma unroll
                for (int h = 0; h < H; ++h) to[j][h] = __fmul2_rn(to[j][h], v[h]);
            }
            if (a.gates && gate_row >= 0) {
                unpack2<T>(from_global(a.gate, gate_row, j, t), v);
#pragma unroll
                for (int h = 0; h < H; ++h) to[j][h] = __fmul2_rn(to[j][h], v[h]);
            }
        }
    };
    // the rows of one gate are done: their share of dw_post, and sum_unit as the gradient of the gate
    auto close_gate = [&](int64_t gate_row) {
        float2 by[VPT][H];
        load_scale(gate_row, false, by);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h) sum_post[j][h] = __ffma2_rn(sum_unit[j][h], by[j][h], sum_post[j][h]);
        load_scale(-1, true, by);
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h) sum_unit[j][h] = __fmul2_rn(sum_unit[j][h], by[j][h]);
    };
    int phase = 0;
    const float inv = 1.f / float(a.cols);
    auto clear = [&](float2 (&acc)[VPT][H]) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int h = 0; h < H; ++h) acc[j][h] = f2(0.f);
    };
    // the groups' sums of a gradient, added in their order, to a partial row `out` or, whole, to row `out_row` of `out_t`
    auto put_sums = [&](const float2 (&v)[H], int j, int t, float* out, void* out_t, int64_t out_row) {
        if (out_t) {
            to_global(out_t, out_row, j, t, pack2x<T>(v));
            return;
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            if constexpr (ELEM) {
                const int at = t + (j * VE + 2 * h) * ELEMS;
                if (at < a.cols) out[at] = v[h].x;
                if (at + ELEMS < a.cols) out[at + ELEMS] = v[h].y;
            } else {
                reinterpret_cast<float2*>(out)[(j * threads + t) * H + h] = v[h];
            }
        }
    };
    auto flush = [&](float2 (&acc)[VPT][H], float* out, void* out_t, int64_t out_row) {
        // (the ring may be in use: its own place, before the ring)
        float* place = reinterpret_cast<float*>(smem + 2 * size_t(nvec) * 16);
        if (g.groups == 1) {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = j * threads + t;
                if (i >= nvec) break;
                put_sums(acc[j], j, t, out, out_t, out_row);
            }
        } else {
            // (more than one group: a thread has one vector or share)  In as many turns as the places need, the sum so far
            // in the first.
            float2* const all = reinterpret_cast<float2*>(place);
            for (int k0 = 0; k0 < g.groups;) {
                const int at = k0 > 0, n = min(g.groups - k0, g.places - at);
                if (group >= k0 && group < k0 + n) {
#pragma unroll
                    for (int h = 0; h < H; ++h) all[((at + group - k0) * H + h) * threads + t] = acc[0][h];
                }
                __syncthreads();
                for (int i = int(threadIdx.x); i < H * threads; i += int(blockDim.x)) {
                    float2 v = all[i];
#pragma unroll 4
                    for (int k = 1; k < at + n; ++k) v = __fadd2_rn(v, all[k * H * threads + i]);
                    all[i] = v;
                }
                __syncthreads();
                k0 += n;
            }
            for (int i = int(threadIdx.x); i < nvec; i += int(blockDim.x)) {
                float2 v[H];
#pragma unroll
                for (int h = 0; h < H; ++h) v[h] = all[h * threads + i];
                put_sums(v, 0, i, out, out_t, out_row);
            }
            __syncthreads();
        }
        clear(acc);
    };

    BlockWalk walk(a, by_gate);
    int64_t first = walk.r;  // of the gate's row's rows in this chunk
    int64_t gate_row = a.gates ? row_div(first, a.per_gate) : 0;
    if (!by_row) load_scale(gate_row, true, scale);
    int slot = -1;
    uint32_t round = 0;
    for (bool begun = false; walk.next(a, g); begun = true) {
        if (++slot == g.slots) {
            slot = 0;
            ++round;
        }
        if (by_gate && walk.r == first && begun) load_scale(gate_row, true, scale);
        const int mine = walk.count - group * ROWS;  // rows of this group, if not all
        // (a group without one waits too: it must not be rounds ahead when it says that it is done with the slot)
        if (!bad && !mbar_wait_bounded(&full[slot], round & 1u, kBlockWaitNs)) bad = true;
        if (mine > 0) {
            auto rows = [&](auto full_rows) {
            constexpr bool FULL = decltype(full_rows)::value;  // all ROWS of them
            const unsigned char* const from = smem + g.ring_at + size_t(slot) * g.slot_bytes +
                                              (ELEM ? int(walk.r * row_bytes & 15) : 0) + group * ROWS * row_bytes;
            const int64_t r = walk.r + group * ROWS;
            // vector or share j of this thread of the group's row k of a tensor
            auto in_slot = [&](int tensor, int k, int j) {
                const unsigned char* row = from + tensor * g.tensor_bytes + k * row_bytes;
                if constexpr (ELEM) return gather([&](int at) { return reinterpret_cast<const bits*>(row)[at]; }, j, t);
                else return reinterpret_cast<const uint4*>(row)[j * threads + t];
            };
            if (by_row) load_scale(r, true, scale);  // (one row at once)
            uint4 dyr[ROWS][VPT], fr[ROWS][VPT], yr[ROWS][VPT];
            float2 big[ROWS][VPT][H];  // dh*w_pre, then dx*scale
            float r1[ROWS], r2[ROWS], s[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                // a row behind the last: statistics of 0, so that whatever its slot holds adds nothing
                r1[k] = !(FULL || k < mine) ? 0.f : post ? ld_after(a.rstd_post + r + k) : 1.f;
                r2[k] = k < mine && has_dh ? ld_after(a.rstd_pre + r + k) : 0.f;
            }
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                float2 sum = f2(0.f);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = j * threads;
                    if ((!FAST && i + t >= nvec) || !(FULL || k < mine)) break;
                    if (has_dy) dyr[k][j] = in_slot(1, k, j);
                    fr[k][j] = in_slot(2, k, j);
                    if (has_dh) {
                        yr[k][j] = in_slot(3, k, j);
                        float2 dh[H], y[H], w[H];
                        unpack2<T>(in_slot(0, k, j), dh);
                        unpack2<T>(yr[k][j], y);
                        unpack2<T>(weights[i + t], w);
#pragma unroll
                        for (int h = 0; h < H; ++h) {
                            big[k][j][h] = __fmul2_rn(dh[h], w[h]);
                            sum = __ffma2_rn(big[k][j][h], y[h], sum);
                            sum_pre[j][h] = __ffma2_rn(dh[h], __fmul2_rn(y[h], f2(r2[k])), sum_pre[j][h]);
                        }
                    }
                }
                s[k] = sum.x + sum.y;
            }
            if (has_dh) group_sums<ROWS>(s, sums[0][phase], group, warps, threads);
            else if (warps > 1) named_barrier(kBlockBar + group, threads);
            if (warps == 1) __syncwarp();  // (a warp's sums are exchanges, which order no reads)
            if (t == 0) mbar_arrive(&empty[slot]);  // (every thread of the group has read its part)
            if (threadIdx.x == 0 && begun && !ask.next(a, g, smem, full, empty, row_bytes, pol, ELEM)) bad = true;
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const float c2 = cubed(r2[k], s[k] * inv);
                float2 sum = f2(0.f);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = j * threads;
                    if ((!FAST && i + t >= nvec) || !(FULL || k < mine)) break;
                    float2 d[H], f[H];
#pragma unroll
                    for (int h = 0; h < H; ++h) d[h] = f2(0.f);
                    if (has_dy) unpack2<T>(dyr[k][j], d);
                    unpack2<T>(fr[k][j], f);
                    if (has_dh) {
                        float2 y[H];
                        unpack2<T>(yr[k][j], y);
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            d[h] = __ffma2_rn(y[h], f2(-c2), __ffma2_rn(f2(r2[k]), big[k][j][h], d[h]));
                    }
                    to_global(a.dx, r + k, j, t, pack2x<T>(d));
#pragma unroll
                    for (int h = 0; h < H; ++h) {
                        big[k][j][h] = __fmul2_rn(d[h], scale[j][h]);
                        sum = __ffma2_rn(big[k][j][h], f[h], sum);
                        const float2 unit = __fmul2_rn(f[h], f2(r1[k]));
                        sum_unit[j][h] = by_row ? __fmul2_rn(d[h], unit) : __ffma2_rn(d[h], unit, sum_unit[j][h]);
                    }
                }
                s[k] = sum.x + sum.y;
            }
            if (by_row) {
                close_gate(r);
#pragma unroll
                for (int j = 0; j < VPT; ++j)
                    if (j * threads + t < nvec && a.dgate)
                        to_global(a.dgate, r, j, t, pack2x<T>(sum_unit[j]));
            }
            if (post) group_sums<ROWS>(s, sums[1][phase], group, warps, threads);
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                const float c1 = cubed(r1[k], s[k] * inv);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = j * threads;
                    if ((!FAST && i + t >= nvec) || !(FULL || k < mine)) break;
                    if (post) {
                        float2 f[H];
                        unpack2<T>(fr[k][j], f);
#pragma unroll
                        for (int h = 0; h < H; ++h)
                            big[k][j][h] = __ffma2_rn(f2(r1[k]), big[k][j][h], __fmul2_rn(f[h], f2(-c1)));
                    }
                    to_global(a.df, r + k, j, t, pack2x<T>(big[k][j]));
                }
            }
            };
            if (mine >= ROWS) rows(std::true_type{});
            else rows(std::false_type{});
            phase ^= 1;
        } else {
            if (t == 0) mbar_arrive(&empty[slot]);  // no row of this slot is this group's
        }
        if (by_gate && (walk.r + walk.count == walk.gate_end || walk.r + walk.count == walk.end)) {
            const bool begins = first == gate_row * a.per_gate.d, ends = walk.r + walk.count == walk.gate_end;
            close_gate(gate_row);
            if (a.dgate)
                flush(sum_unit, part_row(a, begins ? 3 : 2, blockIdx.x), begins && ends ? a.dgate : nullptr, gate_row);
            else clear(sum_unit);
            first = walk.r + walk.count;
            ++gate_row;
        }
    }
    if (!by_gate && !by_row) close_gate(gate_row);
    __syncthreads();
    if (a.dw_post) flush(sum_post, part_row(a, 0, blockIdx.x), nullptr, 0);
    if (a.dw_pre) flush(sum_pre, part_row(a, 1, blockIdx.x), nullptr, 0);
    if (bad) s_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0 && s_bad) {
        atomicOr(a.err, kErrTimeoutStage);
        ask.settle(g, full);
    }
}

// ---------------------------------------------------------------------------
// the chunks' partial rows added, each column in a fixed order with the rounding
// errors carried (the partial rows can be much larger than their sum).  blockIdx.y
// 0 and 1: dw_post, dw_pre; the others the rows of the gate that several chunks
// hold: each of its rows, or, where there are more of them than chunks, the row
// that goes on from one chunk into the next.  The warps of a CTA share a sum's
// partial rows; where the gate's rows are many, and so each has few, a warp takes
// a row of its own (`by_warp`).
// ---------------------------------------------------------------------------
template <typename T, int C>  // C: columns of a lane, 4 where rows of floats are whole vectors (a sum of 152 rows of 4096: 12 -> 7 us)
__global__ void __launch_bounds__(kBlockSumWarps * 32) block_sum_kernel(const BlockArgs a, int by_chunk, int by_warp) {
    __shared__ float part[kBlockSumWarps][2][32 * C + 1];
    pdl_next();
    void* out;
    int64_t c0 = 0, c1 = a.chunks - 1, row = 0;
    int kind = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool alone = by_warp && blockIdx.y >= 2;
    if (blockIdx.y < 2) {
        kind = int(blockIdx.y);
        out = kind == 0 ? a.dw_post : a.dw_pre;
    } else {
        kind = 2;
        out = a.dgate;
        row = alone ? (int64_t(blockIdx.y) - 2) * kBlockSumWarps + warp : int64_t(blockIdx.y) - 2;
        if (row >= (by_chunk ? a.chunks - 1 : a.gates)) return;
        if (by_chunk) {
            const int64_t c = row, r0 = chunk_begin(a, c + 1);
            row = row_div(r0, a.per_gate);
            if (row * a.per_gate.d == r0 || chunk_owner(a, row * a.per_gate.d) != c) return;
        }
        c0 = chunk_owner(a, row * a.per_gate.d);
        c1 = chunk_owner(a, row * a.per_gate.d + a.per_gate.d - 1);
        if (c0 == c1) return;  // written by that chunk
    }
    if (!out) return;
    const int col = (int(blockIdx.x) * 32 + lane) * C;
    // Neumaier's sums
    float s[C] = {}, e[C] = {};
    auto add = [](float& s, float& e, float v) {
        const float t = s + v;
        e += fabsf(s) >= fabsf(v) ? (s - t) + v : (v - t) + s;
        s = t;
    };
    if (col < a.cols) {
        constexpr int AHEAD = 8;
        const int64_t step = alone ? 1 : kBlockSumWarps;
        for (int64_t c = alone ? c0 : c0 + warp; c <= c1; c += AHEAD * step) {
            float v[AHEAD][C];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                const int64_t at = c + k * step;
                if (at > c1) break;
                const float* from = part_row(a, kind == 2 && at == c0 ? 3 : kind, at) + col;
                if constexpr (C == 4) {
                    const uint4 x = ld_after(reinterpret_cast<const uint4*>(from));
                    v[k][0] = __uint_as_float(x.x), v[k][1] = __uint_as_float(x.y);
                    v[k][2] = __uint_as_float(x.z), v[k][3] = __uint_as_float(x.w);
                } else {
                    v[k][0] = ld_after(from);
                }
            }
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) {
                if (c + k * step > c1) break;
#pragma unroll
                for (int i = 0; i < C; ++i) add(s[i], e[i], v[k][i]);
            }
        }
    }
    if (alone) {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (col < a.cols) put<T>(out, row * a.cols + col + i, s[i] + e[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
        part[warp][0][lane * C + i] = s[i];
        part[warp][1][lane * C + i] = e[i];
    }
    __syncthreads();
    const int mine = int(blockIdx.x) * 32 * C + int(threadIdx.x);
    if (threadIdx.x >= 32 * C || mine >= a.cols) return;
    float all = 0.f, lost = 0.f;
#pragma unroll 8
    for (int w = 0; w < kBlockSumWarps; ++w) {
        add(all, lost, part[w][0][threadIdx.x]);
        add(all, lost, part[w][1][threadIdx.x]);
    }
    put<T>(out, row * a.cols + mine, all + lost);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// The ring for four tensors, groups taking `rows` rows at once, behind the weights and the place where the groups' sums
// are added; false: no room for two slots.
template <typename T>
bool block_ring(BlockArgs& a, BlockRing& g, const DevInfo* dev, int vpt, int rows, bool elem, int room) {
    const int nvec = (a.cols + kVec<T> - 1) / kVec<T>;
    g.threads = ((nvec + vpt - 1) / vpt + 31) / 32 * 32;
    if (elem) g.threads = g.threads <= 32 ? 32 : g.threads <= 128 ? 128 : kBlockConsumers;
    g.groups = std::min(kBlockConsumers / g.threads, 14);  // (named barriers)
    g.rows = g.groups * rows;
    g.tensor_bytes = uint32_t(g.rows) * uint32_t(a.cols) * uint32_t(sizeof(T));
    if (elem) g.tensor_bytes = (g.tensor_bytes + 15) / 16 * 16 + 16;  // rounded outwards at both ends
    g.slot_bytes = 4 * g.tensor_bytes;
    // the groups' sums at once, or of a few large ones three and then the others (5 groups of 96 threads: 79 us, all at
    // once, which leaves the L1 cache less, 82; 14 of 32: 34, all at once 32)
    g.places = g.groups > 7 ? g.groups : g.groups > 1 ? std::min(g.groups, 3) : 0;
    const int shares = elem ? vpt * g.threads : nvec;
    g.ring_at = (uint32_t(shares) * 32 + uint32_t(g.places * g.threads) * kVec<T> * 4 + 127) / 128 * 128;
    const int least = int(g.ring_at + 2 * g.slot_bytes), most = dev->max_smem_optin - 2048;
    g.slots = std::min((std::min(most, std::max(room, least)) - int(g.ring_at)) / int(g.slot_bytes), kBlockSlots);
    return g.slots >= 2;
}
inline nrm_status block_ring_launch(const void* fn, BlockArgs& a, BlockRing& g, const DevInfo* dev, cudaStream_t s) {
    // few rows are spread over the GPU, two to a CTA (390 rows of 80, each three with a gate of their own: 22 us; with all
    // the rows of a slot to a CTA 83)
    a.chunks = std::min<int64_t>(dev->sms, (a.rows + 1) / 2);
    const size_t smem = g.ring_at + size_t(g.slots) * g.slot_bytes;
    nrm_status st = prepare_kernel(fn, smem, false);
    if (st != NRM_OK) return st;
    void* p[] = {&a, &g};
    return launch_pdl(fn, dim3(unsigned(a.chunks)), dim3(unsigned(g.groups * g.threads)), p, s, smem);
}

// Rows to a CTA: about 16, such that the CTAs come to whole waves (a wave of 3.4 costs as much as one of 4).
inline nrm_status block_fwd_launch(const void* fn, BlockArgs& a, const DevInfo* dev, int threads, cudaStream_t s) {
    const int64_t resident = int64_t(dev->sms) * std::max(1, cached_occupancy(fn, threads, 0));
    const int64_t waves = (a.rows + 16 * resident - 1) / (16 * resident);
    int per = int((a.rows + waves * resident - 1) / (waves * resident));
    void* p[] = {&a, &per};
    return launch_pdl(fn, dim3(unsigned((a.rows + per - 1) / per)), dim3(unsigned(threads)), p, s);
}
template <typename T, int THREADS, int CTAS>
nrm_status block_fwd_elem(BlockArgs& a, const DevInfo* dev, cudaStream_t s) {
    return block_fwd_launch(reinterpret_cast<const void*>(&block_fwd_elem_kernel<T, THREADS, CTAS>), a, dev, THREADS, s);
}
template <typename T, int VPT, int DEPTH, int MOST, int CTAS>
nrm_status block_fwd_vec(BlockArgs& a, const DevInfo* dev, cudaStream_t s) {
    const int nvec = a.cols / kVec<T>, block = ((nvec + VPT - 1) / VPT + 31) / 32 * 32;
    const void* fn = nvec == VPT * block && a.post && a.h
                         ? reinterpret_cast<const void*>(&block_fwd_vec_kernel<T, VPT, DEPTH, MOST, CTAS, true>)
                         : reinterpret_cast<const void*>(&block_fwd_vec_kernel<T, VPT, DEPTH, MOST, CTAS, false>);
    return block_fwd_launch(fn, a, dev, block, s);
}

template <typename T>
nrm_status block_norm_fwd(const BlockArgs& args, bool vec, cudaStream_t s) {
    BlockArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    if (a.rows == 0) return NRM_OK;
    const int nvec = a.cols / kVec<T>;
    if (vec && nvec <= 2048 && a.rows < (int64_t(1) << 31)) {
        // few rows: all the threads that there are vectors for
        if (nvec <= 512 && a.rows <= 2 * dev->sms) return block_fwd_vec<T, 1, 1, 512, 2>(a, dev, s);
        // a warp to a row of up to 4 vectors a lane, without a barrier; longer rows 2 vectors a thread (what a row costs
        // beside its vectors, 217 of 296 instructions of a warp with one, is then shared by two), the longest 4
        switch ((nvec + 31) / 32) {
        case 1: return block_fwd_vec<T, 1, 3, 32, 28>(a, dev, s);
        case 2: return block_fwd_vec<T, 2, 3, 32, 16>(a, dev, s);
        case 3: return block_fwd_vec<T, 3, 3, 32, 12>(a, dev, s);
        case 4: return block_fwd_vec<T, 4, 2, 32, 12>(a, dev, s);
        default: break;
        }
        if (nvec <= 512) return block_fwd_vec<T, 2, 3, 256, 2>(a, dev, s);
        return nvec <= 1024 ? block_fwd_vec<T, 2, 2, 512, 1>(a, dev, s) : block_fwd_vec<T, 4, 1, 512, 1>(a, dev, s);
    }
    if (a.cols <= 1024 * kBlockElems && a.rows < (int64_t(1) << 31)) {
        const int threads = (a.cols + kBlockElems - 1) / kBlockElems;
        return threads <= 32    ? block_fwd_elem<T, 32, 24>(a, dev, s)
               : threads <= 64  ? block_fwd_elem<T, 64, 16>(a, dev, s)
               : threads <= 128 ? block_fwd_elem<T, 128, 8>(a, dev, s)
               : threads <= 256 ? block_fwd_elem<T, 256, 4>(a, dev, s)
               : threads <= 512 ? block_fwd_elem<T, 512, 2>(a, dev, s)
                                : block_fwd_elem<T, 1024, 1>(a, dev, s);
    }
    void* p[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(&block_fwd_scalar_kernel<T>),
                      dim3(unsigned(std::min<int64_t>(a.rows, int64_t(dev->sms) * 64))), dim3(kBlockThreads), p, s);
}

template <typename T>
nrm_status block_norm_bwd(const BlockArgs& args, bool vec, bool copies, cudaStream_t s) {
    BlockArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    if (a.rows == 0) {
        const size_t row = size_t(a.cols) * sizeof(T);
        for (auto& o : {std::make_pair(a.dw_post, int64_t(1)), std::make_pair(a.dw_pre, int64_t(1)),
                        std::make_pair(a.dgate, a.gates)}) {
            if (!o.first || o.second == 0) continue;
            const cudaError_t e = cudaMemsetAsync(o.first, 0, row * size_t(o.second), s);
            if (e != cudaSuccess) return cuda_status(e, "cudaMemsetAsync");
        }
        return NRM_OK;
    }
    void* p[] = {&a};
    nrm_status st;
    bool sums = a.dgate || a.dw_post || a.dw_pre;
    const int nvec = (a.cols + kVec<T> - 1) / kVec<T>;
    bool ringed = false;
    if ((vec || copies) && nvec <= 2 * kBlockConsumers) {
        static_assert(kBlockConsumers == 512);
        BlockRing g{};
        const bool by_row = a.gates > 0 && a.per_gate.d == 1, elem = !vec;
        const int vpt = nvec > kBlockConsumers ? 2 : 1;
        // two rows of a group at once, for their waits to overlap, where the registers allow
        const bool all = vec && vpt == 1 && !by_row && nvec % 32 == 0 && a.dh && a.dy && a.post;
        // Kernels with branches keep some of their state in local memory, whose cache is what shared memory leaves: theirs
        // is bounded (16 bits, 8192 rows of 6144: 380 us without a bound, 350 with 195 KB, 289 with 163; float32, 17152 of
        // 1878: 249 without, 226 with 195, 253 with 163).
        const int room = all ? dev->max_smem_optin : (sizeof(T) == 2 ? 163 : 195) * 1024;
        // Two rows of a group at once, for their waits to overlap, where the registers allow: in 16 bits only without
        // branches or in groups of one warp (8192 rows of 4095: 243 us with, 201 without; 17168 of 192: 34 and 45).
        const bool two = vpt == 1 && !by_row && (all || sizeof(T) == 4 || nvec <= 32) && block_ring<T>(a, g, dev, 1, 2, elem, room);
        ringed = two || block_ring<T>(a, g, dev, vpt, 1, elem, room);
        const void* fn;
        if (elem) {
            fn = two && g.threads == 32 ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 2, false, 32>)
                 : g.threads == 32      ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 1, false, 32>)
                 : g.threads == 128     ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 1, false, 128>)
                 : vpt == 1             ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 1, false, 512>)
                                        : reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 2, 1, false, 512>);
            if constexpr (sizeof(T) == 4)
                if (two && g.threads > 32)
                    fn = g.threads == 128 ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 2, false, 128>)
                                          : reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 2, false, 512>);
        } else {
            fn = two && all ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 2, true>)
                 : two      ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 2, false>)
                 : vpt == 1 ? reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 1, 1, false>)
                            : reinterpret_cast<const void*>(&block_bwd_ring_kernel<T, 2, 1, false>);
        }
        if (ringed) st = block_ring_launch(fn, a, g, dev, s);
        if (ringed) {
            if (by_row) a.dgate = nullptr;  // done with
            sums = a.dgate || a.dw_post || a.dw_pre;
        }
    }
    if (!ringed) {
        st = launch_pdl(reinterpret_cast<const void*>(&block_bwd_scalar_kernel<T>),
                        dim3(unsigned(std::min<int64_t>(a.rows, int64_t(dev->sms) * 64))), dim3(kBlockThreads), p, s);
        if (st != NRM_OK || !sums) return st;
        st = launch_pdl(reinterpret_cast<const void*>(&block_cols_kernel<T>),
                        dim3(unsigned((a.cols + kBlockThreads - 1) / kBlockThreads), unsigned(a.chunks)),
                        dim3(kBlockThreads), p, s);
    }
    if (st != NRM_OK || !sums) return st;
    int by_chunk = a.gates > a.chunks;
    int64_t gate_rows = a.dgate ? (by_chunk ? a.chunks - 1 : a.gates) : 0;
    int by_warp = gate_rows > 4;
    if (by_warp) gate_rows = (gate_rows + kBlockSumWarps - 1) / kBlockSumWarps;
    void* q[] = {&a, &by_chunk, &by_warp};
    const int columns = a.cols % 4 == 0 ? 128 : 32;
    return launch_pdl(columns == 128 ? reinterpret_cast<const void*>(&block_sum_kernel<T, 4>)
                                     : reinterpret_cast<const void*>(&block_sum_kernel<T, 1>),
                      dim3(unsigned((a.cols + columns - 1) / columns), unsigned(2 + gate_rows)), dim3(kBlockSumWarps * 32), q, s);
}

}  // namespace nrm
