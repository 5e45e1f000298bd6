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
// any layout: a CTA for each row
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
            c2 = r2 * r2 * r2 * (cta_sum(s, sums) / cols);
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
        const float c1 = r1 * r1 * r1 * (cta_sum(s, sums) / cols);
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
// the chunks' partial rows added, each column in a fixed order with the rounding
// errors carried (the partial rows can be much larger than their sum).  blockIdx.y
// 0 and 1: dw_post, dw_pre; the others the rows of the gate that several chunks
// hold: each of its rows, or, where there are more of them than chunks, the row
// that goes on from one chunk into the next.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kBlockSumWarps * 32) block_sum_kernel(const BlockArgs a, int by_chunk) {
    __shared__ float part[kBlockSumWarps][2][33];
    pdl_next();
    void* out;
    int64_t c0 = 0, c1 = a.chunks - 1, row = 0;
    int kind = 0;
    if (blockIdx.y < 2) {
        kind = int(blockIdx.y);
        out = kind == 0 ? a.dw_post : a.dw_pre;
    } else {
        kind = 2;
        out = a.dgate;
        row = int64_t(blockIdx.y) - 2;
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
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = int(blockIdx.x) * 32 + lane;
    // Neumaier's sum
    float s = 0.f, e = 0.f;
    auto add = [&](float v) {
        const float t = s + v;
        e += fabsf(s) >= fabsf(v) ? (s - t) + v : (v - t) + s;
        s = t;
    };
    if (col < a.cols) {
#pragma unroll 4
        for (int64_t c = c0 + warp; c <= c1; c += kBlockSumWarps)
            add(ld_after(part_row(a, kind == 2 && c == c0 ? 3 : kind, c) + col));
    }
    part[warp][0][lane] = s;
    part[warp][1][lane] = e;
    __syncthreads();
    if (warp != 0 || col >= a.cols) return;
    s = e = 0.f;
#pragma unroll 8
    for (int w = 0; w < kBlockSumWarps; ++w) {
        add(part[w][0][lane]);
        add(part[w][1][lane]);
    }
    put<T>(out, row * a.cols + col, s + e);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
template <typename T>
nrm_status block_norm_fwd(const BlockArgs& args, bool vec, cudaStream_t s) {
    BlockArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    (void)vec;
    if (a.rows == 0) return NRM_OK;
    void* p[] = {&a};
    return launch_pdl(reinterpret_cast<const void*>(&block_fwd_scalar_kernel<T>),
                      dim3(unsigned(std::min<int64_t>(a.rows, int64_t(dev->sms) * 64))), dim3(kBlockThreads), p, s);
}

template <typename T>
nrm_status block_norm_bwd(const BlockArgs& args, bool vec, cudaStream_t s) {
    BlockArgs a = args;
    const DevInfo* dev = dev_info();
    if (!dev) return fail(NRM_ERR_CUDA, "no usable CUDA device");
    a.err = dev->err;
    (void)vec;
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
    nrm_status st = launch_pdl(reinterpret_cast<const void*>(&block_bwd_scalar_kernel<T>),
                               dim3(unsigned(std::min<int64_t>(a.rows, int64_t(dev->sms) * 64))), dim3(kBlockThreads),
                               p, s);
    if (st != NRM_OK || (!a.dgate && !a.dw_post && !a.dw_pre)) return st;
    st = launch_pdl(reinterpret_cast<const void*>(&block_cols_kernel<T>),
                    dim3(unsigned((a.cols + kBlockThreads - 1) / kBlockThreads), unsigned(a.chunks)),
                    dim3(kBlockThreads), p, s);
    if (st != NRM_OK) return st;
    int by_chunk = a.gates > a.chunks;
    const int64_t gate_rows = a.dgate ? (by_chunk ? a.chunks - 1 : a.gates) : 0;
    void* q[] = {&a, &by_chunk};
    return launch_pdl(reinterpret_cast<const void*>(&block_sum_kernel<T>),
                      dim3(unsigned((a.cols + 31) / 32), unsigned(2 + gate_rows)), dim3(kBlockSumWarps * 32), q, s);
}

}  // namespace nrm
