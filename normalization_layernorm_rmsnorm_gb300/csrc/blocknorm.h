// blocknorm.h -- host-side declarations of the norms around a block (the norm
// after it, gate, residual scale and add, the norm before the next), shared by
// their C ABI (blocknorm_api.cu) and the kernel translation units.
#pragma once

#include "heads.h"

namespace nrm {

struct BlockArgs {
    const void* x;
    const void* f;
    const void* gate;       // [gates, cols] (nullable)
    const void* w_post;     // [cols] (nullable)
    const void* w_pre;
    void* y;                // forward output, backward input
    void* h;                // (nullable)
    float* rstd_post;       // forward outputs (nullable), backward inputs
    float* rstd_pre;
    const void* dh;         // (nullable)
    const void* dy;         // (nullable)
    void* dx;
    void* df;
    void* dgate;            // (nullable)
    void* dw_post;
    void* dw_pre;
    int64_t rows;
    int cols;
    int64_t gates;          // 0: no gate
    RowDiv per_gate;        // rows of a gate row
    float alpha, eps;
    int post;
    // the backward's workspace
    float* c2;              // [rows]
    float* part;            // [4][chunks][cols]: dw_post, dw_pre, then a chunk's two pieces of dgate
    int64_t chunks;         // of rows, at most; whose partial sums the columns are added from
    unsigned int* err;
};

// Upper bound of the chunks (of the workspace's partial rows).
inline int block_max_chunks(const DevInfo& d) { return 2 * d.sms; }

// `vec`: rows are whole 16-byte vectors at 16-byte aligned addresses.
template <typename T> nrm_status block_norm_fwd(const BlockArgs& a, bool vec, cudaStream_t s);
// `copies`: dh, dy, f and y are at 16-byte aligned addresses.
template <typename T> nrm_status block_norm_bwd(const BlockArgs& a, bool vec, bool copies, cudaStream_t s);

}  // namespace nrm
