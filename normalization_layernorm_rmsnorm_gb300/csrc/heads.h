// heads.h -- host-side declarations of the operators on attention heads (norms
// with position rotation, quantised key/value cache), shared by their C ABI
// (heads_api.cu) and the per-dtype kernel translation units (heads_<dtype>.cu).
#pragma once

#include "internal.h"

namespace nrm {

constexpr int kHeadMaxD = 256;              // elements of a head
constexpr int kHeadMaxPairs = kHeadMaxD / 2;
constexpr int kHeadMaxAxes = 4;

// The bit of the library's error word that reports a cache slot outside its
// cache (the low bits report waits that gave up).
constexpr unsigned int kErrCacheSlot = 1u << 8;

// Division of a row or slot number by a fixed divisor: a multiplication where
// every dividend is below 2^32, else the 64-bit division.
struct RowDiv {
    int64_t d;
    uint64_t m;
    int small;
};
inline RowDiv make_row_div(int64_t d, int64_t below) {
    const bool small = d < (int64_t(1) << 32) && below <= (int64_t(1) << 32);
    return RowDiv{d, small ? make_fast_div(uint32_t(d)).m : 0, small};
}

// A [tokens, heads, d] view; strides in elements.
struct HeadView {
    void* p;
    int64_t ts, hs;
};

// The rotation; the axis of each pair as two bits.
struct RopeDev {
    const int64_t* pos;
    int64_t pos_stride;
    const float* inv_freq;
    uint32_t axis[kHeadMaxPairs / 16];
    int rot;
    int axes;
    int adjacent;   // pair p is (2p, 2p+1), else (p, p + rot/2)
    int inverse;    // turn the other way
};

// The cache's rows; byte and float strides.
struct CacheDev {
    uint8_t* codes[2];   // k, v
    float* scales[2];
    int64_t slots;       // pages * page_size
    RowDiv page;         // by page_size
    int flat;            // pages follow one another slot by slot: a slot's place needs no division
    int64_t page_stride, slot_stride, head_stride;
    int64_t scale_page_stride, scale_slot_stride, scale_head_stride;
    int group;
    int kind;            // nrm_cache_kind
};

// Tensor 0 is q, 1 is k, 2 is v (the cache-writing form only).
struct HeadArgs {
    HeadView x[3];
    HeadView y[2];
    HeadView dy[2];       // backward
    const void* w[2];     // [d] in the storage dtype (nullable)
    float* rstd[2];       // forward output (nullable), backward input
    float* ws;            // backward: partial rows [P][d], q's then k's
    void* dw[2];          // backward outputs [d] (nullable)
    int64_t tokens;
    int heads[3];
    int d;
    float eps;
    RopeDev rope;
    CacheDev cache;
    const int64_t* slots;
    unsigned int* err;
};

// `vec`: the widest accesses (16 or 8 bytes, 4 of a 16-bit type) that every pointer, stride, d, rot
// and group fits, or 0.
template <typename T> nrm_status head_fwd(const HeadArgs& a, bool norm, bool cache, int vec, cudaStream_t s);
template <typename T> nrm_status head_bwd(const HeadArgs& a, int vec, cudaStream_t s);
// Cache rows of a.x[1], a.x[2] (written) or to a.y[0], a.y[1] (read), heads[1] each.
template <typename T> nrm_status cache_write(const HeadArgs& a, int vec, cudaStream_t s);
template <typename T> nrm_status cache_read(const HeadArgs& a, int vec, cudaStream_t s);

// Upper bound of the backward's partial rows.
int head_bwd_max_partials(const DevInfo& d);

}  // namespace nrm
