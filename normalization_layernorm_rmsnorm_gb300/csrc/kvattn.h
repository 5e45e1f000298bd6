// kvattn.h -- host-side declarations of the calls that work on whole cached
// sequences: attention of one new token over the paged cache, and eviction from
// it by weight; shared by their C ABI (kvattn_api.cu) and the kernel
// translation units (kvattn_<dtype>.cu, kvevict.cu).
#pragma once

#include "heads.h"

namespace nrm {

// Sequences of one launch: their work lies in a CTA's shared memory.  A call with
// more is cut into launches.
constexpr int kAttnSequences = 1024;
constexpr int kAttnTile = 32;        // positions of a tile: one to a lane
// What a sequence costs a worker beside its tiles, in tiles: its queries, the first copies' wait, its result.  (0, 2, 5
// and 7 tiles: 64 sequences of 1 to 2048 positions with weights 55.3, 52.3, 50.5, 48.4 us; 250 of up to 120 17.2, 14.8,
// 14.4, 14.7; 16 of up to 16384 on one head of 256 40.8, 39.4, 39.4, 39.4; 9 in a window of 777 20.5, 19.0, 19.1, 19.1;
// one of 131072 in 4 bits 61.2, 60.6, 60.5, 60.5.)
constexpr int kAttnStart = 5;
constexpr int kAttnWarps = 12;       // warps of a CTA at most, each a worker of its own
constexpr int kAttnHeads = 16;       // query heads that a worker takes, at most
constexpr int64_t kAttnTiles = int64_t(1) << 31;  // the work of all pairs of a launch is below it

// Pairs: a head of the cache with a chunk of the query heads that read it.
struct AttnArgs {
    HeadView q, out;          // ts: from sequence to sequence
    CacheDev cache;
    const int64_t* table;
    int64_t table_stride;
    const int64_t* lengths;
    int sequences;            // of this launch
    int hq, hk;
    int shared;               // query heads of a head of the cache: hq / hk
    int heads;                // query heads of a pair, at most
    int chunks;               // pairs of a head of the cache
    int logit_heads;          // heads, made even
    int d;
    int64_t cap;              // positions that a sequence may have
    int64_t window;           // 0: all
    float scale_log2;         // scale * log2(e)
    float* lse;               // [sequences, hq] (nullable)
    float* weights;           // (nullable)
    int64_t weight_ts, weight_hs;
    // workspace
    int* prefix;              // [sequences + 1] work before each sequence
    float* lse2;              // [sequences, hq], base 2
    float* part;              // [shares][pairs][2] partial results
    float* logits;            // [sequences, pairs, logit_stride, logit_heads], base 2 (with weights)
    int64_t logit_stride;
    int workers;
    // on matrix instructions
    int row_bytes, vec;       // of a row of codes, copied in vectors of 16 or 8 bytes
    int snap;                 // pairs of at most so many tiles are not cut
    int q_vec, out_vec;       // queries and outputs are aligned to 16 bytes
    int scale_vec;            // a row's scales are whole aligned 16 bytes
    int near;                 // rows of whole 16 bytes whose places are below 2^32 of them
    int64_t pages;
    unsigned int* err;
};

// The query heads of a head of the cache in chunks of at most `most`, as even as they come.
inline void attn_chunks(AttnArgs& a, int most) {
    a.chunks = (a.shared + most - 1) / most;
    a.heads = (a.shared + a.chunks - 1) / a.chunks;
    a.logit_heads = (a.heads + 1) / 2 * 2;
}
// Tiles of a sequence, at most.
inline int attn_most_tiles(const AttnArgs& a) {
    const int64_t seen = a.window > 0 && a.window < a.cap ? a.window : a.cap;
    return int((seen + kAttnTile - 1) / kAttnTile);
}
// Where there are pairs for a quarter of the workers, short ones are left whole: a worker then takes up to 8 tiles where
// it would have taken 1, but nothing has to be joined.  (250 sequences of up to 120 positions, 4 heads of keys: 14.4 us,
// cut 19.4; 64 of 1 to 2048, 8 heads, of which an eighth are so short: 50.5, cut 47.8.)  Otherwise those of one tile,
// which cannot be cut.
inline void attn_snap(AttnArgs& a) {
    a.snap = 4 * int64_t(a.sequences) * a.hk * a.chunks >= a.workers ? 8 : 1;
}
// Floats of one partial result: accumulator, maximum and sum of each head, in whole 16 bytes.
__host__ __device__ inline int64_t attn_part_row(int d) { return (int64_t(d) + 2 + 3) / 4 * 4; }
__host__ __device__ inline int64_t attn_part_floats(int heads, int d) { return heads * attn_part_row(d); }

// Pairs of a sequence, and floats of a position's logits, at most.
constexpr int kAttnScalarHeads = 4;  // query heads of a worker of the kernel for any layout
inline int64_t attn_most_pairs(int64_t hq, int64_t hk) { return hk * ((hq / hk + kAttnScalarHeads - 1) / kAttnScalarHeads); }
inline int64_t attn_most_logits(int64_t hq, int64_t hk) { return hq + 2 * attn_most_pairs(hq, hk); }

// `vec`: the rows' codes are whole aligned vectors of that many bytes (16 or 8)
// and d and the group are multiples of 16; else 0.
template <typename T> nrm_status kv_attention(const AttnArgs& a, int vec, cudaStream_t s);
// The part of it on matrix instructions (sets a's pairs), for one stored form.
template <typename T, int KIND> nrm_status attn_mma(AttnArgs& a, const DevInfo* dev, cudaStream_t s);

struct EvictArgs {
    CacheDev cache;
    const int64_t* table;
    int64_t table_stride;
    const int64_t* lengths;
    const int64_t* new_table;
    int64_t new_stride;
    int64_t* new_lengths;
    const float* weights;
    int64_t weight_ts, weight_hs;
    float* new_weights;       // (nullable)
    int64_t new_ts, new_hs;
    int64_t* kept;
    int64_t sequences;
    int heads, d;
    int64_t cap;
    int64_t keep, first, recent;
    unsigned int* err;
};
nrm_status kv_evict(const EvictArgs& a, cudaStream_t s);

}  // namespace nrm
