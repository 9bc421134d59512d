// q4mm_moe.h -- the expert sort's and the combining kernels' arguments and
// launchers (internal).
#pragma once

#include "q4mm_internal.h"
#include "q4mm_rows.h"

namespace q4 {

constexpr int kMoeMaxExperts = 4096;
constexpr int kMoeMaxTopK = 1024;
// Most chunks the pairs are cut into for the sort.
constexpr int kMoeMaxChunks = 128;

struct MoeDispatchArgs {
    void *Xs;                // nullptr: no rows are copied
    const void *X;
    int64_t ldxs, ldx;       // bytes
    int64_t bytes;           // of a row
    int64_t *offsets;
    int32_t *row_of, *pair_of;
    const void *ids;
    int id_bytes;
    int64_t tokens, pairs;
    int top_k, experts;
    int32_t *hist;           // [experts + 1][pitch]: pairs of each chunk
    int64_t chunk;           // pairs of a chunk
    int chunks, pitch;
};

struct MoeCombineArgs {
    void *Y;
    const void *base, *Ys;
    int64_t ldy, ldbase, ldys;
    const int32_t *row_of;
    const float *weights;    // nullptr: ones
    int64_t tokens, pairs;
    int top_k;
    int64_t d;
    int segs;                // warps that share a token's columns
};

struct MoeCombineBwdArgs {
    void *dYs;
    float *dweights;         // nullptr: not wanted
    const void *dY, *Ys;
    int64_t lddys, lddy, ldys;
    const int32_t *row_of;
    const float *weights;
    int64_t tokens, pairs;
    int top_k;
    int64_t d;
};

// Scratch bytes of the sort (0 where one launch does it all).
size_t moe_scratch(int64_t pairs, int64_t experts);
// `whole`: every row starts on a 16-byte boundary and is whole 16-byte words.
cudaError_t launch_moe_dispatch(MoeDispatchArgs a, bool whole, int sm_count, cudaStream_t s);
cudaError_t launch_moe_combine(const MoeCombineArgs &a, int type, int vec, cudaStream_t s);
cudaError_t launch_moe_combine_bwd(const MoeCombineBwdArgs &a, int type, int vec, cudaStream_t s);

} // namespace q4
