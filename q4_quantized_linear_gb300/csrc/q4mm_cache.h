// q4mm_cache.h -- the paged cache of keys and values, the attention over it,
// and the verification of drafted tokens: layout, arguments and launchers
// (internal).
//
// A page holds page_tokens tokens of every head. The block of a head in it:
//   K  [chunk of 64 dims][token][64 values]
//   V  the same
//   K scales [token], V scales [token]   fp32, of a cache of int8 codes only
// The 16-byte units of a row of 64 values are permuted among themselves by the
// token's number: unit u of 16-bit values (8 a row of 128 bytes) stands at u ^
// (t & 7), of codes (4 a row of 64 bytes) at u ^ ((t >> 1) & 3). So a chunk's rows
// are one contiguous copy that lands in shared memory as the 128-byte swizzled
// image that the tensor cores read (16-bit values), or without bank conflicts
// for a warp that reads 8 tokens' rows (codes). Dims past d are zeros.
#pragma once

#include "q4mm_internal.h"
#include "q4mm_rows.h"

namespace q4 {

constexpr int kMaxSeqs = 1024;      // sequences of a call
constexpr int kMaxHeadDim = 256;
constexpr int64_t kMaxVerifyVocab = int64_t(1) << 20;
constexpr int kChunk = 64;          // dims of a chunk
constexpr int kErrTimeout = 5, kErrCheck = 10;   // Q4_ERR_DEVICE_TIMEOUT, Q4_ERR_DEVICE_CHECK

struct KvCache {
    uint8_t *pages;
    int64_t page_bytes;
    uint32_t head_bytes;
    int n_pages, page_tokens, log_page, heads, d, chunks, type;
    const int32_t *table;     // [n_seq x ldt]: a sequence's pages in order
    int64_t ldt;
    int capacity;             // tokens that a row of the table can hold
};

inline int log2_of(int64_t x)
{
    int n = 0;
    while ((int64_t(1) << n) < x) ++n;
    return n;
}
inline uint32_t kv_head_bytes(int64_t page_tokens, int64_t d, int ctype)
{
    const int64_t dp = round_up(d, kChunk);
    return static_cast<uint32_t>(page_tokens * (2 * dp * type_size(ctype) + (ctype == Q4_TYPE_I8 ? 8 : 0)));
}

// Rows of K and V (heads next to each other) to the cache, or back.
struct KvRowsArgs {
    KvCache c;
    void *K, *V;              // read by the write, written by the read
    int64_t ldk, ldv;
    const int32_t *at;        // write: lens; read: first positions (nullptr: zeros)
    const int32_t *starts;
    int n_seq;
    int64_t rows;
    int *status;
};
cudaError_t launch_kv_write(const KvRowsArgs &a, int type, bool vec, int sm_count, cudaStream_t s);
cudaError_t launch_kv_read(const KvRowsArgs &a, int type, bool vec, int sm_count, cudaStream_t s);

// Most CTAs of the attention's kernels: what the scratch is laid out for.
constexpr int kAttnMaxCtas = 480, kTensorMaxCtas = 160;
constexpr int kWarpTile = 64;       // tokens of a tile of the warp-MMA kernel
constexpr int kTensorRows = 256, kTensorTile = 128;   // query rows and tokens of a tile of the tcgen05 kernel
// Query rows of a sequence and head (new tokens x query heads that share it)
// above which the tcgen05 kernel takes it.
constexpr int kWarpRows = 64;

struct AttnArgs {
    KvCache c;
    void *O;
    const void *Q;
    int64_t ldo, ldq;
    int type;
    int vec;                  // O's and Q's rows start on 16-byte boundaries
    int group;                // query heads of a cached head
    float scale_log2;         // scale * log2(e)
    int window;               // 0: none
    const int32_t *lens, *starts;
    int n_seq;
    int rows;
    int rows_above, rows_upto;   // the sequences this launch takes: query rows in (above, upto]
    int tile, block;          // tokens of a tile, query rows of a block
    int item_cost;            // tiles' worth of work that an item costs beside its tiles
    int stages;
    float *parts;             // [2 * CTAs] of block x (64 * chunks) sums, then [block] maxima and sums
    int4 *meta;               // [CTAs][2]: an item whose parts are to be joined
    int *status;
    uint64_t wait_ns;
};

// Floats of a part.
__host__ __device__ inline int64_t attn_part_floats(int block, int chunks)
{
    return static_cast<int64_t>(block) * (kChunk * chunks + 2);
}
cudaError_t launch_attn_warp(AttnArgs a, int sm_count, cudaStream_t s);
cudaError_t launch_attn_tensor(AttnArgs a, int sm_count, cudaStream_t s);
cudaError_t launch_attn_join(const AttnArgs &a, int ctas, cudaStream_t s);

struct ProbsArgs {
    float *P;
    const void *X;
    int64_t ldp, ldx;
    const float *temperature;
    int64_t rows, n;
    int *status;
    uint64_t wait_ns;
};
cudaError_t launch_token_probs(const ProbsArgs &a, int type, int sm_count, cudaStream_t s);

struct VerifyArgs {
    int32_t *tokens, *kept;
    const float *P, *Q;       // Q nullptr: the draft was sure of its tokens
    int64_t ldt, ldp, ldq;
    const int32_t *drafted, *counts;
    int64_t ldd;
    const float *accept, *sample;
    int64_t lda;
    int64_t n_seq, n;
    int max_draft;
};
cudaError_t launch_draft_verify(const VerifyArgs &a, int sm_count, cudaStream_t s);

} // namespace q4
