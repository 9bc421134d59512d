// q4mm_w8a8.h -- the int8 product's interfaces between translation units.
#pragma once

#include "q4mm_internal.h"
#include "q4mm_rows.h"

namespace q4 {

// Rows coded to int8 (q4_a8_quantize's rule) by the norm's kernel.
int quantize_rows(int8_t *Xq, int64_t ldq, float *sx, const void *X, int64_t ldx, int type, int64_t m, int64_t k,
                  int sm_count, cudaStream_t s);

struct W8a8Args {
    const uint8_t *W;         // int8 records, codes stored as 128 + c
    const float *row_scale;
    const int8_t *Xq;         // [m x k]
    const float *sx;
    const void *X;            // else rows that each CTA codes, `vec` elements an access
    int64_t ldx;
    int xtype, vec;
    void *Y;
    int64_t ldy;
    int ytype;
    int m, n, k, np, groups;
    int slices;               // of K: warps of a CTA that share 16 rows
    int prefetch_w;           // read W before waiting on the preceding kernel
};

// The tensor-core product (many tokens).
struct W8a8GemmPlan {
    int N = 0;                // tokens of a tile: a multiple of 32, at most 256
    int ts = 0;               // token tiles
    int kslices = 1;          // of K: each slice of a tile is one of `tiles`
    int tiles = 0;            // (256 rows) x (N tokens) x (K slice)
    int pairs = 0;            // CTA pairs of the grid, each taking tiles in turn
    int astages = 0, bstages = 0, wring = 0;
    size_t smem = 0;
    size_t image_bytes = 0;   // the tokens' fp16 tiles; 256-byte aligned; the slices' sums are behind them
};

struct W8a8GemmArgs {
    const uint8_t *W;
    const float *row_scale;
    const uint8_t *ximg;
    const float *sx;
    void *Y;
    int64_t ldy;
    int ytype;
    int *status;
    uint64_t wait_ns;
    int m, n, np, groups;
    int N, ts, tiles, kslices;
    int64_t slice_stride;     // elements from a slice's sums to the next's
    int astages, bstages, wring;
    int prefetch_w;           // read W before waiting on the preceding kernels
};

// Scratch of the tokens' tiles and the slices' sums that every plan for up to m
// tokens fits into: a workspace for a batch serves the smaller ones too.
size_t w8a8_gemm_bytes(int64_t m, int64_t k, int64_t n);
bool plan_w8a8_gemm(int64_t m, int64_t k, int64_t n, int sm_count, W8a8GemmPlan *plan);
// The tokens of a call: codes, or rows to be coded (their scales then go to
// sx; `vec` elements an access).
struct W8a8Tokens {
    const int8_t *Xq = nullptr;
    const void *X = nullptr;
    int64_t ldx = 0;
    int xtype = 0, vec = 1;
    float *sx = nullptr;
};
// The tokens' fp16 tiles, then the product.
cudaError_t launch_w8a8_gemm(const W8a8GemmPlan &plan, const W8a8GemmArgs &args, const W8a8Tokens &tokens, int64_t k,
                             uint8_t *ximg, int sm_count, cudaStream_t s);

} // namespace q4
