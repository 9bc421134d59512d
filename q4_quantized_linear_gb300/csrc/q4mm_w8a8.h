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
    void *Y;
    int64_t ldy;
    int ytype;
    int m, n, k, np, groups;
};

} // namespace q4
