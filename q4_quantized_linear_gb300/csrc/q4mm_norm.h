// q4mm_norm.h -- the norm kernels' arguments and launchers (internal).
#pragma once

#include "q4mm_internal.h"
#include "q4mm_rows.h"

namespace q4 {

// Most rows of partial column sums of a backward call.
constexpr int kNormPartials = 608;

// Rows that are a multiple of this apart start alike within 16 bytes, whatever
// their stride (elements have 2 bytes or more).
constexpr int64_t kRowStep = 8;
inline int64_t round_row_step(int64_t rows) { return rows < kRowStep ? kRowStep : rows / kRowStep * kRowStep; }

// Where a normed row goes: values of the input's type, or int8 codes and a
// scale per row. H == nullptr: nowhere.
struct NormOut {
    void *H;
    int64_t ldh;
    int codes;
    float *h_scale;
    const float *w;      // nullptr: weights of 1
    float w_off;
};

struct NormBeforeArgs {
    NormOut out;
    const void *X;
    int64_t ldx;
    int plain;           // no norm: h = x (the coding of tokens alone)
    float eps;
    int64_t m, d;
    int G;               // threads of a row
};

struct NormAfterArgs {
    NormOut out;         // the next block's norm
    float out_eps;
    void *Y;
    const void *R, *B;
    int64_t ldy, ldr, ldb;
    const float *w;
    float w_off;
    const void *gate;    // fp32 per channel or token; the matrices' type per value
    int64_t ldg;
    int gate_kind;
    float scale, eps;
    int64_t m, d;
    int *status;
    uint64_t wait_ns;
    int G;
};

struct NormBeforeBwdArgs {
    void *dX;
    const void *dH, *dR, *X;   // dR may be nullptr
    int64_t lddx, lddh, lddr, ldx;
    const float *w;
    float w_off, eps;
    float *partials;           // nullptr: no column sums are wanted
    int64_t m, d;
    int *status;
    uint64_t wait_ns;
    int G;
};

struct NormAfterBwdArgs {
    void *dB, *dgate;
    const void *dY, *B, *gate;
    int64_t lddb, lddg, lddy, ldb, ldg;
    const float *w;
    float w_off;
    int gate_kind;
    float scale, eps;
    float *partials;
    int64_t m, d;
    int *status;
    uint64_t wait_ns;
    int G;
};

struct NormColumnArgs {
    const float *partials;
    int rows;
    int64_t d;
    float scale;
    float *dw, *dgate;
    const float *gate, *w;
    float w_off;
};

// The streaming kernels: a CTA per row in turn, the rows of up to `matrices`
// inputs copied ahead into a ring in shared memory.
struct NormStreamPlan {
    int NV = 0;            // 16-byte vectors a thread
    int G = 0;             // threads
    int stages = 0;
    int64_t ctas = 0;
    size_t smem = 0;
    bool any = false;      // rows start anywhere
};
// False where they do not apply: short or very long rows, few rows.
bool plan_norm_stream(int64_t m, int64_t d, int type, bool any, int matrices, int sm_count, NormStreamPlan *plan);
cudaError_t launch_norm_after_stream(const NormStreamPlan &p, const NormAfterArgs &a, int type, cudaStream_t s);
cudaError_t launch_norm_after_stream_any(const NormStreamPlan &p, const NormAfterArgs &a, int type, cudaStream_t s);
cudaError_t launch_norm_before_bwd_stream(const NormStreamPlan &p, const NormBeforeBwdArgs &a, int type, cudaStream_t s);
cudaError_t launch_norm_before_bwd_stream_any(const NormStreamPlan &p, const NormBeforeBwdArgs &a, int type, cudaStream_t s);
cudaError_t launch_norm_after_bwd_stream(const NormStreamPlan &p, const NormAfterBwdArgs &a, int type, cudaStream_t s);
cudaError_t launch_norm_after_bwd_stream_any(const NormStreamPlan &p, const NormAfterBwdArgs &a, int type, cudaStream_t s);

cudaError_t launch_norm_before(const NormBeforeArgs &a, int type, const RowAccess &acc, int sm_count, cudaStream_t s);
cudaError_t launch_norm_after(const NormAfterArgs &a, int type, const RowAccess &acc, int sm_count, cudaStream_t s);
cudaError_t launch_norm_before_bwd(const NormBeforeBwdArgs &a, float *dw, int type, const RowAccess &acc, int sm_count, cudaStream_t s);
cudaError_t launch_norm_after_bwd(const NormAfterBwdArgs &a, float *dw, int type, const RowAccess &acc, int sm_count, cudaStream_t s);

} // namespace q4
