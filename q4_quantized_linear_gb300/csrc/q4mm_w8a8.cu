// q4mm_w8a8.cu -- the product in 8-bit integers with a scale for each token
// and each channel: Y[t][j] = sx[t] * s_j * sum_c xq[t][c] * code[j][c].
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_rows.cuh"
#include "q4mm_w8a8.h"

namespace q4 {
namespace {

constexpr int64_t kMaxK = 131072;   // 127 * 127 * k stays below 2^31
constexpr int kTok = 16;            // tokens of a CTA
constexpr int kThreads = 256;

template <typename T> __global__ void __launch_bounds__(kThreads) product_kernel(const W8a8Args a)
{
    __shared__ uint32_t w[kW8GroupRows][17];
    __shared__ uint32_t x[kTok][16];
    pdl_wait();
    const int tid = threadIdx.x, r = tid & 127, half = tid >> 7;
    const int G = blockIdx.x, t0 = blockIdx.y * kTok;
    int acc[kTok / 2] = {};
    for (int p = 0; p < a.np; ++p) {
        const uint32_t *rec = reinterpret_cast<const uint32_t *>(a.W + (static_cast<int64_t>(G) * a.np + p) * kW8RecordBytes);
        for (int i = tid; i < kW8RecordBytes / 4; i += kThreads) w[i >> 4][i & 15] = rec[i] ^ 0x80808080u;
        {
            const int t = tid >> 4, c = tid & 15, col = p * kPairK + 4 * c;
            x[t][c] = t0 + t < a.m && col < a.k
                          ? *reinterpret_cast<const uint32_t *>(a.Xq + static_cast<int64_t>(t0 + t) * a.k + col)
                          : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int t = 0; t < kTok / 2; ++t)
                acc[t] = __dp4a(static_cast<int>(w[r][c]), static_cast<int>(x[half * (kTok / 2) + t][c]), acc[t]);
        __syncthreads();
    }
    const int row = G * kW8GroupRows + r;
    if (row >= a.n) return;
    const float sw = a.row_scale[row];
    for (int t = 0; t < kTok / 2; ++t) {
        const int tok = t0 + half * (kTok / 2) + t;
        if (tok < a.m)
            static_cast<T *>(a.Y)[tok * a.ldy + row] = from_f32<T>(static_cast<float>(acc[t]) * (a.sx[tok] * sw));
    }
}

cudaError_t launch_product(W8a8Args a, cudaStream_t s)
{
    const void *fn = a.ytype == Q4_TYPE_F32   ? reinterpret_cast<const void *>(&product_kernel<float>)
                     : a.ytype == Q4_TYPE_F16 ? reinterpret_cast<const void *>(&product_kernel<__half>)
                                              : reinterpret_cast<const void *>(&product_kernel<__nv_bfloat16>);
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(a.groups), static_cast<unsigned>(ceil_div(a.m, kTok))), dim3(kThreads),
                      0, s, args);
}

bool valid_sizes(int64_t m, int64_t k, int64_t n)
{
    return m >= 0 && m <= (int64_t(1) << 20) && n >= 1 && n <= (int64_t(1) << 31) - 256 && k >= 32 && k % 32 == 0 && k <= kMaxK;
}

// The workspace: codes [m x k], scales [m], the tokens' tiles.
size_t codes_bytes(int64_t m, int64_t k) { return static_cast<size_t>(round_up(m * k, 256)); }
size_t image_at(int64_t m, int64_t k) { return codes_bytes(m, k) + static_cast<size_t>(round_up(4 * m, 256)); }

constexpr int64_t kFewTokens = 16;

// `tok`: codes with their scales, or rows to be coded.
int product(const void *W8, W8a8Tokens tok, void *Y, int64_t ldy, int ytype, int64_t m, int64_t k, int64_t n,
            void *workspace, size_t workspace_bytes, q4mm_stream_t stream)
{
    DeviceInfo dev;
    int rc = device_info(&dev);
    if (rc != Q4_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool coded = tok.Xq != nullptr;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    if (!coded) tok.sx = reinterpret_cast<float *>(ws + codes_bytes(m, k));
    const uint8_t *W = static_cast<const uint8_t *>(W8);
    const int np = static_cast<int>(ceil_div(k, kPairK)), groups = static_cast<int>(ceil_div(n, kW8GroupRows));
    const float *row_scale = reinterpret_cast<const float *>(W + static_cast<size_t>(groups) * np * kW8RecordBytes);
    if (m > kFewTokens) {
        W8a8GemmPlan plan;
        if (!plan_w8a8_gemm(m, k, n, &plan)) return Q4_ERR_INVALID_ARG;
        if (workspace_bytes < image_at(m, k) + plan.image_bytes) return Q4_ERR_WORKSPACE;
        W8a8GemmArgs g{};
        g.W = W;
        g.np = np;
        g.groups = groups;
        g.row_scale = row_scale;
        g.sx = tok.sx;
        g.Y = Y;
        g.ldy = ldy;
        g.ytype = ytype;
        g.status = dev.status;
        g.wait_ns = wait_limit();
        g.m = static_cast<int>(m);
        g.n = static_cast<int>(n);
        return cuda_status(launch_w8a8_gemm(plan, g, tok, k, ws + image_at(m, k), dev.sm_count, s));
    }
    if (!coded) {
        rc = quantize_rows(reinterpret_cast<int8_t *>(ws), k, tok.sx, tok.X, tok.ldx, tok.xtype, m, k, dev.sm_count, s);
        if (rc != Q4_OK) return rc;
        tok.Xq = reinterpret_cast<const int8_t *>(ws);
    }
    W8a8Args a{};
    a.W = W;
    a.Xq = tok.Xq;
    a.sx = tok.sx;
    a.Y = Y;
    a.ldy = ldy;
    a.ytype = ytype;
    a.m = static_cast<int>(m);
    a.n = static_cast<int>(n);
    a.k = static_cast<int>(k);
    a.np = np;
    a.groups = groups;
    a.row_scale = row_scale;
    return cuda_status(launch_product(a, s));
}

} // namespace
} // namespace q4

using namespace q4;

extern "C" {

Q4MM_API size_t q4_w8a8_workspace_size(int64_t m, int64_t k, int64_t n)
{
    if (m <= 0 || !valid_sizes(m, k, n)) return 0;
    W8a8GemmPlan plan;
    if (m > kFewTokens && plan_w8a8_gemm(m, k, n, &plan)) return image_at(m, k) + plan.image_bytes;
    return image_at(m, k);
}

Q4MM_API int q4_w8a8_matmul(const void *W8_packed, const void *X, int64_t ldx, int xtype, void *Y, int64_t ldy,
                            int ytype, int64_t m, int64_t k, int64_t n, void *workspace, size_t workspace_bytes,
                            q4mm_stream_t stream)
{
    if (!W8_packed || !X || !Y || !is_float_type(xtype) || !is_float_type(ytype) || !valid_sizes(m, k, n) || ldx < k ||
        ldy < n)
        return Q4_ERR_INVALID_ARG;
    if (!aligned_to(W8_packed, 16) || !aligned_to(X, type_size(xtype)) || !aligned_to(Y, type_size(ytype)) ||
        (workspace && !aligned_to(workspace, 256)))
        return Q4_ERR_ALIGNMENT;
    if (m == 0) return Q4_OK;
    if (!workspace || workspace_bytes < q4_w8a8_workspace_size(m, k, n)) return Q4_ERR_WORKSPACE;
    const int size = type_size(xtype);
    RowAlign al;
    al.add(X, ldx * size);
    W8a8Tokens tok;
    tok.X = X;
    tok.ldx = ldx;
    tok.xtype = xtype;
    tok.vec = al.bytes() >= 16 ? 16 / size : size == 2 && al.bytes() >= 4 ? 2 : 1;
    return product(W8_packed, tok, Y, ldy, ytype, m, k, n, workspace, workspace_bytes, stream);
}

Q4MM_API int q4_w8a8_matmul_codes(const void *W8_packed, const int8_t *Xq, const float *sx, void *Y, int64_t ldy,
                                  int ytype, int64_t m, int64_t k, int64_t n, void *workspace, size_t workspace_bytes,
                                  q4mm_stream_t stream)
{
    if (!W8_packed || !Xq || !sx || !Y || !is_float_type(ytype) || !valid_sizes(m, k, n) || ldy < n)
        return Q4_ERR_INVALID_ARG;
    if (!aligned_to(W8_packed, 16) || !aligned_to(Xq, 16) || !aligned_to(sx, 4) || !aligned_to(Y, type_size(ytype)) ||
        (workspace && !aligned_to(workspace, 256)))
        return Q4_ERR_ALIGNMENT;
    if (m == 0) return Q4_OK;
    if (!workspace || workspace_bytes < q4_w8a8_workspace_size(m, k, n)) return Q4_ERR_WORKSPACE;
    W8a8Tokens tok;
    tok.Xq = Xq;
    tok.sx = const_cast<float *>(sx);   // read only: the codes are there
    return product(W8_packed, tok, Y, ldy, ytype, m, k, n, workspace, workspace_bytes, stream);
}

} // extern "C"
