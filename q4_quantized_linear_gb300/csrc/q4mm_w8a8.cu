// q4mm_w8a8.cu -- the product in 8-bit integers with a scale for each token
// and each channel: Y[t][j] = sx[t] * s_j * sum_c xq[t][c] * code[j][c]. Its
// entry points and the kernel for few tokens; many tokens take the tensor
// cores' GEMM (q4mm_w8a8_gemm.cu).
//
// Few tokens are bound by the weight read, n * k bytes. sm_103a's integer MMA
// and its four-way integer dot product both run at about 256 products a clock
// and SM (measured: 0.5 products a picosecond), enough for ten tokens at the
// rate HBM delivers weights; the fp16 warp MMA does 1024. So codes are turned
// into fp16 (exact), multiplied by mma.sync m16n8k16 and summed in fp32, which
// holds the sums exactly for 1024 columns: every 16 records at the latest a
// warp adds its accumulators to 32-bit integers in shared memory. The integers
// are the exact sums whatever the split, so nothing depends on it.
//
// A warp takes 16 weight rows and a slice of K. A lane's 16-byte load holds 16
// codes of one row: eight rows of a record are 512 contiguous bytes. K is
// permuted to suit: lane (g, t) holds columns 16 t .. 16 t + 15 of rows g and
// g + 8 as the A operands of four MMAs, and the same columns of token g as
// their B operands, read from the token's codes as they are.
//   The slices of a unit of 16 rows are warps of one CTA and meet in shared
// memory. Where the caller declared the weights read-only, a whole batch of
// records is loaded before the dependency wait, so the weight stream starts
// while the tokens are still being coded.
//   GB300, us a call (floor at the measured copy rate): 1 x 9728 x 2560 6.8 (3.7),
// 1 x 2560 x 9728 10 (3.7), 1 x 14336 x 4096 14.7 (8.7), 16 x 14336 x 4096 with the
// norm in front 18.1 (8.8). The loads in flight and their conversion bound it.
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_rows.cuh"
#include "q4mm_w8a8.h"

namespace q4 {
namespace {

constexpr int64_t kMaxK = 131072;      // 127 * 127 * k stays below 2^31
constexpr int kUnitRows = 16;
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kExactRecords = 16;      // 1024 * 127^2 < 2^24

// Four codes (128 + c a byte) as two fp16x2: as the low mantissa byte of 1024
// a byte is the fp16 1152 + c.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    lo = hsub2_bits(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_bits(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u);
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3},{%4,%5,%6,%7},{%8,%9},{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint8_t *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Tokens that each CTA codes for itself: codes in shared memory, rows `stride`
// bytes apart, and their scales.
struct OwnCodes {
    int8_t *codes;
    float *scale;
    int stride;
};

// Codes rows 0 .. m - 1 of X (q4_a8_quantize's rule), a row at a time by the
// whole CTA; columns k .. np * 64 - 1 are zeros.
template <typename X, int V> __device__ __forceinline__ void code_rows(const W8a8Args &a, const OwnCodes &o, float *rbuf)
{
    RowReducer red{rbuf, kWarps, false};
    red.clear(kThreads);
    __syncthreads();
    const int kp = a.np * kPairK;
    for (int t = 0; t < a.m; ++t) {
        const X *xr = static_cast<const X *>(a.X) + t * a.ldx;
        uint32_t mb = 0u;
        for (int c = static_cast<int>(threadIdx.x) * V; c < a.k; c += kThreads * V) {
            const Pack<X, V> v = load_pack<X, V>(xr, c, a.k);
#pragma unroll
            for (int i = 0; i < V; ++i) mb = max(mb, abs_bits(elem(v, i)));
        }
        const CodeScale cs = code_scale(red.max_bits(mb));
        if (threadIdx.x == 0) o.scale[t] = cs.scale;
        for (int c = static_cast<int>(threadIdx.x) * V; c < kp; c += kThreads * V) {
            const Pack<X, V> v = load_pack<X, V>(xr, c, a.k);   // zeros past k; from the first-level cache
            int q[V];
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = code_of(elem(v, i), cs.factor);
            store_pack<int8_t, V>(o.codes + t * o.stride, c, kp, pack_codes<V>(q));
        }
    }
}

// NT: groups of eight tokens; U: records in flight a warp; X: int8_t for coded
// tokens, else the type of rows that each CTA codes for itself (few enough that
// this costs less than a launch of its own).
template <typename T, typename X, int NT, int U, int OCC>
__global__ void __launch_bounds__(kThreads, OCC) few_tokens_kernel(const W8a8Args a)
{
    constexpr bool OWN = sizeof(X) != 1;
    extern __shared__ __align__(16) uint8_t own_smem[];
    __shared__ int32_t sums[kWarps][kUnitRows][8 * NT + 1];
    __shared__ float own_scale[8];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int S = a.slices, slice = warp % S;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kWarps / S) + warp / S;
    const int per = (a.np + S - 1) / S, p0 = slice * per, p1 = min(a.np, p0 + per);
    const int64_t row0 = unit * kUnitRows;
    // units past the last row read the last group's rows and write nothing
    const int64_t urow = min(row0, static_cast<int64_t>(a.groups) * kW8GroupRows - kUnitRows);
    const uint8_t *src = a.W + (urow / kW8GroupRows * a.np) * kW8RecordBytes + (urow % kW8GroupRows + g) * kPairK + 16 * t;
    uint4 w0[U], w1[U];
    // What a kernel in front wrote is visible only past the wait: the weights may
    // be read before it only where the caller declared that none writes them.
    if (!a.prefetch_w) pdl_wait();
    auto load = [&](int u, int p) {
        if (p < p1) {
            const uint8_t *r = src + static_cast<int64_t>(p) * kW8RecordBytes;
            w0[u] = load_stream(r);
            w1[u] = load_stream(r + 8 * kPairK);
        }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) load(u, p0 + u);
    for (int i = lane; i < kUnitRows * (8 * NT + 1); i += 32) (&sums[warp][0][0])[i] = 0;
    pdl_wait();
    pdl_launch_dependents();
    const OwnCodes own{reinterpret_cast<int8_t *>(own_smem), own_scale, a.np * kPairK + (a.np % 2 ? 0 : 64)};
    if constexpr (OWN) {
        if (a.vec * sizeof(X) == 16) code_rows<X, 16 / sizeof(X)>(a, own, rbuf);
        else code_rows<X, 1>(a, own, rbuf);
        __syncthreads();
    }
    const float *const sx = OWN ? own_scale : a.sx;
    // this lane's columns of its tokens, one pointer per group of eight
    const int8_t *xq[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int tok = 8 * j + g;
        xq[j] = tok >= a.m ? nullptr : OWN ? own.codes + tok * own.stride + 16 * t : a.Xq + static_cast<int64_t>(tok) * a.k + 16 * t;
    }
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
    const auto flush = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sums[warp][g + 8 * (i >> 1)][8 * j + 2 * t + (i & 1)] += __float2int_rn(acc[j][i]);
                acc[j][i] = 0.0f;
            }
    };
    int held = 0;
    for (int p = p0; p < p1; p += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p + u >= p1) break;
            uint4 x[NT];
            const int col = (p + u) * kPairK;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                x[j] = make_uint4(0u, 0u, 0u, 0u);
                if constexpr (OWN) {
                    if (xq[j]) x[j] = lds128(xq[j] + col);
                } else if (xq[j] && col + 16 * t < a.k) {
                    x[j] = __ldg(reinterpret_cast<const uint4 *>(xq[j] + col));
                }
            }
            const uint32_t r0[4] = {w0[u].x, w0[u].y, w0[u].z, w0[u].w}, r1[4] = {w1[u].x, w1[u].y, w1[u].z, w1[u].w};
            load(u, p + u + U);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint32_t a0, a1, a2, a3;
                codes_f16(r0[s], a0, a2);
                codes_f16(r1[s], a1, a3);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint32_t xs = s == 0 ? x[j].x : s == 1 ? x[j].y : s == 2 ? x[j].z : x[j].w;
                    uint32_t b0, b1;
                    codes_f16(xs ^ 0x80808080u, b0, b1);   // biased like the weights' codes
                    mma_f16(acc[j], a0, a1, a2, a3, b0, b1);
                }
            }
        }
        held += U;
        if (held + U > kExactRecords) {
            flush();
            held = 0;
        }
    }
    flush();
    __syncthreads();
    // rows next to each other in a thread's neighbours: Y's rows are tokens
    const int units = kWarps / S, rows = units * kUnitRows;
    for (int i = threadIdx.x; i < rows * a.m; i += kThreads) {
        const int r = i % rows, tok = i / rows;
        const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + r;
        if (row >= a.n) continue;
        int32_t s = 0;
        for (int k = 0; k < S; ++k) s += sums[(r / kUnitRows) * S + k][r % kUnitRows][tok];
        static_cast<T *>(a.Y)[tok * a.ldy + row] = from_f32<T>(static_cast<float>(s) * (sx[tok] * a.row_scale[row]));
    }
}

// Two records in flight a warp and as many warps as that leaves registers for
// measured best (16 x 14336 x 4096: 17.0 us with 2 records and 3 CTAs an SM, 18.2
// with 2 and 4, 18.8 with 4 and 3; 1 x 9728 x 2560: 6.7 with 2 and 4, 7.3 with 4
// and 4, 8.8 with 5 and 3).
template <typename T> const void *few_tokens_of(const W8a8Args &a)
{
    if (a.X) {
        return a.xtype == Q4_TYPE_F32   ? reinterpret_cast<const void *>(&few_tokens_kernel<T, float, 1, 2, 4>)
               : a.xtype == Q4_TYPE_F16 ? reinterpret_cast<const void *>(&few_tokens_kernel<T, __half, 1, 2, 4>)
                                        : reinterpret_cast<const void *>(&few_tokens_kernel<T, __nv_bfloat16, 1, 2, 4>);
    }
    return a.m <= 8 ? reinterpret_cast<const void *>(&few_tokens_kernel<T, int8_t, 1, 2, 4>)
                    : reinterpret_cast<const void *>(&few_tokens_kernel<T, int8_t, 2, 2, 3>);
}

// Slices of K: the fewest warps that keep the memory busy (24 an SM), but at
// least two records a warp.
cudaError_t launch_few_tokens(W8a8Args a, int sm_count, cudaStream_t s)
{
    const int64_t units = ceil_div(a.n, kUnitRows);
    a.slices = 1;
    while (a.slices < kWarps && units * a.slices < 24 * static_cast<int64_t>(sm_count) && a.np >= 4 * a.slices) a.slices *= 2;
    const void *fn = a.ytype == Q4_TYPE_F32   ? few_tokens_of<float>(a)
                     : a.ytype == Q4_TYPE_F16 ? few_tokens_of<__half>(a)
                                              : few_tokens_of<__nv_bfloat16>(a);
    const size_t smem = a.X ? static_cast<size_t>(a.m) * (a.np * kPairK + 64) : 0;
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(units, kWarps / a.slices))), dim3(kThreads), smem, s, args);
}

// One token of up to so many values is coded by each CTA for itself (1 x 2560 x
// 9728: 10.2 us, with a launch for the coding 13.4; four tokens of 2560 values
// take 10.2 this way and 8.0 with the launch).
constexpr int64_t kOwnValues = 16384;

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
            void *workspace, q4mm_stream_t stream)
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
        if (!plan_w8a8_gemm(m, k, n, dev.sm_count, &plan)) return Q4_ERR_INVALID_ARG;
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
        g.prefetch_w = weight_prefetch();
        g.m = static_cast<int>(m);
        g.n = static_cast<int>(n);
        return cuda_status(launch_w8a8_gemm(plan, g, tok, k, ws + image_at(m, k), dev.sm_count, s));
    }
    const bool own = !coded && m == 1 && k <= kOwnValues;
    if (!coded && !own) {
        rc = quantize_rows(reinterpret_cast<int8_t *>(ws), k, tok.sx, tok.X, tok.ldx, tok.xtype, m, k, dev.sm_count, s);
        if (rc != Q4_OK) return rc;
        tok.Xq = reinterpret_cast<const int8_t *>(ws);
    }
    W8a8Args a{};
    a.W = W;
    a.Xq = tok.Xq;
    if (own) {
        a.X = tok.X;
        a.ldx = tok.ldx;
        a.xtype = tok.xtype;
        a.vec = tok.vec;
    }
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
    a.prefetch_w = weight_prefetch();
    return cuda_status(launch_few_tokens(a, dev.sm_count, s));
}

} // namespace
} // namespace q4

using namespace q4;

extern "C" {

Q4MM_API size_t q4_w8a8_workspace_size(int64_t m, int64_t k, int64_t n)
{
    if (m <= 0 || !valid_sizes(m, k, n)) return 0;
    return image_at(m, k) + (m > kFewTokens ? w8a8_gemm_bytes(m, k, n) : 0);
}

Q4MM_API int q4_w8a8_matmul(const void *W8_packed, const void *X, int64_t ldx, int xtype, void *Y, int64_t ldy,
                            int ytype, int64_t m, int64_t k, int64_t n, void *workspace, size_t workspace_bytes,
                            q4mm_stream_t stream)
{
    if (!W8_packed || (m != 0 && (!X || !Y)) || !is_float_type(xtype) || !is_float_type(ytype) || !valid_sizes(m, k, n) || ldx < k ||
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
    return guarded([&] { return product(W8_packed, tok, Y, ldy, ytype, m, k, n, workspace, stream); });
}

Q4MM_API int q4_w8a8_matmul_codes(const void *W8_packed, const int8_t *Xq, const float *sx, void *Y, int64_t ldy,
                                  int ytype, int64_t m, int64_t k, int64_t n, void *workspace, size_t workspace_bytes,
                                  q4mm_stream_t stream)
{
    if (!W8_packed || (m != 0 && (!Xq || !sx || !Y)) || !is_float_type(ytype) || !valid_sizes(m, k, n) || ldy < n)
        return Q4_ERR_INVALID_ARG;
    if (!aligned_to(W8_packed, 16) || !aligned_to(Xq, 16) || !aligned_to(sx, 4) || !aligned_to(Y, type_size(ytype)) ||
        (workspace && !aligned_to(workspace, 256)))
        return Q4_ERR_ALIGNMENT;
    if (m == 0) return Q4_OK;
    if (!workspace || workspace_bytes < q4_w8a8_workspace_size(m, k, n)) return Q4_ERR_WORKSPACE;
    W8a8Tokens tok;
    tok.Xq = Xq;
    tok.sx = const_cast<float *>(sx);   // read only: the codes are there
    return guarded([&] { return product(W8_packed, tok, Y, ldy, ytype, m, k, n, workspace, stream); });
}

} // extern "C"
