// q4mm_attn.cu -- the attention's launches by kind, and the join of what was cut.
#include <algorithm>

#include "q4mm_attn.cuh"

namespace q4 {

cudaError_t launch_attn_f16(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas);
cudaError_t launch_attn_f16x2(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas);
cudaError_t launch_attn_bf16(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas);
cudaError_t launch_attn_i8(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas);
cudaError_t launch_attn_i8x2(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas);

namespace {

constexpr int kJoinThreads = 256;

// Four dims of a row out.
__device__ __forceinline__ void store4(const AttnArgs &a, int64_t out, int dim, const float (&v)[4])
{
    if (dim >= a.c.d) return;                               // (d is a multiple of 8)
    if (a.type == Q4_TYPE_F32) {
        float *o = static_cast<float *>(a.O) + out + dim;
        if (a.vec) *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = v[e];
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(a.O) + out + dim;
    const bool bf = a.type == Q4_TYPE_BF16;
    const uint2 u = make_uint2(bf ? pack_bf16x2_rn(v[0], v[1]) : pack_f16x2_rn(v[0], v[1]), bf ? pack_bf16x2_rn(v[2], v[3]) : pack_f16x2_rn(v[2], v[3]));
    if (a.vec) {
        *reinterpret_cast<uint2 *>(o) = u;
    } else {
        o[0] = static_cast<uint16_t>(u.x), o[1] = static_cast<uint16_t>(u.x >> 16);
        o[2] = static_cast<uint16_t>(u.y), o[3] = static_cast<uint16_t>(u.y >> 16);
    }
}

// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over an item's parts i, the
// CTAs' that follow the one it starts in. Up to 32 parts (blocks of many rows): a
// warp takes a row, a lane a part's weight and then four dims of all parts in
// order. More parts (few rows of a long sequence): a CTA takes a row, W / 4 threads
// a part; the groups of threads take every n-th part, and their sums are added in
// order.
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const AttnArgs a)
{
    __shared__ float weight[kAttnMaxCtas + 1];
    __shared__ float4 sums[kJoinThreads];
    __shared__ float warp_red[kJoinThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int4 item = a.meta[2 * blockIdx.x];               // parts, rows, the first of them, head
    const int start = a.meta[2 * blockIdx.x + 1].x;
    const int parts = item.x;
    if (parts == 0) return;
    const int W = kChunk * a.c.chunks, lanes = W / 4, groups = kJoinThreads / lanes;
    const int tid = threadIdx.x, grp = tid / lanes, x = tid - grp * lanes;
    const int64_t size = attn_part_floats(a.block, a.c.chunks);
    const int rows = item.y;
    const auto part_at = [&](int i) { return a.parts + (2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0)) * size; };
    const auto out_at = [&](int r) {
        const int row = item.z + r, i = row / a.group, head = item.w * a.group + row - i * a.group;
        return (static_cast<int64_t>(start) + i) * a.ldo + static_cast<int64_t>(head) * a.c.d;
    };
    if (parts <= 32) {
        const int lane = tid % 32;
        for (int r = blockIdx.y * (kJoinThreads / 32) + tid / 32; r < rows; r += gridDim.y * (kJoinThreads / 32)) {
            float mi = neg_inf(), l = 0.0f;
            if (lane < parts) {
                const float *p = part_at(lane);
                mi = p[a.block * W + r], l = p[a.block * W + a.block + r];
            }
            // the first parts' sums are on their way while the weights are made
            constexpr int kAhead = 4;
            float4 u[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                u[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < parts && 4 * lane < W) u[i] = *reinterpret_cast<const float4 *>(part_at(i) + r * W + 4 * lane);
            }
            float m = mi;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float w = mi == neg_inf() ? 1.0f : exp2_fast(mi - m);   // (then its sums are zeros or NaN)
            l *= w;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int64_t out = out_at(r);
            for (int c = 0; c < W; c += 128) {
                const int dim = c + 4 * lane;
                float v[4] = {};
                for (int i0 = 0; i0 < parts; i0 += kAhead) {
                    if (i0 + c > 0) {
#pragma unroll
                        for (int i = 0; i < kAhead; ++i)
                            if (i0 + i < parts && dim < W) u[i] = *reinterpret_cast<const float4 *>(part_at(i0 + i) + r * W + dim);
                    }
#pragma unroll
                    for (int i = 0; i < kAhead; ++i) {
                        const float wi = __shfl_sync(0xFFFFFFFFu, w, min(i0 + i, 31));
                        if (i0 + i < parts) v[0] += wi * u[i].x, v[1] += wi * u[i].y, v[2] += wi * u[i].z, v[3] += wi * u[i].w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= inv;
                if (dim < W) store4(a, out, dim, v);
            }
        }
        return;
    }
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float m = neg_inf();
        for (int i = tid; i < parts; i += kJoinThreads) m = fmaxf(m, part_at(i)[a.block * W + r]);
#pragma unroll
        for (int o = 16; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        __syncthreads();
        if (tid % 32 == 0) warp_red[tid / 32] = m;
        __syncthreads();
        m = warp_red[0];
#pragma unroll
        for (int i = 1; i < kJoinThreads / 32; ++i) m = fmaxf(m, warp_red[i]);
        float l = 0.0f;
        for (int i = tid; i < parts; i += kJoinThreads) {
            const float *p = part_at(i);
            const float mi = p[a.block * W + r];
            const float w = mi == neg_inf() ? 1.0f : exp2_fast(mi - m);   // (then its sums are zeros or NaN)
            weight[i] = w;
            l += w * p[a.block * W + a.block + r];
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        __syncthreads();
        if (tid % 32 == 0) warp_red[tid / 32] = l;
        __syncthreads();
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < kJoinThreads / 32; ++i) l += warp_red[i];
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (grp < groups) {
#pragma unroll 4
            for (int i = grp; i < parts; i += groups) {
                const float4 v = *reinterpret_cast<const float4 *>(part_at(i) + r * W + 4 * x);
                const float w = weight[i];
                s.x += w * v.x, s.y += w * v.y, s.z += w * v.z, s.w += w * v.w;
            }
            sums[tid] = s;
        }
        __syncthreads();
        if (grp == 0) {
            for (int i = 1; i < groups; ++i) {
                const float4 v = sums[i * lanes + x];
                s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const float v[4] = {s.x * inv, s.y * inv, s.z * inv, s.w * inv};
            store4(a, out_at(r), 4 * x, v);
        }
    }
}

} // namespace

cudaError_t launch_attn_join(const AttnArgs &args, int ctas, cudaStream_t s)
{
    AttnArgs a = args;
    void *p[] = {&a};
    const unsigned rows = static_cast<unsigned>(a.block <= 64 ? a.block / 4 : 16);
    return launch_pdl(reinterpret_cast<const void *>(&attn_join_kernel), dim3(static_cast<unsigned>(ctas), rows), dim3(kJoinThreads), 0, s, p);
}

cudaError_t launch_attn_warp(AttnArgs a, int sm_count, cudaStream_t s)
{
    a.tile = kWarpTile;
    a.item_cost = 2;
    int ctas = 0;
    const bool wide = a.type == Q4_TYPE_F32;
    cudaError_t e;
    switch (a.c.type) {
    case Q4_TYPE_F16: e = wide ? launch_attn_f16x2(a, sm_count, s, &ctas) : launch_attn_f16(a, sm_count, s, &ctas); break;
    case Q4_TYPE_BF16: e = launch_attn_bf16(a, sm_count, s, &ctas); break;
    default: e = wide ? launch_attn_i8x2(a, sm_count, s, &ctas) : launch_attn_i8(a, sm_count, s, &ctas); break;
    }
    return e != cudaSuccess ? e : launch_attn_join(a, ctas, s);
}

} // namespace q4
