// q4mm_moe.cu -- tokens sorted by expert and back. A pair p = t * top_k + j is
// token t's j-th choice; the expert-grouped product wants the rows of an
// expert next to one another.
//
//   dispatch: a stable counting sort of the pairs by expert. With count[e] the
//     pairs of expert e, offsets[e] = sum of count[e'] over e' < e, the row of
//     a pair is offsets[e] + (pairs of e before it), and Xs[row] = X[t]. A pair
//     without an expert (an id outside 0 .. E - 1) sorts after the last expert
//     as if it had one of its own; its row is zeros, and row_of holds -1 - row.
//   combine: Y[t] = base[t] + sum over j of weight[t][j] * Ys[row_of[t][j]],
//     in fp32 and in the order of j, rounded once; pairs without an expert
//     are left out, whatever their rows and weights hold. With weights of 1 it
//     is the gradient of dispatch's copy.
//   combine's gradient: dYs[row] = weight * dY[t] and dweight[t][j] =
//     <dY[t], Ys[row]>; zeros for pairs without an expert.
//
// The copies are bound by the memory traffic: dispatch reads each token once
// and writes its top_k rows; combine gathers rows, all top_k of a token's
// column in flight at once. The sort is bound by latency. Ranks come from
// warp matches over consecutive pairs, so no atomic's order enters a result.
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_moe.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
// Up to so many pairs each CTA sorts them all for itself and copies its share
// of the rows in the same launch.
constexpr int64_t kOneLaunchPairs = 1024;
constexpr int kOneLaunchExperts = 512;

// The expert of pair p, `experts` for a pair without one.
__device__ __forceinline__ int key_of(const MoeDispatchArgs &a, int64_t p)
{
    const int64_t id = a.id_bytes == 8 ? static_cast<const int64_t *>(a.ids)[p] : static_cast<const int32_t *>(a.ids)[p];
    return id >= 0 && id < a.experts ? static_cast<int>(id) : a.experts;
}

// Ranks a run of pairs [p0, p1) of a warp: calls put(p, key, rank) with the
// pairs of the same key before p in the run added to cnt[key], which ends as
// the run's total. All 32 lanes take part.
template <typename Put>
__device__ __forceinline__ void rank_run(const MoeDispatchArgs &a, int64_t p0, int64_t p1, int32_t *cnt, Put put)
{
    const int lane = threadIdx.x & 31;
    for (int64_t b = p0; b < p1; b += 32) {
        const int64_t p = b + lane;
        const int key = p < p1 ? key_of(a, p) : -1;
        const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
        const int before = __popc(same & ((1u << lane) - 1u));
        int base = 0;
        if (key >= 0) base = cnt[key];
        __syncwarp();
        if (key >= 0) {
            if (before == 0) cnt[key] = base + __popc(same);
            put(p, key, base + before);
        }
        __syncwarp();
    }
}

// An exclusive sum over v[0 .. n - 1] in shared memory by the whole CTA;
// `tmp` holds a word per warp.
__device__ __forceinline__ void exclusive_scan(int32_t *v, int n, int32_t *tmp)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
    int32_t carry = 0;
    for (int b = 0; b < n; b += threads) {
        const int i = b + tid;
        const int32_t x = i < n ? v[i] : 0;
        int32_t s = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
            if (lane >= o) s += y;
        }
        if (lane == 31) tmp[warp] = s;
        __syncthreads();
        int32_t pre = carry, all = 0;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) pre += tmp[w];
            all += tmp[w];
        }
        if (i < n) v[i] = pre + s - x;
        carry += all;
        __syncthreads();
    }
}

// Pairs of warp w of a CTA that holds [p0, p1), a multiple of 32 but the last.
__device__ __forceinline__ void warp_run(int64_t p0, int64_t p1, int w, int64_t *b, int64_t *e)
{
    const int64_t per = ((p1 - p0 + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    *b = min(p1, p0 + w * per);
    *e = min(p1, *b + per);
}

// Copies token t's row to the rows of its pairs. Row r of a pair: `row_of`'s
// value, negative for zeros. U: one access; threads `t0` of `threads`.
template <typename U>
__device__ __forceinline__ void copy_row(const MoeDispatchArgs &a, int64_t t, const int32_t *rows, int t0, int threads)
{
    const U *x = static_cast<const U *>(a.X) + t * a.ldx;
    U *xs = static_cast<U *>(a.Xs);
    for (int64_t c = t0; c < a.row_units; c += threads) {
        const U v = x[c];
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = rows[j];
            xs[static_cast<int64_t>(r < 0 ? -1 - r : r) * a.ldxs + c] = r < 0 ? U{} : v;
        }
    }
    // the elements past the last whole access
    for (int i = t0; i < a.tail; i += threads) {
        const int64_t c = a.tail_at + i;
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = rows[j];
            U *out = xs + static_cast<int64_t>(r < 0 ? -1 - r : r) * a.ldxs;
            if (a.esize == 4)
                reinterpret_cast<uint32_t *>(out)[c] = r < 0 ? 0u : reinterpret_cast<const uint32_t *>(x)[c];
            else
                reinterpret_cast<uint16_t *>(out)[c] =
                    r < 0 ? static_cast<uint16_t>(0) : reinterpret_cast<const uint16_t *>(x)[c];
        }
    }
}

// One launch for few pairs: every CTA sorts them all in shared memory; CTA 0
// writes the sort's results; the rows are dealt to the CTAs.
template <typename U> __global__ void __launch_bounds__(kSortThreads) dispatch_small_kernel(const MoeDispatchArgs a, int segs)
{
    extern __shared__ int32_t sm[];
    const int E1 = a.experts + 1, tid = threadIdx.x, warp = tid >> 5;
    int32_t *cnt = sm;                       // [kSortWarps][E1]
    int32_t *total = cnt + kSortWarps * E1;  // [E1]
    int32_t *tmp = total + E1;               // [kSortWarps]
    int32_t *rows = tmp + kSortWarps;        // [pairs]
    for (int i = tid; i < kSortWarps * E1; i += kSortThreads) cnt[i] = 0;
    pdl_wait();
    __syncthreads();
    int64_t b, e;
    warp_run(0, a.pairs, warp, &b, &e);
    rank_run(a, b, e, cnt + warp * E1, [&](int64_t p, int, int rank) { rows[p] = rank; });
    __syncthreads();
    for (int k = tid; k < E1; k += kSortThreads) {
        int32_t s = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = cnt[w * E1 + k];
            cnt[w * E1 + k] = s;
            s += c;
        }
        total[k] = s;
    }
    __syncthreads();
    exclusive_scan(total, E1, tmp);
    for (int64_t p = b + (tid & 31); p < e; p += 32) {
        const int key = key_of(a, p);
        const int32_t row = total[key] + cnt[warp * E1 + key] + rows[p];
        rows[p] = key == a.experts ? -1 - row : row;
        if (blockIdx.x == 0) {
            a.row_of[p] = rows[p];
            if (a.pair_of) a.pair_of[row] = static_cast<int32_t>(p);
        }
    }
    if (blockIdx.x == 0)
        for (int k = tid; k < E1; k += kSortThreads) a.offsets[k] = total[k];
    if (!a.Xs) return;
    __syncthreads();
    for (int64_t it = blockIdx.x; it < a.tokens * segs; it += gridDim.x) {
        const int64_t t = it / segs;
        copy_row<U>(a, t, rows + t * a.top_k, static_cast<int>(it % segs) * kSortThreads + tid, segs * kSortThreads);
    }
}

// The chunk's pairs of each expert.
__global__ void __launch_bounds__(kSortThreads) histogram_kernel(const MoeDispatchArgs a)
{
    extern __shared__ int32_t sm[];
    const int E1 = a.experts + 1;
    for (int i = threadIdx.x; i < E1; i += kSortThreads) sm[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int64_t p0 = blockIdx.x * a.chunk, p1 = min(a.pairs, p0 + a.chunk);
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kSortThreads) atomicAdd(&sm[key_of(a, p)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < E1; i += kSortThreads) a.hist[static_cast<int64_t>(blockIdx.x) * E1 + i] = sm[i];
}

// The rows of a chunk's pairs, from every chunk's histogram.
__global__ void __launch_bounds__(kSortThreads) rank_kernel(const MoeDispatchArgs a)
{
    extern __shared__ int32_t sm[];
    const int E1 = a.experts + 1, tid = threadIdx.x, warp = tid >> 5;
    int32_t *cnt = sm;                       // [kSortWarps][E1]
    int32_t *total = cnt + kSortWarps * E1;  // [E1]
    int32_t *tmp = total + E1;               // [kSortWarps]
    for (int i = tid; i < kSortWarps * E1; i += kSortThreads) cnt[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int64_t p0 = blockIdx.x * a.chunk, p1 = min(a.pairs, p0 + a.chunk);
    int64_t b, e;
    warp_run(p0, p1, warp, &b, &e);
    rank_run(a, b, e, cnt + warp * E1, [](int64_t, int, int) {});
    __syncthreads();
    for (int k = tid; k < E1; k += kSortThreads) {
        int32_t before = 0, all = 0;
        for (int c = 0; c < a.chunks; ++c) {
            const int32_t h = a.hist[static_cast<int64_t>(c) * E1 + k];
            if (c < static_cast<int>(blockIdx.x)) before += h;
            all += h;
        }
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t c = cnt[w * E1 + k];
            cnt[w * E1 + k] = before;
            before += c;
        }
        total[k] = all;
    }
    __syncthreads();
    exclusive_scan(total, E1, tmp);
    if (blockIdx.x == 0)
        for (int k = tid; k < E1; k += kSortThreads) a.offsets[k] = total[k];
    rank_run(a, b, e, cnt + warp * E1, [&](int64_t p, int key, int rank) {
        const int32_t row = total[key] + rank;
        a.row_of[p] = key == a.experts ? -1 - row : row;
        if (a.pair_of) a.pair_of[row] = static_cast<int32_t>(p);
    });
}

template <typename U> __global__ void __launch_bounds__(256) copy_rows_kernel(const MoeDispatchArgs a)
{
    pdl_wait();
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x)
        copy_row<U>(a, t, a.row_of + t * a.top_k, threadIdx.x, blockDim.x);
}

// ----------------------------------------------------------------- combine --

template <typename T, int V> __global__ void __launch_bounds__(256) combine_kernel(const MoeCombineArgs a)
{
    pdl_wait();
    const T *Ys = static_cast<const T *>(a.Ys);
    for (int64_t it = blockIdx.x; it < a.tokens * a.segs; it += gridDim.x) {
        const int64_t t = it / a.segs;
        const int seg = static_cast<int>(it % a.segs);
        const int32_t *rows = a.row_of + t * a.top_k;
        const float *w = a.weights ? a.weights + t * a.top_k : nullptr;
        for (int64_t c = (static_cast<int64_t>(seg) * blockDim.x + threadIdx.x) * V; c < a.d;
             c += static_cast<int64_t>(a.segs) * blockDim.x * V) {
            float y[V];
            if (a.base) {
                const Pack<T, V> bv = load_pack<T, V>(static_cast<const T *>(a.base) + t * a.ldbase, c, a.d);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = elem(bv, i);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = 0.0f;
            }
            for (int j0 = 0; j0 < a.top_k; j0 += 4) {
                Pack<T, V> v[4];
                bool has[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int32_t r = j0 + j < a.top_k ? rows[j0 + j] : -1;
                    has[j] = r >= 0 && r < a.pairs;
                    if (has[j]) v[j] = load_pack<T, V>(Ys + static_cast<int64_t>(r) * a.ldys, c, a.d);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (!has[j]) continue;
                    const float wj = w ? w[j0 + j] : 1.0f;
#pragma unroll
                    for (int i = 0; i < V; ++i) y[i] = fmaf(wj, elem(v[j], i), y[i]);
                }
            }
            store_pack<T, V>(static_cast<T *>(a.Y) + t * a.ldy, c, a.d, pack_of<T, V>(y));
        }
    }
}

// A warp per pair: the token's gradient row is read by top_k neighbouring
// warps at about the same time, from memory once.
template <typename T, int V> __global__ void __launch_bounds__(256) combine_bwd_kernel(const MoeCombineBwdArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t p = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5); p < a.pairs; p += warps) {
        const int64_t t = p / a.top_k;
        const int32_t r = a.row_of[p];
        const bool has = r >= 0;
        const int64_t row = has ? r : -1 - static_cast<int64_t>(r);
        if (row >= a.pairs) continue;
        const float w = !has ? 0.0f : a.weights ? a.weights[p] : 1.0f;
        const T *dy = static_cast<const T *>(a.dY) + t * a.lddy;
        const T *ys = static_cast<const T *>(a.Ys) + row * a.ldys;
        T *out = static_cast<T *>(a.dYs) + row * a.lddys;
        float s = 0.0f;
#pragma unroll 4
        for (int64_t c = lane * V; c < a.d; c += 32 * V) {
            Pack<T, V> o = zero_pack<T, V>();
            if (has) {
                const Pack<T, V> gp = load_pack<T, V>(dy, c, a.d), yp = load_pack<T, V>(ys, c, a.d);
                float f[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float gi = elem(gp, i);
                    s = fmaf(gi, elem(yp, i), s);
                    f[i] = w * gi;
                }
                o = pack_of<T, V>(f);
            }
            store_pack<T, V>(out, c, a.d, o);
        }
        if (!a.dweights) continue;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) a.dweights[p] = s;
    }
}

bool one_launch(int64_t pairs, int64_t experts) { return pairs <= kOneLaunchPairs && experts <= kOneLaunchExperts; }

// At least 2048 pairs a chunk (eight warps of 256), at most kMoeMaxChunks.
void moe_chunks(int64_t pairs, int64_t *chunk, int *chunks)
{
    *chunk = std::max<int64_t>(2048, round_up(ceil_div(pairs, kMoeMaxChunks), 32));
    *chunks = static_cast<int>(ceil_div(pairs, *chunk));
}

template <typename U> cudaError_t launch_dispatch(MoeDispatchArgs a, int sm_count, cudaStream_t s)
{
    const int E1 = a.experts + 1;
    const size_t count_smem = sizeof(int32_t) * (static_cast<size_t>(kSortWarps + 1) * E1 + kSortWarps);
    if (one_launch(a.pairs, a.experts)) {
        const int segs = a.Xs ? static_cast<int>(std::max<int64_t>(1, ceil_div(a.row_units, kSortThreads))) : 1;
        const int64_t grid = a.Xs ? std::min<int64_t>(a.tokens * segs, 2 * static_cast<int64_t>(sm_count)) : 1;
        int sg = segs;
        void *args[] = {&a, &sg};
        return launch_pdl(reinterpret_cast<const void *>(&dispatch_small_kernel<U>), dim3(static_cast<unsigned>(grid)),
                          dim3(kSortThreads), count_smem + sizeof(int32_t) * a.pairs, s, args);
    }
    void *args[] = {&a};
    cudaError_t e = launch_pdl(reinterpret_cast<const void *>(&histogram_kernel), dim3(static_cast<unsigned>(a.chunks)),
                               dim3(kSortThreads), sizeof(int32_t) * E1, s, args);
    if (e != cudaSuccess) return e;
    const void *rank = reinterpret_cast<const void *>(&rank_kernel);
    if (count_smem > 48 * 1024) {
        e = set_max_smem(rank, count_smem);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(rank, dim3(static_cast<unsigned>(a.chunks)), dim3(kSortThreads), count_smem, s, args);
    if (e != cudaSuccess || !a.Xs) return e;
    const int64_t grid = std::min<int64_t>(a.tokens, 8 * static_cast<int64_t>(sm_count));
    return launch_pdl(reinterpret_cast<const void *>(&copy_rows_kernel<U>), dim3(static_cast<unsigned>(grid)), dim3(256),
                      0, s, args);
}

template <typename T> cudaError_t launch_combine(MoeCombineArgs a, int vec, int sm_count, cudaStream_t s)
{
    const void *fn = vec * sizeof(T) == 16 ? reinterpret_cast<const void *>(&combine_kernel<T, 16 / sizeof(T)>)
                     : vec == 2            ? reinterpret_cast<const void *>(&combine_kernel<T, 2>)
                                           : reinterpret_cast<const void *>(&combine_kernel<T, 1>);
    const int64_t vecs = ceil_div(a.d, vec);
    const int threads = static_cast<int>(std::min<int64_t>(256, round_up(vecs, 32)));
    a.segs = static_cast<int>(std::min<int64_t>(ceil_div(vecs, threads), 1024));
    const int64_t grid = std::min<int64_t>(a.tokens * a.segs, 8 * static_cast<int64_t>(sm_count));
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, s, args);
}

template <typename T> cudaError_t launch_combine_bwd(MoeCombineBwdArgs a, int vec, int sm_count, cudaStream_t s)
{
    const void *fn = vec * sizeof(T) == 16 ? reinterpret_cast<const void *>(&combine_bwd_kernel<T, 16 / sizeof(T)>)
                     : vec == 2            ? reinterpret_cast<const void *>(&combine_bwd_kernel<T, 2>)
                                           : reinterpret_cast<const void *>(&combine_bwd_kernel<T, 1>);
    const int64_t grid = std::min<int64_t>(ceil_div(a.pairs, 8), 8 * static_cast<int64_t>(sm_count));
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, args);
}

} // namespace

size_t moe_scratch(int64_t pairs, int64_t experts)
{
    if (one_launch(pairs, experts)) return 0;
    int64_t chunk;
    int chunks;
    moe_chunks(pairs, &chunk, &chunks);
    return sizeof(int32_t) * static_cast<size_t>(chunks) * static_cast<size_t>(experts + 1);
}

cudaError_t launch_moe_dispatch(MoeDispatchArgs a, int unit, int sm_count, cudaStream_t s)
{
    moe_chunks(a.pairs, &a.chunk, &a.chunks);
    switch (unit) {
    case 16: return launch_dispatch<uint4>(a, sm_count, s);
    case 4: return launch_dispatch<uint32_t>(a, sm_count, s);
    default: return launch_dispatch<uint16_t>(a, sm_count, s);
    }
}

cudaError_t launch_moe_combine(MoeCombineArgs a, int type, int vec, int sm_count, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_combine<float>(a, vec, sm_count, s);
    case Q4_TYPE_F16: return launch_combine<__half>(a, vec, sm_count, s);
    default: return launch_combine<__nv_bfloat16>(a, vec, sm_count, s);
    }
}

cudaError_t launch_moe_combine_bwd(const MoeCombineBwdArgs &a, int type, int vec, int sm_count, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_combine_bwd<float>(a, vec, sm_count, s);
    case Q4_TYPE_F16: return launch_combine_bwd<__half>(a, vec, sm_count, s);
    default: return launch_combine_bwd<__nv_bfloat16>(a, vec, sm_count, s);
    }
}

} // namespace q4
