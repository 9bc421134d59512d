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
//
// GB300, us a call (floor at the measured copy rate): dispatch 1 x 8 of 128
// experts, 2560 fp32, 3.3 (one launch); 8192 x 8 of 128, 4096 bf16, 102 (89), the
// sort 12 of it; combine 4099 x 4 of 32, 2560 fp32 with a base, 41 (37); its
// gradient 4096 x 8 of 128, 4096 bf16, 85 (84).
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
// the run's total. All 32 lanes take part. Four steps' keys are loaded at once.
template <typename Put>
__device__ __forceinline__ void rank_run(const MoeDispatchArgs &a, int64_t p0, int64_t p1, int32_t *cnt, Put put)
{
    const int lane = threadIdx.x & 31;
    for (int64_t b = p0; b < p1; b += 128) {
        int keys[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) keys[i] = b + 32 * i + lane < p1 ? key_of(a, b + 32 * i + lane) : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (b + 32 * i >= p1) break;
            const int key = keys[i];
            const unsigned same = __match_any_sync(0xFFFFFFFFu, key);
            const int before = __popc(same & ((1u << lane) - 1u));
            int base = 0;
            if (key >= 0) base = cnt[key];
            __syncwarp();
            if (key >= 0) {
                if (before == 0) cnt[key] = base + __popc(same);
                put(b + 32 * i + lane, key, base + before);
            }
            __syncwarp();
        }
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
    const int warps = static_cast<int>(blockDim.x) >> 5;
    const int64_t per = ((p1 - p0 + warps - 1) / warps + 31) / 32 * 32;
    *b = min(p1, p0 + w * per);
    *e = min(p1, *b + per);
}

// Rows of `bytes` bytes on 2-byte boundaries are copied 16 bytes a store,
// wherever they start: `threads` threads, this one `t0`. A store covers an
// aligned 16-byte word of the destination; its bytes come from one or two aligned
// words of the source, each of which holds at least one of them, shifted by what
// the two rows' starts differ. The bytes before the destination's first whole
// word and after its last go two by two.
__device__ __forceinline__ void copy_bytes(uint8_t *dst, const uint8_t *src, int64_t bytes, bool zero, int t0, int threads)
{
    const int64_t head = min(bytes, static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(dst) & 15)) & 15));
    const int64_t words = (bytes - head) / 16, tail = head + 16 * words;
    const uint8_t *from = src + head;
    const int by = static_cast<int>(reinterpret_cast<uintptr_t>(from) & 15);
    const uint4 *in = reinterpret_cast<const uint4 *>(from - by);
    uint4 *out = reinterpret_cast<uint4 *>(dst + head);
    if (zero) {
        for (int64_t i = t0; i < words; i += threads) out[i] = make_uint4(0u, 0u, 0u, 0u);
    } else if (by == 0) {
        for (int64_t i = t0; i < words; i += threads) out[i] = in[i];
    } else {
        for (int64_t i = t0; i < words; i += threads) out[i] = shifted(in[i], in[i + 1], by);
    }
    const int loose = static_cast<int>((head + bytes - tail) / 2), first = static_cast<int>(head / 2);
    for (int i = t0; i < loose; i += threads) {
        const int64_t at = i < first ? 2 * i : tail + 2 * (i - first);
        *reinterpret_cast<uint16_t *>(dst + at) = zero ? static_cast<uint16_t>(0) : *reinterpret_cast<const uint16_t *>(src + at);
    }
}

// Copies token t's row to the rows of its pairs (a negative `rows` entry: zeros
// to row -1 - it). Threads t0 of `threads`. WHOLE: rows start on 16-byte
// boundaries and are whole 16-byte words, so each is read once for all its pairs.
template <bool WHOLE>
__device__ __forceinline__ void copy_row(const MoeDispatchArgs &a, int64_t t, const int32_t *rows, int t0, int threads)
{
    const uint8_t *x = static_cast<const uint8_t *>(a.X) + t * a.ldx;
    uint8_t *xs = static_cast<uint8_t *>(a.Xs);
    if constexpr (WHOLE) {
        const int64_t words = a.bytes / 16;
        for (int64_t c = t0; c < words; c += threads) {
            const uint4 v = reinterpret_cast<const uint4 *>(x)[c];
            for (int j = 0; j < a.top_k; ++j) {
                const int32_t r = rows[j];
                reinterpret_cast<uint4 *>(xs + static_cast<int64_t>(r < 0 ? -1 - r : r) * a.ldxs)[c] = r < 0 ? make_uint4(0u, 0u, 0u, 0u) : v;
            }
        }
    } else {
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = rows[j];
            copy_bytes(xs + static_cast<int64_t>(r < 0 ? -1 - r : r) * a.ldxs, x, a.bytes, r < 0, t0, threads);
        }
    }
}

// One launch for few pairs: every CTA sorts them all in shared memory; CTA 0
// writes the sort's results; the rows are dealt to the CTAs.
template <bool WHOLE> __global__ void __launch_bounds__(kSortThreads) dispatch_small_kernel(const MoeDispatchArgs a, int segs)
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
        copy_row<WHOLE>(a, t, rows + t * a.top_k, static_cast<int>(it % segs) * kSortThreads + tid, segs * kSortThreads);
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
    // an expert's chunks next to each other: the ranks read them as vectors
    for (int i = threadIdx.x; i < E1; i += kSortThreads) a.hist[static_cast<int64_t>(i) * a.pitch + blockIdx.x] = sm[i];
}

// The rows of a chunk's pairs, from every chunk's histogram.
__global__ void __launch_bounds__(1024) rank_kernel(const MoeDispatchArgs a)
{
    extern __shared__ int32_t sm[];
    const int E1 = a.experts + 1, tid = threadIdx.x, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    int32_t *cnt = sm;                  // [warps][E1]
    int32_t *total = cnt + warps * E1;  // [E1]
    int32_t *tmp = total + E1;          // [warps]
    for (int i = tid; i < warps * E1; i += threads) cnt[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int64_t p0 = blockIdx.x * a.chunk, p1 = min(a.pairs, p0 + a.chunk);
    int64_t b, e;
    warp_run(p0, p1, warp, &b, &e);
    rank_run(a, b, e, cnt + warp * E1, [](int64_t, int, int) {});
    __syncthreads();
    const int me = static_cast<int>(blockIdx.x);
    for (int k = tid; k < E1; k += threads) {
        int32_t before = 0, all = 0;
        if (a.chunks == 1)
            for (int w = 0; w < warps; ++w) all += cnt[w * E1 + k];
        const int4 *h = reinterpret_cast<const int4 *>(a.hist + static_cast<int64_t>(k) * a.pitch);
        for (int c = 0; a.chunks > 1 && c < a.chunks; c += 32) {   // eight vectors in flight
            int4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = c + 4 * i < a.chunks ? h[c / 4 + i] : make_int4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int32_t n[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int32_t x = c + 4 * i + u < a.chunks ? n[u] : 0;   // the pitch's padding is not written
                    if (c + 4 * i + u < me) before += x;
                    all += x;
                }
            }
        }
        for (int w = 0; w < warps; ++w) {
            const int32_t c = cnt[w * E1 + k];
            cnt[w * E1 + k] = before;
            before += c;
        }
        total[k] = all;
    }
    __syncthreads();
    exclusive_scan(total, E1, tmp);
    if (me == 0)
        for (int k = tid; k < E1; k += threads) a.offsets[k] = total[k];
    rank_run(a, b, e, cnt + warp * E1, [&](int64_t p, int key, int rank) {
        const int32_t row = total[key] + rank;
        a.row_of[p] = key == a.experts ? -1 - row : row;
        if (a.pair_of) a.pair_of[row] = static_cast<int32_t>(p);
    });
}

// A token per CTA. (A warp per pair took 48 us instead of 31 for 16384 x 8 rows
// of 1022 bytes: the token's row is read again for each.)
template <bool WHOLE> __global__ void __launch_bounds__(256) copy_rows_kernel(const MoeDispatchArgs a)
{
    pdl_wait();
    const int64_t t = blockIdx.x;
    copy_row<WHOLE>(a, t, a.row_of + t * a.top_k, threadIdx.x, blockDim.x);
}

// ----------------------------------------------------------------- combine --

// A warp takes 32 U vectors of a token. Its lanes read the token's rows and
// weights first, J at a time, then all J U vectors are in flight at once.
template <typename T, int V, int U, int J> __global__ void __launch_bounds__(256) combine_kernel(const MoeCombineArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = it / a.segs;
    if (t >= a.tokens) return;
    const T *Ys = static_cast<const T *>(a.Ys);
    const int32_t *rows = a.row_of + t * a.top_k;
    const float *w = a.weights ? a.weights + t * a.top_k : nullptr;
    const int64_t c0 = ((it - t * a.segs) * (32 * U) + lane) * V;
    float y[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * 32 * V;
        const Pack<T, V> b = a.base && c < a.d ? load_pack<T, V>(static_cast<const T *>(a.base) + t * a.ldbase, c, a.d) : zero_pack<T, V>();
#pragma unroll
        for (int i = 0; i < V; ++i) y[u][i] = elem(b, i);
    }
    for (int j0 = 0; j0 < a.top_k; j0 += 32) {
        const int32_t mine = j0 + lane < a.top_k ? rows[j0 + lane] : -1;
        const float my_w = j0 + lane < a.top_k && w ? w[j0 + lane] : 1.0f;
        const int n = min(32, a.top_k - j0);
        for (int j1 = 0; j1 < n; j1 += J) {
            Pack<T, V> v[J][U];
            bool has[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int32_t r = __shfl_sync(0xFFFFFFFFu, mine, (j1 + j) & 31);
                has[j] = j1 + j < n && r >= 0 && r < a.pairs;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t c = c0 + u * 32 * V;
                    if (has[j] && c < a.d) v[j][u] = load_pack<T, V>(Ys + static_cast<int64_t>(r) * a.ldys, c, a.d);
                    else v[j][u] = zero_pack<T, V>();
                }
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float wj = __shfl_sync(0xFFFFFFFFu, my_w, (j1 + j) & 31);
                if (!has[j]) continue;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < V; ++i) y[u][i] = fmaf(wj, elem(v[j][u], i), y[u][i]);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t c = c0 + u * 32 * V;
        if (c < a.d) store_pack<T, V>(static_cast<T *>(a.Y) + t * a.ldy, c, a.d, pack_of<T, V>(y[u]));
    }
}

// A warp per pair: the token's gradient row is read by top_k neighbouring warps
// at about the same time, from memory once. U vectors of both rows are in flight.
template <typename T, int V, int U> __global__ void __launch_bounds__(256) combine_bwd_kernel(const MoeCombineBwdArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (p >= a.pairs) return;
    const int64_t t = p / a.top_k;
    const int32_t r = a.row_of[p];
    const bool has = r >= 0;
    const int64_t row = has ? r : -1 - static_cast<int64_t>(r);
    if (row >= a.pairs) return;
    const float w = !has ? 0.0f : a.weights ? a.weights[p] : 1.0f;
    const T *dy = static_cast<const T *>(a.dY) + t * a.lddy;
    const T *ys = static_cast<const T *>(a.Ys) + row * a.ldys;
    T *out = static_cast<T *>(a.dYs) + row * a.lddys;
    const int d = static_cast<int>(a.d);
    float s = 0.0f;
    for (int c0 = lane * V; c0 < d; c0 += 32 * U * V) {
        Pack<T, V> g[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * V;
            g[u] = has && c < d ? load_pack<T, V>(dy, c, d) : zero_pack<T, V>();
            y[u] = has && c < d ? load_pack<T, V>(ys, c, d) : zero_pack<T, V>();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * 32 * V;
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float gi = elem(g[u], i);
                s = fmaf(gi, elem(y[u], i), s);
                f[i] = has ? w * gi : 0.0f;
            }
            if (c < d) store_pack<T, V>(out, c, d, pack_of<T, V>(f));
        }
    }
    if (!a.dweights) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) a.dweights[p] = s;
}

// 16-bit rows that start anywhere: the vectors are the aligned 16-byte words of
// the row that is written, the rows that are read are shifted to it, and the
// elements before its first whole word and after its last go one by one (with
// 2-byte accesses all over, 8000 x 2 x 1023 took 40 us; the accesses, not the
// memory, bounded it).
struct Words {
    int first, count, loose, after;   // element of the first whole word, words, elements outside, the one after the words
};
template <typename T> __device__ __forceinline__ Words words_of(const T *row, int d)
{
    Words w;
    w.first = min(d, static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 2));
    w.count = (d - w.first) / 8;
    w.after = w.first + 8 * w.count;
    w.loose = w.first + d - w.after;
    return w;
}

template <typename T> __global__ void __launch_bounds__(256) combine_anywhere_kernel(const MoeCombineArgs a)
{
    constexpr int J = 4;
    pdl_wait();
    const int lane = threadIdx.x & 31, d = static_cast<int>(a.d);
    const int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t t = it / a.segs;
    if (t >= a.tokens) return;
    const int seg = static_cast<int>(it - t * a.segs);
    const T *Ys = static_cast<const T *>(a.Ys), *base = a.base ? static_cast<const T *>(a.base) + t * a.ldbase : nullptr;
    T *out = static_cast<T *>(a.Y) + t * a.ldy;
    const int32_t *rows = a.row_of + t * a.top_k;
    const float *w = a.weights ? a.weights + t * a.top_k : nullptr;
    const Words wd = words_of(out, d);
    for (int i = seg * 32 + lane; i < wd.count; i += a.segs * 32) {
        const int c = wd.first + 8 * i;
        float y[8] = {};
        if (base) {
            const Pack<T, 8> b = load_anywhere(base, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = elem(b, e);
        }
        for (int j0 = 0; j0 < a.top_k; j0 += J) {
            Pack<T, 8> v[J];
            bool has[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int32_t r = j0 + j < a.top_k ? rows[j0 + j] : -1;
                has[j] = r >= 0 && r < a.pairs;
                v[j] = has[j] ? load_anywhere(Ys + static_cast<int64_t>(r) * a.ldys, c) : zero_pack<T, 8>();
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!has[j]) continue;
                const float wj = w ? w[j0 + j] : 1.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(wj, elem(v[j], e), y[e]);
            }
        }
        store_pack<T, 8>(out, c, d, pack_of<T, 8>(y));
    }
    for (int i = seg * 32 + lane; i < wd.loose; i += a.segs * 32) {
        const int c = i < wd.first ? i : wd.after + i - wd.first;
        float y = base ? elem(load_pack<T, 1>(base, c, d), 0) : 0.0f;
        for (int j = 0; j < a.top_k; ++j) {
            const int32_t r = rows[j];
            if (r >= 0 && r < a.pairs) y = fmaf(w ? w[j] : 1.0f, elem(load_pack<T, 1>(Ys + static_cast<int64_t>(r) * a.ldys, c, d), 0), y);
        }
        const float one[1] = {y};
        store_pack<T, 1>(out, c, d, pack_of<T, 1>(one));
    }
}

template <typename T> __global__ void __launch_bounds__(256) combine_bwd_anywhere_kernel(const MoeCombineBwdArgs a)
{
    constexpr int U = 2;
    pdl_wait();
    const int lane = threadIdx.x & 31, d = static_cast<int>(a.d);
    const int64_t p = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (p >= a.pairs) return;
    const int64_t t = p / a.top_k;
    const int32_t r = a.row_of[p];
    const bool has = r >= 0;
    const int64_t row = has ? r : -1 - static_cast<int64_t>(r);
    if (row >= a.pairs) return;
    const float w = !has ? 0.0f : a.weights ? a.weights[p] : 1.0f;
    const T *dy = static_cast<const T *>(a.dY) + t * a.lddy, *ys = static_cast<const T *>(a.Ys) + row * a.ldys;
    T *out = static_cast<T *>(a.dYs) + row * a.lddys;
    const Words wd = words_of(out, d);
    float s = 0.0f;
    for (int i0 = lane; i0 < wd.count; i0 += 32 * U) {
        Pack<T, 8> g[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = has && i0 + 32 * u < wd.count;
            g[u] = in ? load_anywhere(dy, wd.first + 8 * (i0 + 32 * u)) : zero_pack<T, 8>();
            y[u] = in ? load_anywhere(ys, wd.first + 8 * (i0 + 32 * u)) : zero_pack<T, 8>();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float ge = elem(g[u], e);
                s = fmaf(ge, elem(y[u], e), s);
                f[e] = has ? w * ge : 0.0f;
            }
            if (i0 + 32 * u < wd.count) store_pack<T, 8>(out, wd.first + 8 * (i0 + 32 * u), d, pack_of<T, 8>(f));
        }
    }
    for (int i = lane; i < wd.loose; i += 32) {
        const int c = i < wd.first ? i : wd.after + i - wd.first;
        float f[1] = {0.0f};
        if (has) {
            const float ge = elem(load_pack<T, 1>(dy, c, d), 0);
            s = fmaf(ge, elem(load_pack<T, 1>(ys, c, d), 0), s);
            f[0] = w * ge;
        }
        store_pack<T, 1>(out, c, d, pack_of<T, 1>(f));
    }
    if (!a.dweights) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) a.dweights[p] = s;
}

bool one_launch(int64_t pairs, int64_t experts) { return pairs <= kOneLaunchPairs && experts <= kOneLaunchExperts; }

// Up to 8192 pairs one CTA, which needs no histogram of others; then at least
// 2048 pairs a chunk, at most kMoeMaxChunks chunks.
void moe_chunks(int64_t pairs, int64_t *chunk, int *chunks)
{
    *chunk = pairs <= 8192 ? pairs : std::max<int64_t>(2048, round_up(ceil_div(pairs, kMoeMaxChunks), 32));
    *chunks = static_cast<int>(ceil_div(pairs, *chunk));
}

template <bool WHOLE> cudaError_t launch_dispatch(MoeDispatchArgs a, int sm_count, cudaStream_t s)
{
    const int E1 = a.experts + 1;
    const size_t count_smem = sizeof(int32_t) * (static_cast<size_t>(kSortWarps + 1) * E1 + kSortWarps);
    // one 16-byte word a thread, at most 256 threads
    const int64_t words = std::max<int64_t>(1, ceil_div(a.bytes, 16));
    if (one_launch(a.pairs, a.experts)) {
        int segs = a.Xs ? static_cast<int>(ceil_div(words, kSortThreads)) : 1;
        const int64_t grid = a.Xs ? std::min<int64_t>(a.tokens * segs, 2 * static_cast<int64_t>(sm_count)) : 1;
        void *args[] = {&a, &segs};
        return launch_pdl(reinterpret_cast<const void *>(&dispatch_small_kernel<WHOLE>), dim3(static_cast<unsigned>(grid)),
                          dim3(kSortThreads), count_smem + sizeof(int32_t) * a.pairs, s, args);
    }
    void *args[] = {&a};
    cudaError_t e = cudaSuccess;
    if (a.chunks > 1)
        e = launch_pdl(reinterpret_cast<const void *>(&histogram_kernel), dim3(static_cast<unsigned>(a.chunks)),
                       dim3(kSortThreads), sizeof(int32_t) * E1, s, args);
    if (e != cudaSuccess) return e;
    // a warp's counts of every expert are in shared memory: 32 warps up to 1024
    // experts, else eight
    const void *rank = reinterpret_cast<const void *>(&rank_kernel);
    const int warps = a.experts <= 1024 ? 32 : kSortWarps;
    const size_t rank_smem = sizeof(int32_t) * (static_cast<size_t>(warps + 1) * E1 + warps);
    e = set_max_smem(rank, rank_smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(rank, dim3(static_cast<unsigned>(a.chunks)), dim3(static_cast<unsigned>(32 * warps)), rank_smem, s, args);
    if (e != cudaSuccess || !a.Xs) return e;
    const int threads = static_cast<int>(std::min<int64_t>(256, round_up(words, 32)));
    return launch_pdl(reinterpret_cast<const void *>(&copy_rows_kernel<WHOLE>), dim3(static_cast<unsigned>(a.tokens)),
                      dim3(static_cast<unsigned>(threads)), 0, s, args);
}

template <typename T> cudaError_t launch_combine(MoeCombineArgs a, int vec, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const void *fn;
    int per;   // elements of a warp
    if constexpr (sizeof(T) == 4) {
        fn = vec == W ? reinterpret_cast<const void *>(&combine_kernel<T, W, 2, 4>)
                      : reinterpret_cast<const void *>(&combine_kernel<T, 1, 4, 4>);
        per = vec == W ? 64 * W : 128;
    } else {
        fn = vec == W ? reinterpret_cast<const void *>(&combine_kernel<T, W, 1, 8>)
                      : reinterpret_cast<const void *>(&combine_anywhere_kernel<T>);
        per = 32 * W;
    }
    a.segs = static_cast<int>(ceil_div(a.d, per));
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(a.tokens * a.segs, 8))), dim3(256), 0, s, args);
}

template <typename T> cudaError_t launch_combine_bwd(MoeCombineBwdArgs a, int vec, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const void *fn;
    if (vec == W) fn = reinterpret_cast<const void *>(&combine_bwd_kernel<T, W, 4>);
    else if constexpr (sizeof(T) == 4) fn = reinterpret_cast<const void *>(&combine_bwd_kernel<T, 1, 8>);
    else fn = reinterpret_cast<const void *>(&combine_bwd_anywhere_kernel<T>);
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(a.pairs, 8))), dim3(256), 0, s, args);
}

} // namespace

size_t moe_scratch(int64_t pairs, int64_t experts)
{
    if (one_launch(pairs, experts)) return 0;
    int64_t chunk;
    int chunks;
    moe_chunks(pairs, &chunk, &chunks);
    if (chunks == 1) return 0;
    return sizeof(int32_t) * static_cast<size_t>(round_up(chunks, 4)) * static_cast<size_t>(experts + 1);
}

cudaError_t launch_moe_dispatch(MoeDispatchArgs a, bool whole, int sm_count, cudaStream_t s)
{
    moe_chunks(a.pairs, &a.chunk, &a.chunks);
    a.pitch = static_cast<int>(round_up(a.chunks, 4));
    return whole ? launch_dispatch<true>(a, sm_count, s) : launch_dispatch<false>(a, sm_count, s);
}

cudaError_t launch_moe_combine(const MoeCombineArgs &a, int type, int vec, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_combine<float>(a, vec, s);
    case Q4_TYPE_F16: return launch_combine<__half>(a, vec, s);
    default: return launch_combine<__nv_bfloat16>(a, vec, s);
    }
}

cudaError_t launch_moe_combine_bwd(const MoeCombineBwdArgs &a, int type, int vec, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_combine_bwd<float>(a, vec, s);
    case Q4_TYPE_F16: return launch_combine_bwd<__half>(a, vec, s);
    default: return launch_combine_bwd<__nv_bfloat16>(a, vec, s);
    }
}

} // namespace q4
