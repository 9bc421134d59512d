// q4mm_draft.cu -- what turns the logit head's rows into tokens: probabilities
// at a temperature, and the verification of drafted tokens.
//
// Both read rows as long as the vocabulary, few of them at a time, so a
// thread-block cluster takes a row: each CTA a contiguous segment, and the CTAs'
// sums meet in shared memory. The probabilities' values stay in registers between
// the pass that needs the row's sum and the one that uses it (what a longer row
// has beyond them is read again): a row is read once and written once.
#include <algorithm>

#include "q4mm_cache.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

constexpr int kMaxThreads = 1024, kMaxCluster = 8;
constexpr int kHeldValues = 32;            // of a thread, in registers

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool SUM> __device__ __forceinline__ float block_reduce(float v, float *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = SUM ? v + u : fmaxf(v, u);
    }
    __syncthreads();
    if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
    __syncthreads();
    v = buf[0];
    for (int i = 1; i < static_cast<int>(blockDim.x) / 32; ++i) v = SUM ? v + buf[i] : fmaxf(v, buf[i]);
    return v;
}
// To the same place in CTA `rank` of the cluster.
__device__ __forceinline__ void put_far(const unsigned long long *here, uint32_t rank, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(mapa_shared(smem_u32(here), rank)), "l"(v) : "memory");
}
// Every CTA's value to every CTA: all[i] is CTA i's.
__device__ __forceinline__ void exchange(unsigned long long *all, unsigned long long mine, uint32_t rank, int cluster)
{
    if (cluster == 1) {
        if (threadIdx.x == 0) all[0] = mine;
        __syncthreads();
        return;
    }
    if (static_cast<int>(threadIdx.x) < cluster) put_far(&all[rank], threadIdx.x, mine);
    cluster_sync();
}

// Elements lo .. hi - 1 of a row of n are CTA `rank`'s of `cluster`, in whole vectors.
struct Segment {
    int64_t lo, hi;
    __device__ __forceinline__ Segment(int64_t n, int cluster, uint32_t rank)
    {
        const int64_t per = ((n + cluster - 1) / cluster + 7) / 8 * 8;
        lo = per * rank < n ? per * rank : n;
        hi = lo + per < n ? lo + per : n;
    }
};

// --------------------------------------------------------- probabilities --

template <typename T, int V> __global__ void __launch_bounds__(kMaxThreads) probs_kernel(const ProbsArgs a, const int cluster)
{
    constexpr int NV = kHeldValues / V;
    __shared__ float buf[32];
    __shared__ unsigned long long all[kMaxCluster], first[kMaxCluster];
    __shared__ unsigned int lowest;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    if (cluster > 1) cluster_sync();   // every CTA runs before anything is written into its shared memory
    const int64_t row = blockIdx.x / cluster;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    float *p = a.P + row * a.ldp;
    const Segment seg(a.n, cluster, rank);
    const int step = static_cast<int>(blockDim.x) * V;
    const float temperature = a.temperature ? a.temperature[row] : 1.0f;
    const float inf = __int_as_float(0x7F800000);
    float v[NV][V];
    float m = -inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = seg.lo + static_cast<int64_t>(i) * step + threadIdx.x * V;
        if (c < seg.hi) {
            const Pack<T, V> u = load_pack<T, V>(x, c, seg.hi);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = c + j < seg.hi ? elem(u, j) : -inf;
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[i][j] = -inf;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, v[i][j]);
    const int64_t rest = seg.lo + static_cast<int64_t>(NV) * step + threadIdx.x * V;
    for (int64_t c = rest; c < seg.hi; c += step) {
        const Pack<T, V> u = load_pack<T, V>(x, c, seg.hi);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < seg.hi) m = fmaxf(m, elem(u, j));
    }
    m = block_reduce<false>(m, buf);
    if (temperature == 0.0f) {
        // the largest value, the lowest of its places
        if (threadIdx.x == 0) lowest = 0xFFFFFFFFu;
        __syncthreads();
        unsigned int at = 0xFFFFFFFFu;
        if (m > -inf)
            for (int64_t c = seg.lo + threadIdx.x * V; c < seg.hi; c += step) {
                const Pack<T, V> u = load_pack<T, V>(x, c, seg.hi);
#pragma unroll
                for (int j = V - 1; j >= 0; --j)
                    if (c + j < seg.hi && elem(u, j) == m) at = min(at, static_cast<unsigned int>(c + j));
            }
        atomicMin(&lowest, at);
        __syncthreads();
        exchange(first, static_cast<unsigned long long>(lowest) << 32 | __float_as_uint(m), rank, cluster);
        float best = -inf;
        for (int i = 0; i < cluster; ++i) best = fmaxf(best, __uint_as_float(static_cast<uint32_t>(first[i])));
        at = 0xFFFFFFFFu;
        for (int i = 0; i < cluster; ++i)
            if (__uint_as_float(static_cast<uint32_t>(first[i])) == best) at = min(at, static_cast<unsigned int>(first[i] >> 32));
        for (int64_t c = seg.lo + threadIdx.x; c < seg.hi; c += blockDim.x) p[c] = c == at ? 1.0f : 0.0f;
        return;
    }
    // 2^((x - m) f); nothing but -inf: zeros
    const float f = temperature > 0.0f ? __fdiv_rn(1.4426950408889634f, temperature) : __int_as_float(0x7FC00000);
    const float base = m == -inf ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[i][j] = exp2_fast((v[i][j] - base) * f);
            s += v[i][j];
        }
    for (int64_t c = rest; c < seg.hi; c += step) {
        const Pack<T, V> u = load_pack<T, V>(x, c, seg.hi);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < seg.hi) s += exp2_fast((elem(u, j) - base) * f);
    }
    s = block_reduce<true>(s, buf);
    exchange(all, static_cast<unsigned long long>(__float_as_uint(s)) << 32 | __float_as_uint(m), rank, cluster);
    float best = -inf, total = 0.0f;
    for (int i = 0; i < cluster; ++i) best = fmaxf(best, __uint_as_float(static_cast<uint32_t>(all[i])));
    for (int i = 0; i < cluster; ++i) {
        const float mi = __uint_as_float(static_cast<uint32_t>(all[i]));
        total += __uint_as_float(static_cast<uint32_t>(all[i] >> 32)) * (mi == best || mi == -inf ? 1.0f : exp2_fast((mi - best) * f));
    }
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    const float scale = (m == best || m == -inf ? 1.0f : exp2_fast((m - best) * f)) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t c = seg.lo + static_cast<int64_t>(i) * step + threadIdx.x * V;
        if (c >= seg.hi) continue;
        if constexpr (V == 1) {
            p[c] = v[i][0] * scale;
        } else {
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float w[4] = {v[i][j] * scale, v[i][j + 1] * scale, v[i][j + 2] * scale, v[i][j + 3] * scale};
                if (c + j < seg.hi) store_pack<float, 4>(p, c + j, seg.hi, pack_of<float, 4>(w));
            }
        }
    }
    for (int64_t c = rest; c < seg.hi; c += step) {
        const Pack<T, V> u = load_pack<T, V>(x, c, seg.hi);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < seg.hi) p[c + j] = exp2_fast((elem(u, j) - base) * f) * scale;
    }
}

template <typename T, int V> cudaError_t launch_probs(ProbsArgs a, int sm_count, cudaStream_t s)
{
    // as many CTAs a row as fill the device, while each has some work
    int cluster = 1, threads = 128;
    while (cluster < kMaxCluster && (a.n / cluster > kMaxThreads * kHeldValues || (a.rows * cluster < 2 * sm_count && a.n / cluster > 4096)))
        cluster *= 2;
    while (threads < kMaxThreads && a.n / cluster > threads * 16) threads *= 2;
    void *args[] = {&a, &cluster};
    return launch_pdl(reinterpret_cast<const void *>(&probs_kernel<T, V>), dim3(static_cast<unsigned>(a.rows * cluster)),
                      dim3(static_cast<unsigned>(threads)), 0, s, args, cluster);
}

// ---------------------------------------------------------- verification --

// The draw is by whole numbers: probabilities in steps of 2^-60 (exact from
// 2^-36 on), their sums exact whatever the order, and the place of u times the
// sum is found without a rounding; so the same numbers always give the same
// token, on any number of CTAs.
__device__ __forceinline__ unsigned long long fixed60(float p)
{
    return __float2ull_rn(fminf(fmaxf(p, 0.0f), 1.0f) * 1152921504606846976.0f);   // (NaN: 0)
}
// floor(u r), 0 <= u < 1.
__device__ __forceinline__ unsigned long long share_of(float u, unsigned long long r)
{
    u = fminf(fmaxf(u, 0.0f), 0.99999994f);
    const uint32_t bits = __float_as_uint(u);
    const int ex = static_cast<int>(bits >> 23);
    const unsigned long long mant = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int e = 150 - (ex ? ex : 1);                       // u = mant 2^-e, 24 <= e <= 149
    const unsigned long long lo = r * mant, hi = __umul64hi(r, mant);
    if (e < 64) return hi << (64 - e) | lo >> e;
    return e < 128 ? hi >> (e - 64) : 0ull;
}

constexpr int kVerifyThreads = 512;
constexpr int kMaxSpans = 4096;            // spans of a warp's access in a CTA's segment

struct Rest {
    const float *p, *q;
    int64_t known;                         // without q: the token the draft was sure of (-1: none)
    int64_t hi;
    template <int V> __device__ __forceinline__ void at(int64_t c, unsigned long long (&r)[V]) const
    {
        const Pack<float, V> x = load_pack<float, V>(p, c, hi);
        Pack<float, V> y = zero_pack<float, V>();
        if (q) y = load_pack<float, V>(q, c, hi);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const unsigned long long a = fixed60(elem(x, j)), b = fixed60(elem(y, j));
            r[j] = c + j >= hi || a <= b || c + j == known ? 0ull : a - b;
        }
    }
};

template <int V> __global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a, const int cluster)
{
    __shared__ unsigned long long spans[kMaxSpans], sums[2][kMaxCluster];
    __shared__ int kept_shared;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    if (cluster > 1) cluster_sync();   // every CTA runs before anything is written into its shared memory
    const int64_t seq = blockIdx.x / cluster;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    constexpr int kWarps = kVerifyThreads / 32;
    const int count = a.counts ? min(max(a.counts[seq], 0), a.max_draft) : a.max_draft;
    if (warp == 0) {
        int kept = count;
        for (int i0 = 0; i0 < count; i0 += 32) {
            const int i = i0 + lane;
            bool stays = false;
            if (i < count) {
                const int64_t x = a.drafted[seq * a.ldd + i];
                if (x >= 0 && x < a.n) {
                    const double px = a.P[(seq * (a.max_draft + 1) + i) * a.ldp + x];
                    const double qx = a.Q ? static_cast<double>(a.Q[(seq * a.max_draft + i) * a.ldq + x]) : 1.0;
                    stays = static_cast<double>(a.accept[seq * a.lda + i]) * qx < px;   // the product is exact
                }
            }
            const unsigned gone = __ballot_sync(0xFFFFFFFFu, i < count && !stays);
            if (gone) {
                kept = i0 + __ffs(gone) - 1;
                break;
            }
        }
        if (lane == 0) kept_shared = kept;
    }
    __syncthreads();
    const int kept = kept_shared;
    const bool refused = kept < count;
    const Segment seg(a.n, cluster, rank);
    Rest rest;
    rest.p = a.P + (seq * (a.max_draft + 1) + kept) * a.ldp;
    rest.q = refused && a.Q ? a.Q + (seq * a.max_draft + kept) * a.ldq : nullptr;
    rest.known = refused && !a.Q ? a.drafted[seq * a.ldd + kept] : -1;
    rest.hi = seg.hi;
    const int64_t step = static_cast<int64_t>(kVerifyThreads) * V;
    unsigned long long total = 0;
    // once; and once more, of p alone, where the draft leaves nothing of it
    for (int turn = 0; turn < 2; ++turn) {
        int i = 0;
        for (int64_t c0 = seg.lo; c0 < seg.hi; c0 += step, ++i) {
            unsigned long long r[V], s = 0;
            const int64_t c = c0 + tid * V;
            if (c < seg.hi) {
                rest.at<V>(c, r);
#pragma unroll
                for (int j = 0; j < V; ++j) s += r[j];
            }
#pragma unroll
            for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (lane == 0) spans[i * kWarps + warp] = s;
        }
        const int n_spans = i * kWarps;
        __syncthreads();
        unsigned long long mine = 0;
        for (int k = lane; k < n_spans; k += 32) mine += spans[k];
#pragma unroll
        for (int o = 16; o > 0; o /= 2) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
        exchange(sums[turn], mine, rank, cluster);
        total = 0;
        for (int k = 0; k < cluster; ++k) total += sums[turn][k];
        if (total > 0 || turn == 1 || (!rest.q && rest.known < 0)) {
            unsigned long long target = share_of(a.sample[seq], total), before = 0;
            for (int k = 0; k < static_cast<int>(rank); ++k) before += sums[turn][k];
            // the one CTA whose segment holds the place, and CTA 0 where there is none
            const bool here = total > 0 ? target >= before && target - before < sums[turn][rank] : rank == 0;
            if (here && warp == 0) {
                int64_t token = 0;
                if (total > 0) {
                    target -= before;
                    unsigned long long run = 0;
                    int k0 = 0;
                    for (; k0 < n_spans; k0 += 32) {
                        unsigned long long v = k0 + lane < n_spans ? spans[k0 + lane] : 0ull;
#pragma unroll
                        for (int o = 1; o < 32; o *= 2) {
                            const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                            if (lane >= o) v += u;
                        }
                        const unsigned past = __ballot_sync(0xFFFFFFFFu, run + v > target);
                        if (past) {
                            const int at = __ffs(past) - 1;
                            const unsigned long long upto = __shfl_sync(0xFFFFFFFFu, v, at > 0 ? at - 1 : 0);
                            if (at > 0) run += upto;
                            k0 += at;
                            break;
                        }
                        run += __shfl_sync(0xFFFFFFFFu, v, 31);
                    }
                    const int64_t c = seg.lo + (static_cast<int64_t>(k0) * 32 + lane) * V;
                    unsigned long long r[V] = {}, s = 0;
                    if (c < seg.hi) rest.at<V>(c, r);
#pragma unroll
                    for (int j = 0; j < V; ++j) s += r[j];
                    unsigned long long v = s;
#pragma unroll
                    for (int o = 1; o < 32; o *= 2) {
                        const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                        if (lane >= o) v += u;
                    }
                    run += v - s;                            // before this lane
                    int found = 0x7FFFFFFF;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        run += r[j];
                        if (run > target && found == 0x7FFFFFFF) found = lane * V + j;
                    }
                    found = __reduce_min_sync(0xFFFFFFFFu, found);
                    token = min(seg.lo + static_cast<int64_t>(k0) * 32 * V + found, a.n - 1);
                }
                for (int j = lane; j <= a.max_draft; j += 32)
                    a.tokens[seq * a.ldt + j] = j < kept ? a.drafted[seq * a.ldd + j] : j == kept ? static_cast<int32_t>(token) : -1;
                if (lane == 0) a.kept[seq] = kept;
            }
            return;
        }
        rest.q = nullptr;
        rest.known = -1;
        __syncthreads();
    }
}

template <int V> cudaError_t launch_verify(VerifyArgs a, cudaStream_t s)
{
    int cluster = kMaxCluster;
    while (cluster > 1 && a.n / cluster < 2048) cluster /= 2;
    void *args[] = {&a, &cluster};
    return launch_pdl(reinterpret_cast<const void *>(&verify_kernel<V>), dim3(static_cast<unsigned>(a.n_seq * cluster)),
                      dim3(kVerifyThreads), 0, s, args, cluster);
}

} // namespace

cudaError_t launch_token_probs(const ProbsArgs &a, int type, int sm_count, cudaStream_t s)
{
    RowAlign al;
    al.add(a.X, a.ldx * type_size(type));
    al.add(a.P, a.ldp * 4);
    const bool vec = al.bytes() == 16;
    switch (type) {
    case Q4_TYPE_F32: return vec ? launch_probs<float, 4>(a, sm_count, s) : launch_probs<float, 1>(a, sm_count, s);
    case Q4_TYPE_F16: return vec ? launch_probs<__half, 8>(a, sm_count, s) : launch_probs<__half, 1>(a, sm_count, s);
    default: return vec ? launch_probs<__nv_bfloat16, 8>(a, sm_count, s) : launch_probs<__nv_bfloat16, 1>(a, sm_count, s);
    }
}

cudaError_t launch_draft_verify(const VerifyArgs &a, int, cudaStream_t s)
{
    RowAlign al;
    al.add(a.P, a.ldp * 4);
    al.add(a.Q, a.ldq * 4);
    return al.bytes() == 16 ? launch_verify<4>(a, s) : launch_verify<1>(a, s);
}

} // namespace q4
