// q4mm_draft.cu -- what turns the logit head's rows into tokens: probabilities
// at a temperature, and the verification of drafted tokens.
//
// Both read rows as long as the vocabulary, few of them at a time, so a
// thread-block cluster takes a row: each CTA a contiguous segment, and the CTAs'
// sums meet in shared memory.
#include <algorithm>

#include "q4mm_cache.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

constexpr int kMaxCluster = 8;

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
// Says that this CTA runs; cluster_wait: that all do, so that their shared memory may
// be written.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
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

constexpr int kProbsMaxThreads = 512;
constexpr int kProbsBytes = 80 * 1024;     // of a segment, in shared memory at once

// P = 2^((x - max) f) / sum, f = log2(e) / T. A segment comes into shared memory by one
// bulk copy (of the aligned 16-byte words that hold some of it: a row starts
// anywhere) and is looked at twice: for a running maximum and sum a thread, and for the
// results. So a row is read once and written once (a segment past kProbsBytes is
// copied piece by piece, and again for the results). Several CTAs an SM cover one
// another's waits: 320 rows of 151936 bf16 63 us (4.6 TB/s; by 1024 threads that held
// values in registers, one CTA an SM, 205). A row alone is bound by its two passes and
// the exchange between them: 4 rows of fp32 6.9 us.
template <typename T> __global__ void __launch_bounds__(kProbsMaxThreads) probs_kernel(const ProbsArgs a, const int cluster)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(128) uint8_t piece[];
    __shared__ float buf[32];
    __shared__ unsigned long long all[kMaxCluster], first[kMaxCluster];
    __shared__ unsigned int lowest;
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    if (cluster > 1) cluster_arrive();
    __syncthreads();
    const int64_t row = blockIdx.x / cluster;
    const T *x = static_cast<const T *>(a.X) + row * a.ldx;
    const Segment seg(a.n, cluster, rank);
    const int tid = threadIdx.x, step = blockDim.x;
    const float inf = __int_as_float(0x7F800000);
    const uintptr_t begin = reinterpret_cast<uintptr_t>(x + seg.lo), end = reinterpret_cast<uintptr_t>(x + seg.hi);
    const uintptr_t base = begin & ~uintptr_t(15);
    const int64_t words = seg.hi > seg.lo ? static_cast<int64_t>((end - base + 15) / 16) : 0;
    const int64_t e0 = seg.lo - static_cast<int64_t>(begin - base) / static_cast<int64_t>(sizeof(T));   // the element at `base`
    const int64_t piece_words = kProbsBytes / 16;
    const int pieces = static_cast<int>((words + piece_words - 1) / piece_words);
    uint32_t phase = 0;
    bool ok = true;
    // f(first word, words) of each piece, in shared memory
    const auto over = [&](bool again, auto f) {
        for (int i = 0; i < pieces; ++i) {
            const int64_t w0 = i * piece_words;
            const int n = static_cast<int>(min(piece_words, words - w0));
            if (!again || pieces > 1) {
                __syncthreads();                             // the piece before has been read
                if (tid == 0) {
                    mbar_arrive_expect_tx(&bar, static_cast<uint32_t>(n) * 16u);
                    bulk_g2s(piece, reinterpret_cast<const void *>(base + w0 * 16), static_cast<uint32_t>(n) * 16u, &bar);
                }
                if (!mbar_wait(&bar, phase, landing_limit(a.wait_ns))) {
                    record_status(a.status, kErrTimeout);
                    ok = false;
                }
                phase ^= 1u;
            }
            f(w0, n);
        }
    };
    const auto word = [&](int w) {
        Pack<T, V> p;
        const uint4 u = lds128(piece + 16 * w);
        p.w[0] = u.x, p.w[1] = u.y, p.w[2] = u.z, p.w[3] = u.w;
        return p;
    };
    const float temperature = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = temperature == 0.0f;
    // (0 < f < infinity: a difference of 0 stays 0 and one of -infinity what it is)
    const float f = temperature > 0.0f ? __fdiv_rn(1.4426950408889634f, fminf(fmaxf(temperature, 1.17549435e-38f), 3.40282347e38f))
                                       : __int_as_float(0x7FC00000);
    float m = -inf, s = 0.0f;
    over(false, [&](int64_t w0, int n) {
        for (int w = tid; w < n; w += step) {
            const Pack<T, V> p = word(w);
            const int64_t e = e0 + (w0 + w) * V;
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = elem(p, j);
            if (e < seg.lo || e + V > seg.hi) {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (e + j < seg.lo || e + j >= seg.hi) v[j] = -inf;
            }
            float top = v[0];
#pragma unroll
            for (int j = 1; j < V; ++j) top = fmaxf(top, v[j]);
            if (greedy) {
                m = fmaxf(m, top);
                continue;
            }
            if (top > m) {
                s *= m == -inf ? 1.0f : exp2_fast((m - top) * f);   // (s: 0 or NaN so far where m is -inf)
                m = top;
            }
            const float from = m == -inf ? 0.0f : m;
#pragma unroll
            for (int j = 0; j < V; ++j) s += exp2_fast((v[j] - from) * f);
        }
    });
    const float mine = m;
    m = block_reduce<false>(m, buf);
    float *p = a.P + row * a.ldp;
    if (greedy) {
        // the largest value, the lowest of its places
        if (tid == 0) lowest = 0xFFFFFFFFu;
        __syncthreads();
        unsigned int at = 0xFFFFFFFFu;
        if (m > -inf)
            over(true, [&](int64_t w0, int n) {
                for (int w = tid; w < n; w += step) {
                    const Pack<T, V> u = word(w);
                    const int64_t e = e0 + (w0 + w) * V;
#pragma unroll
                    for (int j = V - 1; j >= 0; --j)
                        if (e + j >= seg.lo && e + j < seg.hi && elem(u, j) == m) at = min(at, static_cast<unsigned int>(e + j));
                }
            });
        atomicMin(&lowest, at);
        __syncthreads();
        if (cluster > 1) cluster_wait();
        exchange(first, static_cast<unsigned long long>(lowest) << 32 | __float_as_uint(m), rank, cluster);
        float best = -inf;
        for (int i = 0; i < cluster; ++i) best = fmaxf(best, __uint_as_float(static_cast<uint32_t>(first[i])));
        at = 0xFFFFFFFFu;
        for (int i = 0; i < cluster; ++i)
            if (__uint_as_float(static_cast<uint32_t>(first[i])) == best) at = min(at, static_cast<unsigned int>(first[i] >> 32));
        for (int64_t c = seg.lo + tid; c < seg.hi; c += step) p[c] = c == at ? 1.0f : 0.0f;
        return;
    }
    s = block_reduce<true>(mine == -inf || mine == m ? s : s * exp2_fast((mine - m) * f), buf);
    if (cluster > 1) cluster_wait();
    exchange(all, static_cast<unsigned long long>(__float_as_uint(s)) << 32 | __float_as_uint(m), rank, cluster);
    float best = -inf, total = 0.0f;
    for (int i = 0; i < cluster; ++i) best = fmaxf(best, __uint_as_float(static_cast<uint32_t>(all[i])));
    for (int i = 0; i < cluster; ++i) {
        const float mi = __uint_as_float(static_cast<uint32_t>(all[i]));
        total += __uint_as_float(static_cast<uint32_t>(all[i] >> 32)) * (mi == best || mi == -inf ? 1.0f : exp2_fast((mi - best) * f));
    }
    if (!ok) total = __int_as_float(0x7FC00000);
    // nothing but -inf: zeros
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total), from = best == -inf ? 0.0f : best;
    // whole vectors of results where they start on 16 bytes as the words of x do
    const bool vec = ((reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(e0) * 4) & 15) == 0;
    over(true, [&](int64_t w0, int n) {
        if (vec) {
            for (int w = tid; w < n; w += step) {
                const Pack<T, V> u = word(w);
                const int64_t e = e0 + (w0 + w) * V;
                float v[V];
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = exp2_fast((elem(u, j) - from) * f) * inv;
                if (e >= seg.lo && e + V <= seg.hi) {
#pragma unroll
                    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(p + e + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        if (e + j >= seg.lo && e + j < seg.hi) p[e + j] = v[j];
                }
            }
        } else {
            const T *values = reinterpret_cast<const T *>(piece);
            const int64_t at = e0 + w0 * V;
            for (int i = tid; i < n * V; i += step) {
                const int64_t e = at + i;
                if (e >= seg.lo && e < seg.hi) p[e] = exp2_fast((elem(load_pack<T, 1>(values, i, n * V), 0) - from) * f) * inv;
            }
        }
    });
}

template <typename T> cudaError_t launch_probs(ProbsArgs a, int sm_count, cudaStream_t s)
{
    // CTAs enough for four an SM while each has some work, and segments that fit
    int cluster = 1;
    const auto bytes = [&] { return static_cast<int64_t>(sizeof(T)) * ceil_div(a.n, cluster); };
    while (cluster < kMaxCluster && (bytes() > kProbsBytes / 2 || (a.rows * cluster < 4 * sm_count && a.n / cluster > 4096))) cluster *= 2;
    const size_t smem = static_cast<size_t>(std::min<int64_t>(kProbsBytes, round_up(bytes() + 8 * static_cast<int64_t>(sizeof(T)) + 32, 128)));
    const void *f = reinterpret_cast<const void *>(&probs_kernel<T>);
    const cudaError_t e = set_max_smem(f, kProbsBytes);
    if (e != cudaSuccess) return e;
    // (4 rows of 151936: 512 threads 6.7 us, 256 7.3; 320 rows: 78 and 68)
    const unsigned threads = a.rows * cluster > sm_count ? 256 : kProbsMaxThreads;
    void *args[] = {&a, &cluster};
    return launch_pdl(f, dim3(static_cast<unsigned>(a.rows * cluster)), dim3(threads), smem, s, args, cluster);
}

// ---------------------------------------------------------- verification --

__device__ __forceinline__ float probability(float p) { return fminf(fmaxf(p, 0.0f), 1.0f); }   // (NaN: 0)

// The draw is by whole numbers: probabilities in steps of 2^-60 (exact from 2^-36
// on), their sums exact whatever the order, and the place of u times the sum is
// found without a rounding; so the same numbers always give the same token, on any
// number of CTAs.
//   A probability x is cut into steps of 2^-22, 2^-45 and 2^-60 by adding 1.5 2^23
// steps in fp32: the sum is rounded to whole steps, its bits count them, and what is
// left over is exact. The counts of p - q are differences of those bits: no
// conversion to 64-bit integers and no shifts by a variable, which bound this kernel
// (64 slots of 151936: 23 us; 32 by shifts, 57 by conversions).
struct Steps {
    int a = 0, b = 0, c = 0;               // of 2^-22, 2^-45 and 2^-60
    __device__ __forceinline__ void add(float p, float q)
    {
        constexpr float kA = 3.0f, kB = 3.0f * 1.1920928955078125e-7f, kC = 1.5f * 7.275957614183426e-12f;   // 1.5 2^1, 2^-22, 2^-37
        p = probability(p), q = probability(q);
        const float pa = p + kA, qa = q + kA, p1 = p - (pa - kA), q1 = q - (qa - kA);
        const float pb = p1 + kB, qb = q1 + kB, p2 = p1 - (pb - kB), q2 = q1 - (qb - kB);
        const float pc = p2 + kC, qc = q2 + kC;
        if (p > q) {
            a += __float_as_int(pa) - __float_as_int(qa);
            b += __float_as_int(pb) - __float_as_int(qb);
            c += __float_as_int(pc) - __float_as_int(qc);
        }
    }
    __device__ __forceinline__ unsigned long long total() const
    {
        return static_cast<unsigned long long>((static_cast<long long>(a) << 38) + (static_cast<long long>(b) << 15) + c);
    }
};
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

constexpr int kVerifyThreads = 1024, kVerifyWarps = kVerifyThreads / 32;   // at most

struct Rest {
    const float *p, *q;
    int64_t known;                         // without q: the token the draft was sure of (-1: none)
    int64_t hi;
    template <int V> __device__ __forceinline__ void load(int64_t c, Pack<float, V> &x, Pack<float, V> &y) const
    {
        x = zero_pack<float, V>(), y = x;
        if (c >= hi) return;
        x = load_pack<float, V>(p, c, hi);
        if (q) y = load_pack<float, V>(q, c, hi);
    }
    // what is left of elements c ..: added to s, or one by one
    template <int V> __device__ __forceinline__ void add(int64_t c, const Pack<float, V> &x, const Pack<float, V> &y, Steps &s) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) s.add(c + j == known ? 0.0f : elem(x, j), elem(y, j));
    }
    template <int V> __device__ __forceinline__ void of(int64_t c, const Pack<float, V> &x, const Pack<float, V> &y, unsigned long long (&r)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Steps s;
            s.add(c + j == known ? 0.0f : elem(x, j), elem(y, j));
            r[j] = s.total();
        }
    }
};
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long s)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}
// The first of n sums (a lane each) at which the running sum from `run` on passes
// `target`, and the running sum before it. n - 1 if none does.
__device__ __forceinline__ int find(unsigned long long own, int n, unsigned long long target, unsigned long long &run)
{
    const int lane = threadIdx.x % 32;
    unsigned long long v = lane < n ? own : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
    }
    const unsigned past = __ballot_sync(0xFFFFFFFFu, lane < n && run + v > target);
    const int at = past ? __ffs(past) - 1 : n - 1;
    const unsigned long long before = __shfl_sync(0xFFFFFFFFu, v, at > 0 ? at - 1 : 0);
    if (at > 0) run += before;
    return at;
}

// A CTA's segment is cut into a contiguous stretch a warp, and that into batches of
// kAhead accesses, whose sums are kept: they give the total, and the batch that holds
// the drawn place, which one warp reads once more (a search by all the CTA's warps, a
// stretch, an access and a lane at a time: 64 slots 24.6 us for 22.8). One slot is bound by
// what follows one another: the acceptance test, a segment's read, the exchange, the
// search's read (11.7 us, of which a launch takes 2).
constexpr int kAhead = 4, kMaxBatches = 1024;
static_assert(kMaxVerifyVocab / kMaxCluster <= kMaxBatches * kAhead * 32, "a segment's batches, of one element an access");

template <int V> __global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const VerifyArgs a, const int cluster)
{
    __shared__ unsigned long long spans[kMaxBatches], sums[2][kMaxCluster];
    __shared__ int kept_shared;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t rank = cluster > 1 ? cluster_ctarank() : 0u;
    if (cluster > 1) cluster_arrive();
    const int64_t seq = blockIdx.x / cluster;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, warps = blockDim.x / 32;
    int count = a.max_draft;
    if (a.counts) count = min(max(a.counts[seq], 0), a.max_draft);
    if (warp == 0) {
        int kept = count;
        for (int i0 = 0; i0 < a.max_draft; i0 += 32) {
            const int i = i0 + lane;
            bool stays = false;
            if (i < a.max_draft) {                           // (count may still be on its way)
                const float u = a.accept[seq * a.lda + i];
                const int64_t x = a.drafted[seq * a.ldd + i];
                if (x >= 0 && x < a.n) {
                    const double px = probability(a.P[(seq * (a.max_draft + 1) + i) * a.ldp + x]);
                    const double qx = a.Q ? static_cast<double>(probability(a.Q[(seq * a.max_draft + i) * a.ldq + x])) : 1.0;
                    stays = static_cast<double>(u) * qx < px;   // the product is exact
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
    const float u = a.sample[seq];
    __syncthreads();
    const int kept = kept_shared;
    const bool refused = kept < count;
    const Segment seg(a.n, cluster, rank);
    Rest rest;
    rest.p = a.P + (seq * (a.max_draft + 1) + kept) * a.ldp;
    rest.q = refused && a.Q ? a.Q + (seq * a.max_draft + kept) * a.ldq : nullptr;
    rest.known = refused && !a.Q ? a.drafted[seq * a.ldd + kept] : -1;
    rest.hi = seg.hi;
    constexpr int kBatch = kAhead * 32 * V;
    const int64_t per = ((seg.hi - seg.lo + warps - 1) / warps + 7) / 8 * 8;      // a warp's stretch, whole vectors
    const int batches = static_cast<int>((per + kBatch - 1) / kBatch);
    // a batch's accesses, in flight together
    const auto fetch = [&](int64_t from, int64_t to, Pack<float, V> (&x)[kAhead], Pack<float, V> (&y)[kAhead]) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t c = from + (i * 32 + lane) * V;
            rest.load<V>(c < to ? c : rest.hi, x[i], y[i]);
        }
    };
    unsigned long long total = 0;
    // once; and once more, of p alone, where the draft leaves nothing of it
    for (int turn = 0; turn < 2; ++turn) {
        const int64_t lo = seg.lo + warp * per, hi = min(lo + per, seg.hi);
        for (int b = 0; b < batches; ++b) {
            Pack<float, V> x[kAhead], y[kAhead];
            fetch(lo + b * kBatch, hi, x, y);
            Steps st;
#pragma unroll
            for (int i = 0; i < kAhead; ++i) rest.add<V>(lo + b * kBatch + (i * 32 + lane) * V, x[i], y[i], st);
            const unsigned long long s = warp_sum(st.total());
            if (lane == 0) spans[warp * batches + b] = s;
        }
        __syncthreads();
        const int n_spans = warps * batches;
        unsigned long long mine = 0;
        for (int k = lane; k < n_spans; k += 32) mine += spans[k];
        mine = warp_sum(mine);
        if (cluster > 1 && turn == 0) cluster_wait();
        exchange(sums[turn], mine, rank, cluster);
        total = 0;
        for (int k = 0; k < cluster; ++k) total += sums[turn][k];
        if (total > 0 || turn == 1 || (!rest.q && rest.known < 0)) {
            unsigned long long target = share_of(u, total), before = 0;
            for (int k = 0; k < static_cast<int>(rank); ++k) before += sums[turn][k];
            // the one CTA whose segment holds the place, and CTA 0 where there is none
            const bool here = total > 0 ? target >= before && target - before < sums[turn][rank] : rank == 0;
            if (!here) return;
            if (warp != 0) return;
            int64_t token = 0;
            if (total > 0) {
                target -= before;
                unsigned long long run = 0;
                int k0 = 0;
                for (; k0 + 32 < n_spans; k0 += 32) {
                    const unsigned long long s = warp_sum(spans[k0 + lane]);
                    if (run + s > target) break;
                    run += s;
                }
                const int k = k0 + find(k0 + lane < n_spans ? spans[k0 + lane] : 0ull, min(32, n_spans - k0), target, run);
                const int64_t from = seg.lo + k / batches * per, c0 = from + k % batches * kBatch;
                Pack<float, V> x[kAhead], y[kAhead];
                fetch(c0, min(from + per, seg.hi), x, y);
                bool found = false;
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    unsigned long long r[V], s = 0;
                    rest.of<V>(c0 + (i * 32 + lane) * V, x[i], y[i], r);
#pragma unroll
                    for (int j = 0; j < V; ++j) s += r[j];
                    const unsigned long long all = warp_sum(s);
                    if (found || run + all <= target) {
                        run += all;
                        continue;
                    }
                    found = true;
                    const int at = find(s, 32, target, run);
                    int which = 0;
#pragma unroll
                    for (int j = V - 1; j >= 0; --j) {
                        unsigned long long upto = run;
#pragma unroll
                        for (int e = 0; e <= j; ++e) upto += r[e];
                        if (upto > target) which = j;
                    }
                    which = __shfl_sync(0xFFFFFFFFu, which, at);
                    token = min(c0 + (i * 32 + at) * V + which, a.n - 1);
                }
            }
            for (int j = lane; j <= a.max_draft; j += 32)
                a.tokens[seq * a.ldt + j] = j < kept ? a.drafted[seq * a.ldd + j] : j == kept ? static_cast<int32_t>(token) : -1;
            if (lane == 0) a.kept[seq] = kept;
            return;
        }
        rest.q = nullptr;
        rest.known = -1;
        __syncthreads();
    }
}

template <int V> cudaError_t launch_verify(VerifyArgs a, int sm_count, cudaStream_t s)
{
    int cluster = kMaxCluster;
    while (cluster > 1 && a.n / cluster < 2048) cluster /= 2;
    // few CTAs: many threads each, to have a segment in flight at once; many: small ones,
    // which all fit at once (64 slots: 512 threads 71 us)
    const unsigned threads = a.n_seq * cluster > sm_count ? 256 : kVerifyThreads;
    void *args[] = {&a, &cluster};
    return launch_pdl(reinterpret_cast<const void *>(&verify_kernel<V>), dim3(static_cast<unsigned>(a.n_seq * cluster)), dim3(threads), 0, s,
                      args, cluster);
}

} // namespace

cudaError_t launch_token_probs(const ProbsArgs &a, int type, int sm_count, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_probs<float>(a, sm_count, s);
    case Q4_TYPE_F16: return launch_probs<__half>(a, sm_count, s);
    default: return launch_probs<__nv_bfloat16>(a, sm_count, s);
    }
}

cudaError_t launch_draft_verify(const VerifyArgs &a, int sm_count, cudaStream_t s)
{
    RowAlign al;
    al.add(a.P, a.ldp * 4);
    al.add(a.Q, a.ldq * 4);
    return al.bytes() == 16 ? launch_verify<4>(a, sm_count, s) : launch_verify<1>(a, sm_count, s);
}

} // namespace q4
