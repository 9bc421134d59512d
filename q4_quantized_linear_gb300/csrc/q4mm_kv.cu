// q4mm_kv.cu -- keys and values into the pages of the cache, coded to int8
// where it holds codes, and back as values.
//
// Memory-bound: each value is read once and written once. A row of one head (d
// values of K and d of V) is taken by L = 8, 16 or 32 lanes, eight values a
// lane: a lane's access is one 16-byte unit of the page's row (8 bytes of codes),
// 16 bytes of a 16-bit input or two of fp32, and the lanes of a row cover whole
// 32-byte sectors on both sides. K's and V's loads are in flight together.
#include <algorithm>

#include "q4mm_cache.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;

// Eight values of a row from dim c on, zeros past d (a multiple of 8).
template <typename T, bool VEC> __device__ __forceinline__ void load8(const T *row, int c, int d, float (&f)[8])
{
    if (c >= d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.0f;
    } else if constexpr (VEC) {
        constexpr int V = 16 / sizeof(T);
#pragma unroll
        for (int j = 0; j < 8 / V; ++j) {
            const Pack<T, V> p = load_pack<T, V>(row, c + j * V, d);
#pragma unroll
            for (int i = 0; i < V; ++i) f[j * V + i] = elem(p, i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Pack<T, 1> p = load_pack<T, 1>(row, c + i, d);
            f[i] = elem(p, 0);
        }
    }
}
template <typename T, bool VEC> __device__ __forceinline__ void store8(T *row, int c, int d, const float (&f)[8])
{
    if (c >= d) return;
    constexpr int V = VEC ? 16 / sizeof(T) : 1;
#pragma unroll
    for (int j = 0; j < 8 / V; ++j) {
        float e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = f[j * V + i];
        store_pack<T, V>(row, c + j * V, d, pack_of<T, V>(e));
    }
}

// Which sequence a row belongs to (-1: none) and its place in the cache. The
// batch's description is read once into shared memory.
struct Batch {
    const int32_t *starts, *at;
    int n_seq;
    __device__ __forceinline__ int seq_of(int64_t row) const
    {
        int lo = 0, hi = n_seq;   // the last s with starts[s] <= row
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (starts[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        return lo < n_seq && starts[lo] <= row && row < starts[lo + 1] ? lo : -1;
    }
    // the place of the sequence's first row of the batch
    template <bool WRITE> __device__ __forceinline__ int64_t first(int s) const
    {
        return WRITE ? static_cast<int64_t>(at[s]) - (starts[s + 1] - starts[s]) : at[s];
    }
};
__device__ __forceinline__ Batch load_batch(const KvRowsArgs &a, int32_t *starts, int32_t *at)
{
    for (int i = threadIdx.x; i <= a.n_seq; i += blockDim.x) {
        starts[i] = a.starts[i];
        if (i < a.n_seq) at[i] = a.at ? a.at[i] : 0;
    }
    __syncthreads();
    return Batch{starts, at, a.n_seq};
}
// The block of head h in the page of position pos, or nullptr: a position or a
// page that the cache does not have is recorded and left out.
__device__ __forceinline__ uint8_t *block_of(const KvRowsArgs &a, int seq, int64_t pos, int h)
{
    const KvCache &c = a.c;
    if (pos < 0 || pos >= c.capacity) {
        record_status(a.status, kErrCheck);
        return nullptr;
    }
    const int page = c.table[seq * c.ldt + (pos >> c.log_page)];
    if (page < 0 || page >= c.n_pages) {
        record_status(a.status, kErrCheck);
        return nullptr;
    }
    return c.pages + page * c.page_bytes + static_cast<int64_t>(h) * c.head_bytes;
}

template <typename C> __device__ __forceinline__ bool finite8(const Pack<C, 8> &p)
{
    constexpr uint32_t inf = __is_same(C, __nv_bfloat16) ? 0x7F80u : 0x7C00u;
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && (p.w[i] & 0x7FFFu) < inf && ((p.w[i] >> 16) & 0x7FFFu) < inf;
    return ok;
}

// code_of() of eight values: the product, rounded, plus 1.5 2^23 has the nearest
// integer (halves to even) in its low bits, without a conversion a value.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float factor)
{
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(__fadd_rn(__fmul_rn(x[i], factor), 12582912.0f));
    uint2 w;
    w.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    if (factor == 0.0f) w = make_uint2(0u, 0u);
    return w;
}

// Heads' rows that a thread has in flight, and CTAs an SM at most. The write alone, 6554
// tokens of 8 heads of 128: fp32 into int8 16.1 us (67 MB, 4.2 TB/s), into fp16 15.9 (5.1), bf16
// into bf16 15.9 (3.4), into int8 16.2 (2.5): by the rows, not by the bytes. The read alone, 3
// sequences of up to 8000: int8 into bf16 21.9 (97 MB, 4.4 TB/s), bf16 into bf16 23.6 (128 MB,
// 5.4); the write's tokens int8 into fp32 21.1 (67 MB, 3.2). Both together within a
// microsecond: two and four rows, 8 and 64 CTAs, the next row's loads before a row is
// stored, a CTA's rows along a head instead of a token; slower: 32-byte loads, 16 codes a lane.
constexpr int kWriteAhead = 1, kReadAhead = 2, kBlocksPerSM = 16;

// C: the cache's element type (int8_t: codes).
template <typename T, typename C, int L, bool VEC> __global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvRowsArgs a)
{
    __shared__ int32_t starts[kMaxSeqs + 1], at[kMaxSeqs];
    constexpr int U = kWriteAhead, G = kThreads / L;
    pdl_wait();
    pdl_launch_dependents();
    const KvCache &kc = a.c;
    const int l = threadIdx.x % L, c = 8 * l, chunk = c / kChunk, u = l % 8;
    const int items = static_cast<int>(a.rows) * kc.heads;
    float k[U][8], v[U][8];
    int row[U], h[U];
    const auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int it = base + i * G + threadIdx.x / L;
            row[i] = it / kc.heads, h[i] = it - row[i] * kc.heads;
            const bool there = it < items;
            if (!there) row[i] = -1;
            load8<T, VEC>(static_cast<const T *>(a.K) + row[i] * a.ldk + h[i] * kc.d, there ? c : kc.d, kc.d, k[i]);
            load8<T, VEC>(static_cast<const T *>(a.V) + row[i] * a.ldv + h[i] * kc.d, there ? c : kc.d, kc.d, v[i]);
        }
    };
    int base = static_cast<int>(blockIdx.x) * (U * G);
    load(base);                                             // next to the batch's description
    const Batch batch = load_batch(a, starts, at);
    while (true) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int seq = row[i] < 0 ? -1 : batch.seq_of(row[i]);
            const int64_t pos = seq < 0 ? 0 : batch.first<true>(seq) + (row[i] - starts[seq]);
            uint8_t *block = seq < 0 ? nullptr : block_of(a, seq, pos, h[i]);
            const bool store = block && chunk < kc.chunks;
            const int t = static_cast<int>(pos) & (kc.page_tokens - 1);
            if constexpr (sizeof(C) == 1) {
                uint32_t mk = 0, mv = 0;
#pragma unroll
                for (int j = 0; j < 8; ++j) mk = max(mk, abs_bits(k[i][j])), mv = max(mv, abs_bits(v[i][j]));
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2) {
                    mk = max(mk, __shfl_xor_sync(0xFFFFFFFFu, mk, o));
                    mv = max(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, o));
                }
                // a token whose keys or values are not all finite: NaN keys, no values
                const uint32_t bad = max(mk, mv) >= 0x7F800000u ? 0x7F800000u : 0u;
                const CodeScale sk = code_scale(max(mk, bad)), sv = code_scale(bad ? 0u : mv);
                const uint2 ck = codes8(k[i], sk.factor), cv = codes8(v[i], sv.factor);
                const int place = (chunk * kc.page_tokens + t) * kChunk + (((u >> 1) ^ ((t >> 1) & 3)) << 4) + 8 * (u & 1);
                const int half = kc.chunks * kc.page_tokens * kChunk;
                if (store) {
                    *reinterpret_cast<uint2 *>(block + place) = ck;
                    *reinterpret_cast<uint2 *>(block + half + place) = cv;
                    if (l == 0) {
                        float *scales = reinterpret_cast<float *>(block + 2 * half);
                        scales[t] = sk.scale;
                        scales[kc.page_tokens + t] = sv.scale;
                    }
                }
            } else {
                Pack<C, 8> pk = pack_of<C, 8>(k[i]), pv = pack_of<C, 8>(v[i]);
                uint32_t bad = finite8(pk) && finite8(pv) ? 0u : 1u;
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2) bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, o);
                if (bad) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) pk.w[j] = 0x7FFF7FFFu, pv.w[j] = 0u;
                }
                const int place = (chunk * kc.page_tokens + t) * 128 + ((u ^ (t & 7)) << 4);
                if (store) {
                    store_pack<C, 8>(reinterpret_cast<C *>(block + place), 0, 8, pk);
                    store_pack<C, 8>(reinterpret_cast<C *>(block + kc.chunks * kc.page_tokens * 128 + place), 0, 8, pv);
                }
            }
        }
        const int64_t next = static_cast<int64_t>(base) + static_cast<int64_t>(gridDim.x) * (U * G);
        if (next >= items) break;
        base = static_cast<int>(next);
        load(base);
    }
}

template <typename T, typename C, int L, bool VEC> __global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvRowsArgs a)
{
    __shared__ int32_t starts[kMaxSeqs + 1], at[kMaxSeqs];
    constexpr int U = kReadAhead, G = kThreads / L;
    pdl_wait();
    pdl_launch_dependents();
    const Batch batch = load_batch(a, starts, at);
    const KvCache &kc = a.c;
    const int l = threadIdx.x % L, c = 8 * l, chunk = c / kChunk, u = l % 8;
    const int items = static_cast<int>(a.rows) * kc.heads;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * (U * G); base < items; base += static_cast<int64_t>(gridDim.x) * (U * G)) {
        const uint8_t *block[U];
        int row[U], h[U], t[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int it = static_cast<int>(base) + i * G + threadIdx.x / L;
            row[i] = it / kc.heads, h[i] = it - row[i] * kc.heads;
            const int seq = it < items && c < kc.d ? batch.seq_of(row[i]) : -1;
            if (seq < 0) row[i] = -1;
            const int64_t pos = seq < 0 ? 0 : batch.first<false>(seq) + (row[i] - starts[seq]);
            block[i] = seq < 0 ? nullptr : block_of(a, seq, pos, h[i]);
            t[i] = static_cast<int>(pos) & (kc.page_tokens - 1);
        }
        if constexpr (sizeof(C) == 1) {
            uint2 wk[U], wv[U];
            float sk[U], sv[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int place = (chunk * kc.page_tokens + t[i]) * kChunk + (((u >> 1) ^ ((t[i] >> 1) & 3)) << 4) + 8 * (u & 1);
                const int half = kc.chunks * kc.page_tokens * kChunk;
                wk[i] = make_uint2(0u, 0u), wv[i] = wk[i], sk[i] = 0.0f, sv[i] = 0.0f;
                if (block[i]) {
                    wk[i] = *reinterpret_cast<const uint2 *>(block[i] + place), wv[i] = *reinterpret_cast<const uint2 *>(block[i] + half + place);
                    const float *scales = reinterpret_cast<const float *>(block[i] + 2 * half);
                    sk[i] = scales[t[i]], sv[i] = scales[kc.page_tokens + t[i]];
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (row[i] < 0) continue;
                float k[8], v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t a4 = j < 4 ? wk[i].x : wk[i].y, b4 = j < 4 ? wv[i].x : wv[i].y;
                    k[j] = sk[i] * static_cast<float>(static_cast<int8_t>(a4 >> (8 * (j & 3))));
                    v[j] = sv[i] * static_cast<float>(static_cast<int8_t>(b4 >> (8 * (j & 3))));
                }
                store8<T, VEC>(static_cast<T *>(a.K) + row[i] * a.ldk + h[i] * kc.d, c, kc.d, k);
                store8<T, VEC>(static_cast<T *>(a.V) + row[i] * a.ldv + h[i] * kc.d, c, kc.d, v);
            }
        } else {
            Pack<C, 8> pk[U], pv[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int place = (chunk * kc.page_tokens + t[i]) * 128 + ((u ^ (t[i] & 7)) << 4);
                pk[i] = zero_pack<C, 8>(), pv[i] = pk[i];
                if (block[i]) {
                    pk[i] = load_pack<C, 8>(reinterpret_cast<const C *>(block[i] + place), 0, 8);
                    pv[i] = load_pack<C, 8>(reinterpret_cast<const C *>(block[i] + kc.chunks * kc.page_tokens * 128 + place), 0, 8);
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (row[i] < 0) continue;
                float k[8], v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] = elem(pk[i], j), v[j] = elem(pv[i], j);
                store8<T, VEC>(static_cast<T *>(a.K) + row[i] * a.ldk + h[i] * kc.d, c, kc.d, k);
                store8<T, VEC>(static_cast<T *>(a.V) + row[i] * a.ldv + h[i] * kc.d, c, kc.d, v);
            }
        }
    }
}

template <typename T, typename C, int L, bool VEC, bool WRITE> cudaError_t launch(KvRowsArgs a, int sm_count, cudaStream_t s)
{
    const int64_t items = a.rows * a.c.heads, block = (WRITE ? kWriteAhead : kReadAhead) * (kThreads / L);
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ceil_div(items, block), int64_t(sm_count) * kBlocksPerSM));
    void *args[] = {&a};
    const void *f = WRITE ? reinterpret_cast<const void *>(&kv_write_kernel<T, C, L, VEC>)
                          : reinterpret_cast<const void *>(&kv_read_kernel<T, C, L, VEC>);
    return launch_pdl(f, dim3(grid), dim3(kThreads), 0, s, args);
}
template <typename T, typename C, bool WRITE> cudaError_t by_width(const KvRowsArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    const int L = a.c.chunks == 1 ? 8 : a.c.chunks == 2 ? 16 : 32;
    if (vec) {
        return L == 8 ? launch<T, C, 8, true, WRITE>(a, sm_count, s)
               : L == 16 ? launch<T, C, 16, true, WRITE>(a, sm_count, s) : launch<T, C, 32, true, WRITE>(a, sm_count, s);
    }
    return L == 8 ? launch<T, C, 8, false, WRITE>(a, sm_count, s)
           : L == 16 ? launch<T, C, 16, false, WRITE>(a, sm_count, s) : launch<T, C, 32, false, WRITE>(a, sm_count, s);
}
template <typename T, bool WRITE> cudaError_t by_cache(const KvRowsArgs &a, bool vec, int sm_count, cudaStream_t s)
{
    switch (a.c.type) {
    case Q4_TYPE_F16: return by_width<T, __half, WRITE>(a, vec, sm_count, s);
    case Q4_TYPE_BF16: return by_width<T, __nv_bfloat16, WRITE>(a, vec, sm_count, s);
    default: return by_width<T, int8_t, WRITE>(a, vec, sm_count, s);
    }
}
template <bool WRITE> cudaError_t by_type(const KvRowsArgs &a, int type, bool vec, int sm_count, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return by_cache<float, WRITE>(a, vec, sm_count, s);
    case Q4_TYPE_F16: return by_cache<__half, WRITE>(a, vec, sm_count, s);
    default: return by_cache<__nv_bfloat16, WRITE>(a, vec, sm_count, s);
    }
}

} // namespace

cudaError_t launch_kv_write(const KvRowsArgs &a, int type, bool vec, int sm_count, cudaStream_t s)
{
    return by_type<true>(a, type, vec, sm_count, s);
}
cudaError_t launch_kv_read(const KvRowsArgs &a, int type, bool vec, int sm_count, cudaStream_t s)
{
    return by_type<false>(a, type, vec, sm_count, s);
}

} // namespace q4
