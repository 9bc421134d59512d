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

// C: the cache's element type (int8_t: codes).
template <typename T, typename C, int L, bool VEC> __global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvRowsArgs a)
{
    __shared__ int32_t starts[kMaxSeqs + 1], at[kMaxSeqs];
    pdl_wait();
    pdl_launch_dependents();
    const KvCache &kc = a.c;
    const int l = threadIdx.x % L, c = 8 * l, chunk = c / kChunk, u = l % 8;
    const unsigned lanes = L == 32 ? 0xFFFFFFFFu : ((1u << L) - 1u) << (threadIdx.x % 32 / L * L);
    const int64_t items = a.rows * kc.heads, step = static_cast<int64_t>(gridDim.x) * (kThreads / L);
    int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L;
    float k[8], v[8];
    const auto load = [&] {
        const int64_t row = it / kc.heads;
        const int h = static_cast<int>(it - row * kc.heads);
        load8<T, VEC>(static_cast<const T *>(a.K) + row * a.ldk + h * kc.d, c, kc.d, k);
        load8<T, VEC>(static_cast<const T *>(a.V) + row * a.ldv + h * kc.d, c, kc.d, v);
    };
    if (it < items) load();                                 // next to the batch's description
    const Batch batch = load_batch(a, starts, at);
    for (bool first = true; it < items; it += step, first = false) {
        const int64_t row = it / kc.heads;
        const int h = static_cast<int>(it - row * kc.heads);
        const int seq = batch.seq_of(row);
        if (seq < 0) continue;
        if (!first) load();
        const int64_t pos = batch.first<true>(seq) + (row - starts[seq]);
        uint8_t *block = block_of(a, seq, pos, h);
        const int t = static_cast<int>(pos) & (kc.page_tokens - 1);
        if constexpr (sizeof(C) == 1) {
            uint32_t mk = 0, mv = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) mk = max(mk, abs_bits(k[i])), mv = max(mv, abs_bits(v[i]));
#pragma unroll
            for (int o = L / 2; o > 0; o /= 2) {
                mk = max(mk, __shfl_xor_sync(lanes, mk, o));
                mv = max(mv, __shfl_xor_sync(lanes, mv, o));
            }
            if (!block || chunk >= kc.chunks) continue;
            // a token whose keys or values are not all finite: NaN keys, no values
            const uint32_t bad = max(mk, mv) >= 0x7F800000u ? 0x7F800000u : 0u;
            const CodeScale sk = code_scale(max(mk, bad)), sv = code_scale(bad ? 0u : mv);
            int ck[8], cv[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) ck[i] = code_of(k[i], sk.factor), cv[i] = code_of(v[i], sv.factor);
            const int place = (chunk * kc.page_tokens + t) * kChunk + (((u >> 1) ^ ((t >> 1) & 3)) << 4) + 8 * (u & 1);
            const int half = kc.chunks * kc.page_tokens * kChunk;
            store_pack<int8_t, 8>(reinterpret_cast<int8_t *>(block + place), 0, 8, pack_codes<8>(ck));
            store_pack<int8_t, 8>(reinterpret_cast<int8_t *>(block + half + place), 0, 8, pack_codes<8>(cv));
            if (l == 0) {
                float *scales = reinterpret_cast<float *>(block + 2 * half);
                scales[t] = sk.scale;
                scales[kc.page_tokens + t] = sv.scale;
            }
        } else {
            Pack<C, 8> pk = pack_of<C, 8>(k), pv = pack_of<C, 8>(v);
            const bool fine = __all_sync(lanes, finite8(pk) && finite8(pv)) != 0;
            if (!block || chunk >= kc.chunks) continue;
            if (!fine) {
#pragma unroll
                for (int i = 0; i < 4; ++i) pk.w[i] = 0x7FFF7FFFu, pv.w[i] = 0u;
            }
            const int place = (chunk * kc.page_tokens + t) * 128 + ((u ^ (t & 7)) << 4);
            store_pack<C, 8>(reinterpret_cast<C *>(block + place), 0, 8, pk);
            store_pack<C, 8>(reinterpret_cast<C *>(block + kc.chunks * kc.page_tokens * 128 + place), 0, 8, pv);
        }
    }
}

template <typename T, typename C, int L, bool VEC> __global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvRowsArgs a)
{
    __shared__ int32_t starts[kMaxSeqs + 1], at[kMaxSeqs];
    pdl_wait();
    pdl_launch_dependents();
    const Batch batch = load_batch(a, starts, at);
    const KvCache &kc = a.c;
    const int l = threadIdx.x % L, c = 8 * l, chunk = c / kChunk, u = l % 8;
    const int64_t items = a.rows * kc.heads, step = static_cast<int64_t>(gridDim.x) * (kThreads / L);
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * (kThreads / L) + threadIdx.x / L; it < items; it += step) {
        const int64_t row = it / kc.heads;
        const int h = static_cast<int>(it - row * kc.heads);
        const int seq = batch.seq_of(row);
        if (seq < 0 || c >= kc.d) continue;
        const int64_t pos = batch.first<false>(seq) + (row - starts[seq]);
        const uint8_t *block = block_of(a, seq, pos, h);
        const int t = static_cast<int>(pos) & (kc.page_tokens - 1);
        float k[8] = {}, v[8] = {};
        if (block) {
            if constexpr (sizeof(C) == 1) {
                const int place = (chunk * kc.page_tokens + t) * kChunk + (((u >> 1) ^ ((t >> 1) & 3)) << 4) + 8 * (u & 1);
                const int half = kc.chunks * kc.page_tokens * kChunk;
                const uint2 wk = *reinterpret_cast<const uint2 *>(block + place), wv = *reinterpret_cast<const uint2 *>(block + half + place);
                const float *scales = reinterpret_cast<const float *>(block + 2 * half);
                const float sk = scales[t], sv = scales[kc.page_tokens + t];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t a4 = i < 4 ? wk.x : wk.y, b4 = i < 4 ? wv.x : wv.y;
                    k[i] = sk * static_cast<float>(static_cast<int8_t>(a4 >> (8 * (i & 3))));
                    v[i] = sv * static_cast<float>(static_cast<int8_t>(b4 >> (8 * (i & 3))));
                }
            } else {
                const int place = (chunk * kc.page_tokens + t) * 128 + ((u ^ (t & 7)) << 4);
                const Pack<C, 8> pk = load_pack<C, 8>(reinterpret_cast<const C *>(block + place), 0, 8);
                const Pack<C, 8> pv = load_pack<C, 8>(reinterpret_cast<const C *>(block + kc.chunks * kc.page_tokens * 128 + place), 0, 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) k[i] = elem(pk, i), v[i] = elem(pv, i);
            }
        }
        store8<T, VEC>(static_cast<T *>(a.K) + row * a.ldk + h * kc.d, c, kc.d, k);
        store8<T, VEC>(static_cast<T *>(a.V) + row * a.ldv + h * kc.d, c, kc.d, v);
    }
}

template <typename T, typename C, int L, bool VEC, bool WRITE> cudaError_t launch(KvRowsArgs a, int sm_count, cudaStream_t s)
{
    const int64_t items = a.rows * a.c.heads;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(ceil_div(items, kThreads / L), int64_t(sm_count) * 16));
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
