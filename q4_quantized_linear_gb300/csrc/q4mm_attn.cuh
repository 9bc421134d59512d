// q4mm_attn.cuh -- what the attention kernels share: which work a CTA takes,
// the copies of a tile, and small pieces of arithmetic.
//
// An item is a block of query rows of one sequence and one cached head: row r of
// a sequence stands for new token r / group and query head head * group + r %
// group, so that all query heads of a cached head share what is read of it. An
// item's work is its tiles of tokens, from the first that any row sees to the last,
// and a.item_cost tiles more for what an item costs beside them (windowed prompts,
// whose first blocks have a tile or two: without, the CTA with the most items took
// twice the average). The work of all items in a row (sequence, head, block, tile) is
// dealt to the CTAs in equal contiguous shares: no host code needs to know the
// sequences' lengths, and a long sequence is spread over many CTAs. An item that is
// cut leaves parts (sums without their denominator, maxima, denominators), which the
// join adds in the order of the tiles.
#pragma once

#include "q4mm_cache.h"
#include "q4mm_rows.cuh"

namespace q4 {

struct Seq {
    int n, len, start, rows, blocks;   // new tokens, tokens with them, first row, query rows, blocks of them
};

__device__ __forceinline__ Seq seq_at(const AttnArgs &a, int s)
{
    const int lo = min(max(a.starts[s], 0), a.rows), hi = min(max(a.starts[s + 1], 0), a.rows);
    Seq q;
    q.n = max(hi - lo, 0);
    q.start = lo;
    q.len = max(a.lens[s], 0);
    q.rows = q.n * a.group;
    if (q.rows <= a.rows_above || q.rows > a.rows_upto) q.rows = 0;
    q.blocks = (q.rows + a.block - 1) / a.block;
    return q;
}
// Tokens lo .. hi - 1 that query row r sees. Its place is where the write puts its
// keys, past the table's end too; tokens there are not in the cache.
__device__ __forceinline__ void row_range(const AttnArgs &a, const Seq &q, int r, int &lo, int &hi)
{
    const int pos = q.len - q.n + r / a.group;
    const int upto = max(pos + 1, 0);
    hi = min(upto, a.c.capacity);
    lo = a.window > 0 ? min(max(upto - a.window, 0), hi) : 0;
}
// Tiles of block b: the first, and how many (one at least, so that rows that see
// nothing are written too); `hi`: tokens past it are seen by none of its rows.
__device__ __forceinline__ void block_tiles(const AttnArgs &a, const Seq &q, int b, int &first, int &count, int &hi)
{
    int lo, x;
    row_range(a, q, b * a.block, lo, x);
    row_range(a, q, min((b + 1) * a.block, q.rows) - 1, x, hi);
    first = lo / a.tile;
    count = max((hi + a.tile - 1) / a.tile - first, 1);
}

// The items of a CTA's share, in order. Every thread of the CTA walks alike.
struct Walk {
    int s, h, b;              // the item
    Seq q;
    int first, count, hi;     // its tiles
    int from, upto;           // those of them that are this CTA's
    int left;                 // work of the share from this item on
    int used;                 // of it in this item
    int share;

    __device__ __forceinline__ bool whole() const { return from == 0 && upto == count; }
    // The share starts at `y` of the item's work: first its cost, then a tile each.
    __device__ __forceinline__ void clip(const AttnArgs &a, int y)
    {
        used = min(left, count + a.item_cost - y);
        from = max(y - a.item_cost, 0);
        upto = max(y + used - a.item_cost, 0);
    }
    // `scan`: shared memory of n_seq + 1 numbers, free again after the next barrier.
    __device__ __forceinline__ void begin(const AttnArgs &a, long long *scan)
    {
        // few sequences: a warp's lanes share the blocks of one; many: a thread each
        // (a prompt of 2000 tokens in four, a thread each: 10 us)
        const int lanes = a.n_seq * 32 <= static_cast<int>(blockDim.x) ? 32 : a.n_seq * 8 <= static_cast<int>(blockDim.x) ? 8 : 1;
        for (int i0 = 0; i0 < a.n_seq; i0 += blockDim.x / lanes) {
            const int i = i0 + threadIdx.x / lanes;
            long long w = 0;
            if (i < a.n_seq) {
                const Seq x = seq_at(a, i);
                for (int j = threadIdx.x % lanes; j < x.blocks; j += lanes) {
                    int f, n, e;
                    block_tiles(a, x, j, f, n, e);
                    w += n + a.item_cost;
                }
            }
            for (int o = lanes / 2; o > 0; o /= 2) w += __shfl_xor_sync(0xFFFFFFFFu, w, o);
            if (i < a.n_seq && threadIdx.x % lanes == 0) scan[i] = w;
        }
        __syncthreads();
        if (threadIdx.x < 32) {
            long long carry = 0;
            for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
                const int i = i0 + threadIdx.x;
                long long v = i < a.n_seq ? scan[i] * a.c.heads : 0;
                const long long own = v;
#pragma unroll
                for (int o = 1; o < 32; o *= 2) {
                    const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
                    if (threadIdx.x >= o) v += u;
                }
                if (i < a.n_seq) scan[i] = carry + v - own;
                carry += __shfl_sync(0xFFFFFFFFu, v, 31);
            }
            if (threadIdx.x == 0) scan[a.n_seq] = carry;
        }
        __syncthreads();
        const long long total = scan[a.n_seq];
        share = total < 0x7FFFFFFF ? static_cast<int>((static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x)
                                   : static_cast<int>((total + gridDim.x - 1) / gridDim.x);
        const long long at = static_cast<long long>(share) * blockIdx.x;
        left = static_cast<int>(min(max(total - at, 0ll), static_cast<long long>(share)));
        if (left == 0) return;
        int lo = 0, hi_s = a.n_seq - 1;   // the last sequence whose work starts at or before `at`
        while (lo < hi_s) {
            const int mid = (lo + hi_s + 1) >> 1;
            if (scan[mid] <= at) lo = mid;
            else hi_s = mid - 1;
        }
        s = lo;
        q = seq_at(a, s);
        const long long own = scan[s + 1] - scan[s], x = at - scan[s];
        long long y;
        if (own < 0x7FFFFFFF) {   // (a 64-bit division takes several times as long)
            const int per = static_cast<int>(own) / a.c.heads;
            h = static_cast<int>(x) / per;
            y = static_cast<int>(x) - h * per;
        } else {
            const long long per = own / a.c.heads;
            h = static_cast<int>(x / per);
            y = x - h * per;
        }
        // the block that tile y is in: a warp looks at 32 at a time
        const int lane = threadIdx.x & 31;
        for (b = 0; b + 1 < q.blocks; b += 32) {
            long long upto_b = 0;
            if (b + lane < q.blocks) {
                block_tiles(a, q, b + lane, first, count, hi);
                upto_b = count + a.item_cost;
            }
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const long long u = __shfl_up_sync(0xFFFFFFFFu, upto_b, o);
                if (lane >= o) upto_b += u;
            }
            const unsigned past = __ballot_sync(0xFFFFFFFFu, upto_b > y);
            const int skip = past ? __ffs(past) - 1 : 32;
            if (skip > 0) y -= __shfl_sync(0xFFFFFFFFu, upto_b, skip - 1);
            if (past) {
                b += skip;
                break;
            }
        }
        block_tiles(a, q, b, first, count, hi);
        clip(a, static_cast<int>(y));
        if (from >= upto) next(a);
    }
    __device__ __forceinline__ bool valid() const { return left > 0; }
    // The next item that the share has tiles of.
    __device__ __forceinline__ void next(const AttnArgs &a)
    {
        do {
            left -= used;
            if (left <= 0) return;
            if (++b >= q.blocks) {
                b = 0;
                if (++h >= a.c.heads) {
                    h = 0;
                    do {
                        if (++s >= a.n_seq) {
                            left = 0;
                            return;
                        }
                        q = seq_at(a, s);
                    } while (q.blocks == 0);
                }
            }
            block_tiles(a, q, b, first, count, hi);
            clip(a, 0);
        } while (from >= upto);
    }
    // Parts of an item that starts in this CTA and is not finished in it.
    __device__ __forceinline__ int parts() const
    {
        return 1 + (count - upto + share - 1) / share;
    }
};

// What the join needs to know of an item that starts in this CTA and is not finished
// in it: its parts, rows, first row in the sequence and head; the sequence's first row.
__device__ __forceinline__ void put_meta(const AttnArgs &a, const Walk &w)
{
    a.meta[2 * blockIdx.x] = make_int4(w.parts(), min(a.block, w.q.rows - w.b * a.block), w.b * a.block, w.h);
    a.meta[2 * blockIdx.x + 1] = make_int4(w.q.start, 0, 0, 0);
}

// The first token that some row of the item's block sees. What lies before it is not
// there: its table entries are not looked at (a server may have given the pages back),
// its places may never have been written, and a tile that holds some of them has no
// values there (0, for a term of 0 times NaN is NaN).
__device__ __forceinline__ int first_seen(const AttnArgs &a, const Walk &w)
{
    int lo, x;
    row_range(a, w.q, w.b * a.block, lo, x);
    return lo;
}
// Page i of a sequence of which an item needs first .. upto - 1 (-1: not one of them).
// One that the cache does not have is recorded: -2, nothing is read in its place, and
// its values are 0, so that rows that do not see its tokens are what they are without it.
__device__ __forceinline__ int page_of(const AttnArgs &a, const int32_t *table, int i, int first, int upto)
{
    if (i < first || i >= upto) return -1;
    const int page = table[i];
    if (page >= 0 && page < a.c.n_pages) return page;
    record_status(a.status, kErrCheck);
    return -2;
}

// ----------------------------------------------------------- arithmetic --

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xFF800000); }
__device__ __forceinline__ uint32_t pack_f16x2_rn(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Four codes of a word to fp16, exact: the code plus 128 in the low byte of
// 1024 + (code + 128), less 1152.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t x = w ^ 0x80808080u;
    lo = hsub2_bits(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_bits(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
}

// How far a row's running maximum may be passed before the sums are scaled to
// the new one: terms stay below 2^kSlack, and most tiles scale nothing.
constexpr float kSlack = 8.0f;
// Terms are held 2^kLift times larger (below 2^15), so that small ones keep their
// bits in fp16: what is lost is below 2^-32 of the largest term.
constexpr float kLift = 7.0f;

// Values of O from element `at` on, rounded once; `at` is a multiple of 2 (8) beyond a
// row's start.
__device__ __forceinline__ void store2_out(const AttnArgs &a, int64_t at, float v0, float v1)
{
    if (a.type == Q4_TYPE_F32) {
        float *o = static_cast<float *>(a.O) + at;
        if (a.vec) *reinterpret_cast<float2 *>(o) = make_float2(v0, v1);
        else o[0] = v0, o[1] = v1;
    } else {
        uint16_t *o = static_cast<uint16_t *>(a.O) + at;
        const uint32_t u = a.type == Q4_TYPE_BF16 ? pack_bf16x2_rn(v0, v1) : pack_f16x2_rn(v0, v1);
        if (a.vec) *reinterpret_cast<uint32_t *>(o) = u;
        else o[0] = static_cast<uint16_t>(u), o[1] = static_cast<uint16_t>(u >> 16);
    }
}
__device__ __forceinline__ void store8_out(const AttnArgs &a, int64_t at, const float (&v)[8])
{
    if (a.type != Q4_TYPE_F32 && a.vec) {
        const bool bf = a.type == Q4_TYPE_BF16;
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = bf ? pack_bf16x2_rn(v[2 * i], v[2 * i + 1]) : pack_f16x2_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.O) + at) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) store2_out(a, at + i, v[i], v[i + 1]);
    }
}

// Eight values from element `at` on as words (16-bit values: 4, fp32: 8).
template <bool VEC, int N> __device__ __forceinline__ void load_raw(const void *src, int64_t at, uint32_t (&w)[N])
{
    if constexpr (VEC) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(src) + at * (N / 2));
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = p[i];
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = static_cast<const uint32_t *>(src)[at + i];
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(src) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = p[2 * i] | static_cast<uint32_t>(p[2 * i + 1]) << 16;
    }
}

} // namespace q4
