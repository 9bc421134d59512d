// q4mm_attn_warp.cuh -- attention of few query rows over the paged cache, on the
// warp-level MMA: o = sum_j p_j v_j / sum_j p_j, p_j = 2^(s_j - m), s_j = scale
// log2(e) <q, k_j>, in one pass over the tokens with a running maximum m.
//
// For few rows the bound is the read of the cache. A warp of the CTA copies tiles
// of 64 tokens into a ring, as the pages have them: a page of a head is one copy (by
// rows of 64 dims of K and of V, 16 copies of 2 KB a tile of 16-token pages, the copies'
// issue took 1250 clocks a tile); four warps compute. A block of 16 query
// rows: each warp takes 16 of a tile's tokens, with a running state of its own,
// joined at the item's end; of 32 rows: two warps by rows, two by tokens; of 64:
// four by rows. So each value of the cache is turned into an operand once for 16
// and 32 rows, and by four warps for 64 rows.
//   Scores and terms stay in registers: the accumulator of S = Q K^T has the
// layout of the A operand of P V.
//   Codes of an int8 cache are exact in fp16; a token's key scale multiplies its
// scores, its value scale its term. Terms times value scales are brought into
// fp16's range by a power of two of the tokens that the row has seen (E), the sums
// with them.
//   TERMS = 2 (fp32 queries and outputs): queries, scaled by a power of two a row,
// and terms are split into two fp16 numbers (22 bits); the MMA cuts its running
// sum to fp32, so the sums over a tile start at zero and are added in fp32.
//   A running maximum is raised only where a row's scores pass it by 2^8, and what
// a row's four lanes have seen is brought together only then.
//   Places before a block's first visible token and past its last are never looked at
// as values: what is in their place in the ring may be another sequence's, of a page
// that was never written at that, so the warps that multiply by it clear it first.
//   Measured, 32 heads on 8 of 128: 16 x 5 tokens over up to 4096, bf16 44 us (203 MB,
// 4.6 TB/s); 16 x 1 over up to 8192, int8 45 with its write (153 MB; the chains from
// codes to products, 55 % of the issue slots), without it 42, fp32 over int8 54; one token
// over 1000, fp32 15 with its write (three launches that wait for one another; 12 with
// inputs in L2); 540 over 8100, fp32 over fp16 363 and over int8 577 (products: four for
// the two of 16-bit types). At 128 dims the blocks of 64 rows spill: 260 bytes a thread for
// 16-bit types, 428 over codes, 484 and 692 for fp32; a block of 16 over codes 32.
#pragma once

#include <type_traits>

#include "q4mm_attn.cuh"

namespace q4 {
namespace {

constexpr int kF16 = 0, kBF16 = 1, kI8 = 2;   // operands: fp16 or bf16 as cached, or codes as fp16
constexpr int kComputeWarps = 4;
constexpr int kAttnThreads = (kComputeWarps + 1) * 32;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF> __device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128_at(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
// Value scales up to v: e is raised so that they are below 2^e, and what the sums
// so far are multiplied by is returned.
__device__ __forceinline__ float raise(int &e, float v)
{
    if (v < pow2(e)) return 1.0f;
    const int to = min(((__float_as_int(v) >> 23) & 255) - 126, 126);
    const float down = to - e > 126 ? 0.0f : pow2(e - to);
    e = to;
    return down;
}
__device__ __forceinline__ void compute_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kComputeWarps * 32) : "memory"); }

// DP: 64 x chunks, or 256 for three and four chunks. WM: 16-row slices of a block.
template <int KIND, int TERMS, int WM, int DP> struct WarpShape {
    static constexpr int kBlock = 16 * WM, kWN = kComputeWarps / WM, kTokens = kWarpTile / kWN;
    static constexpr int kNT = kTokens / 8;                 // score column tiles of a warp
    static constexpr int kRowBytes = KIND == kI8 ? 64 : 128;   // of a token in a chunk
    static constexpr int kMaxChunks = DP / kChunk;
    static constexpr int kQStride = DP * 2 + 16;            // bytes of a query row in shared memory
    static constexpr int kQBytes = kBlock * kQStride * TERMS;
    static constexpr int kRedBytes = WM * (kWN - 1) * 16 * DP / 2 * 4;   // sums handed over at an item's end, half the dims at once
    static constexpr int kFixed = kQBytes + kRedBytes + kBlock * 4 + 4 * 16 * 8 + 144;
    // Decode over codes is bound by its instructions' latencies: three CTAs an SM (128
    // registers, queries from shared memory each time) instead of two.
    static constexpr int kPerSM = DP > 128 ? 1 : KIND == kI8 && TERMS == 1 && WM == 1 ? 3 : 2;
    static constexpr bool kQInRegs = DP <= 128 && TERMS == 1 && kPerSM == 2;
};
inline int warp_stage_bytes(int chunks, int ctype)
{
    return ctype == Q4_TYPE_I8 ? kWarpTile * (2 * chunks * 64 + 8) : kWarpTile * 2 * chunks * 128;
}

// A wait that pauses little: a suspended one resumes some 170 ns late.
__device__ __forceinline__ bool tile_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    for (int i = 0; i < 64; ++i) {
        if (mbar_test_wait(bar, parity)) return true;
        __nanosleep(20);
    }
    return mbar_wait(bar, parity, limit_ns);
}

template <int KIND, int TERMS, int WM, int DP>
__global__ void __launch_bounds__(kAttnThreads, WarpShape<KIND, TERMS, WM, DP>::kPerSM) attn_warp_kernel(const AttnArgs a)
{
    using S = WarpShape<KIND, TERMS, WM, DP>;
    constexpr bool BF = KIND == kBF16;
    constexpr int WN = S::kWN, NT = S::kNT, NG = NT / 2, RB = S::kRowBytes, OT = DP / 8;
    extern __shared__ __align__(128) uint8_t ring[];        // tiles, then what follows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int chunks = DP <= 128 ? DP / kChunk : a.c.chunks;
    // A tile in the ring: blocks of `together` tokens (a page, or the tile where pages
    // are longer), each K [chunk][token], V the same, K's scales, V's.
    const int log_together = min(a.c.log_page, 6), together = 1 << log_together;
    const int chunk_bytes = together * RB, v_at = chunks * chunk_bytes, scales_at = 2 * v_at;
    const int block_bytes = scales_at + (KIND == kI8 ? together * 8 : 0);
    const int stage_bytes = (kWarpTile >> log_together) * block_bytes;
    uint8_t *qs = ring + a.stages * stage_bytes;
    float *red = reinterpret_cast<float *>(qs + S::kQBytes);
    float *row_factor = red + S::kRedBytes / 4;
    float2 *red_ml = reinterpret_cast<float2 *>(row_factor + S::kBlock);   // [4 warps][16]
    uint64_t *full = reinterpret_cast<uint64_t *>(red_ml + 4 * 16), *empty = full + 8;
    int *abort = reinterpret_cast<int *>(empty + 8);
    if (tid == 0) {
        for (int i = 0; i < a.stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kComputeWarps);
        *abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_launch_dependents();
    Walk w;
    static_assert(S::kQBytes + S::kRedBytes >= 8 * (kMaxSeqs + 1), "room for the walk's scan");
    w.begin(a, reinterpret_cast<long long *>(qs));
    __syncthreads();
    if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);

    if (warp == kComputeWarps) {
        // ---------------------------------------------------------- copies
        int stage = 0;
        uint32_t phase = 0;
        long long issued = 0;
        bool ok = true;
        const int in_page = a.c.page_tokens, log_page = a.c.log_page;
        const int per_page = 2 * chunks + (KIND == kI8 ? 2 : 0);
        for (; ok && w.valid(); w.next(a)) {
            const int32_t *table = a.c.table + w.s * a.c.ldt;
            const uint8_t *head = a.c.pages + static_cast<int64_t>(w.h) * a.c.head_bytes;
            const int end = w.hi, pages = (end + in_page - 1) >> log_page, first_page = first_seen(a, w) >> log_page;
            // lane l holds page held + l of the sequence, and the one 32 further on
            int held = ((w.first + w.from) * kWarpTile) >> log_page;
            int page = page_of(a, table, held + lane, first_page, pages), ahead = page_of(a, table, held + 32 + lane, first_page, pages);
            for (int t = w.from; t < w.upto; ++t) {
                const int t0 = (w.first + t) * kWarpTile, tokens = min(max(end - t0, 0), kWarpTile);
                const int p0 = t0 >> log_page;
                // whole pages, and the tokens of one that is not (or is longer than a tile)
                const int whole = in_page <= kWarpTile ? tokens >> log_page : 0, rest = tokens - (whole << log_page);
                if (p0 >= held + 32) {                      // (a tile's pages never straddle: 32 is a multiple of their number)
                    page = ahead;
                    held += 32;
                    ahead = page_of(a, table, held + 32 + lane, first_page, pages);
                }
                if (*reinterpret_cast<volatile int *>(abort)) { ok = false; break; }
                if (issued >= a.stages && !tile_wait(&empty[stage], phase ^ 1u, a.wait_ns)) {
                    *reinterpret_cast<volatile int *>(abort) = 1;
                    record_status(a.status, kErrTimeout);
                    ok = false;
                }
                ok = __all_sync(0xFFFFFFFFu, ok) != 0;
                if (!ok) break;
                uint8_t *dst = ring + stage * stage_bytes;
                const int rest_scales = KIND == kI8 ? (rest + 3) & ~3 : 0;
                const int y = lane - 8;                     // lanes 8 and on: a piece each of the page that is not whole
                const int pg = __shfl_sync(0xFFFFFFFFu, page, min(p0 - held + min(lane, whole), 31));
                const bool mine = lane < whole || (y >= 0 && y < per_page && rest > 0);   // the lane has something to copy
                const bool there = mine && pg >= 0;
                uint32_t bytes = static_cast<uint32_t>(whole * block_bytes + rest * 2 * chunks * RB + 8 * rest_scales);
                if (__any_sync(0xFFFFFFFFu, there != mine)) {
                    // pages behind the window are left out; one that the cache does not have has no
                    // values and no scales
                    for (unsigned bad = __ballot_sync(0xFFFFFFFFu, mine && pg == -2 && y <= 0); bad != 0; bad &= bad - 1) {
                        const int at = min(__ffs(bad) - 1, whole) * block_bytes + v_at;
                        for (int x = lane; x < (block_bytes - v_at) / 16; x += 32) sts128(dst + at + 16 * x, make_uint4(0u, 0u, 0u, 0u));
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const int own = !there ? 0 : lane < whole ? block_bytes : y < 2 * chunks ? rest * RB : rest_scales * 4;
                    bytes = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(own));
                }
                if (lane == 0) mbar_arrive_expect_tx(&full[stage], bytes);
                __syncwarp();
                const uint8_t *src = head + pg * a.c.page_bytes;
                if (there && lane < whole) {
                    bulk_g2s(dst + lane * block_bytes, src, static_cast<uint32_t>(block_bytes), &full[stage]);
                } else if (there) {
                    const int in = in_page <= kWarpTile ? 0 : t0 & (in_page - 1);
                    dst += whole * block_bytes;
                    if (y < 2 * chunks)
                        bulk_g2s(dst + y * chunk_bytes, src + (y * in_page + in) * RB, static_cast<uint32_t>(rest * RB), &full[stage]);
                    else
                        bulk_g2s(dst + scales_at + (y - 2 * chunks) * (together * 4), src + 2 * chunks * in_page * RB + ((y - 2 * chunks) * in_page + in) * 4,
                                 static_cast<uint32_t>(rest_scales * 4), &full[stage]);
                }
                ++issued;
                if (++stage == a.stages) stage = 0, phase ^= 1u;
            }
        }
        // no copy may be landing when the CTA leaves
        for (long long i = issued > a.stages ? issued - a.stages : 0; i < issued; ++i)
            if (!mbar_wait(&full[i % a.stages], static_cast<uint32_t>(i / a.stages) & 1u, landing_limit(a.wait_ns)))
                record_status(a.status, kErrTimeout);
        return;
    }

    // ------------------------------------------------------------- compute
    const int wm = warp / WN, wn = warp % WN;
    const uint32_t qbase = smem_u32(qs), ring_at = smem_u32(ring);
    // Where a lane reads: of K (ldmatrix: 8 tokens x 32 dims; codes: 16 bytes of token
    // g), of V (ldmatrix: 16 tokens x 16 dims; codes: 8 dims of tokens 2 c, 2 c + 1, ..),
    // and the blocks of the warp's tokens, 16 at a time.
    const uint32_t k_lane = KIND == kI8 ? g * 64 + ((c ^ ((g >> 1) & 3)) << 4) : (lane & 7) * 128 + (((lane >> 3) ^ (lane & 7)) << 4);
    const uint32_t v_lane = v_at + (KIND == kI8 ? 2 * c * 64 + (((g >> 1) ^ c) << 4) + 8 * (g & 1)
                                                : (lane & 15) * 128 + (((lane >> 4) ^ (lane & 7)) << 4));
    uint32_t off[NG], scale_off[KIND == kI8 ? NG : 1];
#pragma unroll
    for (int i = 0; i < NG; ++i) {
        const int tok = wn * S::kTokens + 16 * i, block = (tok >> log_together) * block_bytes, in = tok & (together - 1);
        off[i] = block + in * RB;
        if constexpr (KIND == kI8) scale_off[i] = block + scales_at + in * 4;
    }
    int stage = 0;
    uint32_t phase = 0;
    bool alive = true;                                      // a wait ran out: no tile is looked at any more
    for (; w.valid(); w.next(a)) {
        // Queries: DP / 8 threads a row, eight dims each, four rows of a thread in flight.
        compute_barrier();                                  // the item before is done with them
        {
            constexpr int L = DP / 8, kRows = kComputeWarps * 32 / L, kPasses = S::kBlock / kRows, kBatch = kPasses < 4 ? kPasses : 4;
            const int x = tid % L;
            for (int r0 = tid / L; r0 < S::kBlock; r0 += kBatch * kRows) {
                // (raw values first: all rows' loads are in flight together)
                using Raw = Pack<float, TERMS == 2 ? 8 : 4, TERMS == 2 ? 32 : 16>;
                Raw raw[kBatch];
                const auto fetch = [&](auto whole_vectors) {
#pragma unroll
                    for (int p = 0; p < kBatch; ++p) {
                        const int row = w.b * S::kBlock + r0 + p * kRows;
#pragma unroll
                        for (int i = 0; i < Raw::kWords; ++i) raw[p].w[i] = 0u;
                        if (row < w.q.rows && 8 * x < a.c.d) {
                            const int i = row / a.group, head = w.h * a.group + row - i * a.group;
                            const int64_t at = (static_cast<int64_t>(w.q.start) + i) * a.ldq + static_cast<int64_t>(head) * a.c.d + 8 * x;
                            load_raw<decltype(whole_vectors)::value>(a.Q, at, raw[p].w);
                        }
                    }
                };
                if (a.vec) fetch(std::true_type{});
                else fetch(std::false_type{});
                float f[kBatch][8];
#pragma unroll
                for (int p = 0; p < kBatch; ++p)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if constexpr (TERMS == 2) {
                            f[p][i] = __uint_as_float(raw[p].w[i]);
                        } else {
                            const uint32_t u = raw[p].w[i / 2] >> (16 * (i & 1));
                            const float as_half = __half2float(__ushort_as_half(static_cast<unsigned short>(u))), as_bf = __uint_as_float(u << 16);
                            f[p][i] = KIND == kF16 ? as_half : KIND == kBF16 ? as_bf : a.type == Q4_TYPE_BF16 ? as_bf : as_half;
                        }
                    }
#pragma unroll
                for (int p = 0; p < kBatch; ++p) {
                    const int r = r0 + p * kRows;
                    float factor = a.scale_log2;
                    if (KIND == kI8 || TERMS == 2) {
                        // to fp16's range by a power of two: the largest in 2^12 .. 2^13
                        uint32_t mb = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) mb = max(mb, abs_bits(f[p][i]));
#pragma unroll
                        for (int o = L / 2; o > 0; o /= 2) mb = max(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, o));
                        if (mb >= 0x7F800000u) {
                            factor = __uint_as_float(0x7FC00000u);  // a query that is not finite: NaN
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[p][i] = 0.0f;
                        } else if (mb != 0u) {
                            const int e = min(max(139 - static_cast<int>(mb >> 23), -126), 126);   // 12 - exponent
                            const float up = pow2(e);
#pragma unroll
                            for (int i = 0; i < 8; ++i) f[p][i] *= up;
                            factor *= pow2(-e);
                        }
                    }
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (BF) {
                            hi[i] = pack_bf16x2_rn(f[p][2 * i], f[p][2 * i + 1]);
                        } else {
                            hi[i] = pack_f16x2_rn(f[p][2 * i], f[p][2 * i + 1]);
                            if (TERMS == 2) {
                                const __half2 h2 = *reinterpret_cast<__half2 *>(&hi[i]);
                                lo[i] = pack_f16x2_rn(f[p][2 * i] - __low2float(h2), f[p][2 * i + 1] - __high2float(h2));
                            }
                        }
                    }
                    sts128(qs + r * S::kQStride + 16 * x, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                    if (TERMS == 2)
                        sts128(qs + S::kBlock * S::kQStride + r * S::kQStride + 16 * x, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                    if (x == 0) row_factor[r] = factor;
                }
            }
        }
        compute_barrier();
        // A operand of 16 dims (k-step ks): for codes the dims in the order in which a
        // lane's 16 bytes of a token hold them.
        const auto load_q = [&](int term, int ks, uint32_t (&q)[4]) {
            const uint32_t at = qbase + term * (S::kBlock * S::kQStride) + (wm * 16 + g) * S::kQStride;
            if constexpr (KIND == kI8) {
                const uint32_t dim = (ks / 4) * kChunk + 16 * c + 4 * (ks % 4);
                const uint2 x = lds64(at + 2 * dim), y = lds64(at + 8 * S::kQStride + 2 * dim);
                q[0] = x.x, q[1] = y.x, q[2] = x.y, q[3] = y.y;
            } else {
                const uint32_t dim = 16 * ks + 2 * c;
                q[0] = lds32(at + 2 * dim);
                q[1] = lds32(at + 8 * S::kQStride + 2 * dim);
                q[2] = lds32(at + 2 * dim + 16);
                q[3] = lds32(at + 8 * S::kQStride + 2 * dim + 16);
            }
        };
        uint32_t qr[S::kQInRegs ? DP / 16 : 1][4];
        if constexpr (S::kQInRegs) {
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) load_q(0, ks, qr[ks]);
        }
        const float rf0 = row_factor[wm * 16 + g], rf1 = row_factor[wm * 16 + g + 8];
        int lo0, hi0, lo1, hi1, full_from, full_upto;
        {
            const int r0 = min(w.b * S::kBlock + wm * 16 + g, w.q.rows - 1), r1 = min(w.b * S::kBlock + wm * 16 + g + 8, w.q.rows - 1);
            row_range(a, w.q, r0, lo0, hi0);
            row_range(a, w.q, r1, lo1, hi1);
            int x;
            row_range(a, w.q, w.b * S::kBlock, x, full_upto);                                  // the first row's end
            row_range(a, w.q, min((w.b + 1) * S::kBlock, w.q.rows) - 1, full_from, x);         // the last row's start
        }
        float o[OT][4] = {};
        float m0 = neg_inf(), m1 = neg_inf(), l0 = 0.0f, l1 = 0.0f;
        int E0 = -118, E1 = -118;                           // value scales that the rows have seen are below 2^E
        for (int t = w.from; alive && t < w.upto; ++t) {
            if (!__all_sync(0xFFFFFFFFu, tile_wait(&full[stage], phase, a.wait_ns))) {
                if (lane == 0) {
                    *reinterpret_cast<volatile int *>(abort) = 1;
                    record_status(a.status, kErrTimeout);
                }
                alive = false;                              // (the warps still meet at the items' barriers)
                break;
            }
            const uint32_t kv = ring_at + stage * stage_bytes;
            const int t0 = (w.first + t) * kWarpTile + wn * S::kTokens;
            float s[NT][4] = {};
            float s2[TERMS == 2 ? NT : 1][4] = {};
#pragma unroll
            for (int ch = 0; ch < S::kMaxChunks; ++ch) {
                if (ch < chunks) {
                    const uint32_t kb = kv + ch * chunk_bytes + k_lane;
                    if constexpr (KIND == kI8) {
                        uint4 x[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) x[nt] = lds128_at(kb + off[nt / 2] + (nt & 1) * (8 * RB));
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            uint32_t q[4], q2[4];
                            if constexpr (!S::kQInRegs) load_q(0, ch * 4 + k4, q);
                            if constexpr (TERMS == 2) load_q(1, ch * 4 + k4, q2);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t b0, b1;
                                codes_f16(k4 == 0 ? x[nt].x : k4 == 1 ? x[nt].y : k4 == 2 ? x[nt].z : x[nt].w, b0, b1);
                                if constexpr (S::kQInRegs) mma16816<BF>(s[nt], qr[ch * 4 + k4], b0, b1);
                                else mma16816<BF>(s[nt], q, b0, b1);
                                if constexpr (TERMS == 2) mma16816<BF>(s2[nt], q2, b0, b1);
                            }
                        }
                    } else {
#pragma unroll
                        for (int p = 0; p < 2; ++p) {       // 32 dims
                            uint32_t q[2][4], q2[2][4], b[NT][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) ldsm4((kb ^ (64 * p)) + off[nt / 2] + (nt & 1) * (8 * RB), b[nt]);
                            if constexpr (!S::kQInRegs) load_q(0, ch * 4 + 2 * p, q[0]), load_q(0, ch * 4 + 2 * p + 1, q[1]);
                            if constexpr (TERMS == 2) load_q(1, ch * 4 + 2 * p, q2[0]), load_q(1, ch * 4 + 2 * p + 1, q2[1]);
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    if constexpr (S::kQInRegs) mma16816<BF>(s[nt], qr[ch * 4 + 2 * p + h], b[nt][2 * h], b[nt][2 * h + 1]);
                                    else mma16816<BF>(s[nt], q[h], b[nt][2 * h], b[nt][2 * h + 1]);
                                    if constexpr (TERMS == 2) mma16816<BF>(s2[nt], q2[h], b[nt][2 * h], b[nt][2 * h + 1]);
                                }
                        }
                    }
                }
            }
            // scores in powers of two
            float sv[KIND == kI8 ? NT : 1][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (TERMS == 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[nt][i] += s2[nt][i];
                }
                float f0 = rf0, f1 = rf0, f2v = rf1, f3 = rf1;
                if constexpr (KIND == kI8) {
                    const uint32_t at = kv + scale_off[nt / 2] + 4 * ((nt & 1) * 8 + 2 * c);
                    const uint2 k2 = lds64(at), v2 = lds64(at + 4 * together);
                    f0 *= __uint_as_float(k2.x), f1 *= __uint_as_float(k2.y);
                    f2v *= __uint_as_float(k2.x), f3 *= __uint_as_float(k2.y);
                    sv[nt][0] = __uint_as_float(v2.x), sv[nt][1] = __uint_as_float(v2.y);
                }
                s[nt][0] *= f0, s[nt][1] *= f1, s[nt][2] *= f2v, s[nt][3] *= f3;
            }
            float v0max = 0.0f, v1max = 0.0f;               // value scales that the rows see
            if (t0 + S::kTokens > full_upto || t0 < full_from) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int x = t0 + nt * 8 + 2 * c + i;
                        const bool sees0 = x >= lo0 && x < hi0, sees1 = x >= lo1 && x < hi1;
                        if (!sees0) s[nt][i] = neg_inf();
                        if (!sees1) s[nt][2 + i] = neg_inf();
                        if constexpr (KIND == kI8) {
                            if (!sees0 && !sees1) sv[nt][i] = 0.0f;   // (it may not be there)
                            if (sees0) v0max = fmaxf(v0max, sv[nt][i]);
                            if (sees1) v1max = fmaxf(v1max, sv[nt][i]);
                        }
                    }
                }
                const int begin = KIND != kI8 ? first_seen(a, w) : t0, end = w.hi;
                if (KIND != kI8 && (t0 < begin || t0 + S::kTokens > end)) {
                    // no values before the block's first token and past its last (each warp that
                    // reads them clears them: the others write the same)
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
#pragma unroll 1
                        for (int y = lane >> 3; y < 16; y += 4) {
                            const int x = t0 + 16 * i + y;
                            if (x >= begin && x < end) continue;
                            for (int ch = 0; ch < chunks; ++ch)
                                sts128(ring + stage * stage_bytes + v_at + ch * chunk_bytes + off[i] + y * RB + 16 * (lane & 7), make_uint4(0u, 0u, 0u, 0u));
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
            } else if constexpr (KIND == kI8) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) v0max = fmaxf(v0max, fmaxf(sv[nt][0], sv[nt][1]));
                v1max = v0max;
            }
            float x0 = neg_inf(), x1 = neg_inf();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                x0 = fmaxf(x0, fmaxf(s[nt][0], s[nt][1]));
                x1 = fmaxf(x1, fmaxf(s[nt][2], s[nt][3]));
            }
            const bool wide = KIND == kI8 && (v0max >= pow2(E0) || v1max >= pow2(E1));
            if (__any_sync(0xFFFFFFFFu, x0 > m0 + kSlack || x1 > m1 + kSlack || wide)) {
                x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 1));
                x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 1));
                x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, 2));
                x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, 2));
                const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
                float a0 = m0 == neg_inf() ? 0.0f : exp2_fast(m0 - n0), a1 = m1 == neg_inf() ? 0.0f : exp2_fast(m1 - n1);
                m0 = n0, m1 = n1;
                l0 *= a0, l1 *= a1;
                if constexpr (KIND == kI8) {
                    v0max = fmaxf(v0max, __shfl_xor_sync(0xFFFFFFFFu, v0max, 1));
                    v1max = fmaxf(v1max, __shfl_xor_sync(0xFFFFFFFFu, v1max, 1));
                    v0max = fmaxf(v0max, __shfl_xor_sync(0xFFFFFFFFu, v0max, 2));
                    v1max = fmaxf(v1max, __shfl_xor_sync(0xFFFFFFFFu, v1max, 2));
                    a0 *= raise(E0, v0max), a1 *= raise(E1, v1max);
                }
#pragma unroll
                for (int j = 0; j < OT; ++j) o[j][0] *= a0, o[j][1] *= a0, o[j][2] *= a1, o[j][3] *= a1;
            }
            const float u0 = m0 == neg_inf() ? 0.0f : m0 - kLift, u1 = m1 == neg_inf() ? 0.0f : m1 - kLift;
            const float down0 = KIND == kI8 ? pow2(-E0) : 1.0f, down1 = KIND == kI8 ? pow2(-E1) : 1.0f;
            uint32_t p[NG][4], p2[TERMS == 2 ? NG : 1][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float e[4] = {exp2_fast(s[nt][0] - u0), exp2_fast(s[nt][1] - u0), exp2_fast(s[nt][2] - u1), exp2_fast(s[nt][3] - u1)};
                l0 += e[0] + e[1], l1 += e[2] + e[3];
                if constexpr (KIND == kI8) {
                    // (below 1 where the row sees the token; finite times 0 where not)
                    e[0] *= fminf(sv[nt][0] * down0, 1.0f), e[1] *= fminf(sv[nt][1] * down0, 1.0f);
                    e[2] *= fminf(sv[nt][0] * down1, 1.0f), e[3] *= fminf(sv[nt][1] * down1, 1.0f);
                }
                const int at = 2 * (nt & 1);
                if constexpr (BF) {
                    p[nt / 2][at] = pack_bf16x2_rn(e[0], e[1]), p[nt / 2][at + 1] = pack_bf16x2_rn(e[2], e[3]);
                } else {
                    p[nt / 2][at] = pack_f16x2_rn(e[0], e[1]), p[nt / 2][at + 1] = pack_f16x2_rn(e[2], e[3]);
                    if constexpr (TERMS == 2) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const __half2 h2 = *reinterpret_cast<__half2 *>(&p[nt / 2][at + i]);
                            p2[nt / 2][at + i] = pack_f16x2_rn(e[2 * i] - __low2float(h2), e[2 * i + 1] - __high2float(h2));
                        }
                    }
                }
            }
            // sums of values
#pragma unroll
            for (int ch = 0; ch < S::kMaxChunks; ++ch) {
                if (ch < chunks) {
                    const uint32_t vb = kv + ch * chunk_bytes + v_lane;
                    if constexpr (KIND == kI8) {
                        // eight dims of a lane (8 g ..), as the n of eight column tiles
                        float fresh[TERMS == 2 ? 8 : 1][4] = {};
#pragma unroll
                        for (int k = 0; k < NG; ++k) {
                            uint2 x[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i] = lds64(vb + off[k] + RB * ((i & 1) + 8 * (i >> 1)));
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[i].x ^= 0x80808080u, x[i].y ^= 0x80808080u;
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t sel = 0x40u + 0x11u * (j & 3);   // byte j of the first token, of the second
                                const uint32_t t01 = __byte_perm(j < 4 ? x[0].x : x[0].y, j < 4 ? x[1].x : x[1].y, sel);
                                const uint32_t t23 = __byte_perm(j < 4 ? x[2].x : x[2].y, j < 4 ? x[3].x : x[3].y, sel);
                                const uint32_t b0 = hsub2_bits(__byte_perm(t01, 0x64646464u, 0x4140), 0x64806480u);
                                const uint32_t b1 = hsub2_bits(__byte_perm(t23, 0x64646464u, 0x4140), 0x64806480u);
                                if constexpr (TERMS == 2) {
                                    mma16816<BF>(fresh[j], p[k], b0, b1);
                                    mma16816<BF>(fresh[j], p2[k], b0, b1);
                                } else {
                                    mma16816<BF>(o[ch * 8 + j], p[k], b0, b1);
                                }
                            }
                        }
                        if constexpr (TERMS == 2) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) o[ch * 8 + j][i] += fresh[j][i];
                        }
                    } else if constexpr (TERMS == 2) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {       // 16 dims
                            float fresh[2][4] = {};
#pragma unroll
                            for (int k = 0; k < NG; ++k) {
                                uint32_t b[4];
                                ldsm4_t((vb ^ (32 * j)) + off[k], b);
                                mma16816<BF>(fresh[0], p[k], b[0], b[1]);
                                mma16816<BF>(fresh[1], p[k], b[2], b[3]);
                                mma16816<BF>(fresh[0], p2[k], b[0], b[1]);
                                mma16816<BF>(fresh[1], p2[k], b[2], b[3]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[ch * 8 + 2 * j][i] += fresh[0][i];
                                o[ch * 8 + 2 * j + 1][i] += fresh[1][i];
                            }
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < NG; ++k) {
                            uint32_t b[4][4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) ldsm4_t((vb ^ (32 * j)) + off[k], b[j]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                mma16816<BF>(o[ch * 8 + 2 * j], p[k], b[j][0], b[j][1]);
                                mma16816<BF>(o[ch * 8 + 2 * j + 1], p[k], b[j][2], b[j][3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
            if (++stage == a.stages) stage = 0, phase ^= 1u;
        }
        // ------------------------------------------------- the item's end
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1), l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
        l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2), l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);
        // the warps of a row slice come to one maximum, then add up
        float f0 = KIND == kI8 ? pow2(E0) : 1.0f, f1 = KIND == kI8 ? pow2(E1) : 1.0f;
        if constexpr (WN > 1) {
            if (c == 0) {
                red_ml[warp * 16 + g] = make_float2(m0, l0);
                red_ml[warp * 16 + g + 8] = make_float2(m1, l1);
            }
            compute_barrier();
            float n0 = neg_inf(), n1 = neg_inf();
            float2 y0[WN], y1[WN];
#pragma unroll
            for (int i = 0; i < WN; ++i) {
                y0[i] = red_ml[(wm * WN + i) * 16 + g], y1[i] = red_ml[(wm * WN + i) * 16 + g + 8];
                n0 = fmaxf(n0, y0[i].x), n1 = fmaxf(n1, y1[i].x);
            }
            l0 = 0.0f, l1 = 0.0f;
#pragma unroll
            for (int i = 0; i < WN; ++i) {
                l0 += y0[i].y * (y0[i].x == neg_inf() ? 1.0f : exp2_fast(y0[i].x - n0));
                l1 += y1[i].y * (y1[i].x == neg_inf() ? 1.0f : exp2_fast(y1[i].x - n1));
            }
            f0 *= m0 == neg_inf() ? 1.0f : exp2_fast(m0 - n0);
            f1 *= m1 == neg_inf() ? 1.0f : exp2_fast(m1 - n1);
            m0 = n0, m1 = n1;
        }
        const bool whole = w.whole();
        if (whole) f0 *= l0 == 0.0f ? 0.0f : 1.0f / l0, f1 *= l1 == 0.0f ? 0.0f : 1.0f / l1;
#pragma unroll
        for (int j = 0; j < OT; ++j) o[j][0] *= f0, o[j][1] *= f0, o[j][2] *= f1, o[j][3] *= f1;
        if constexpr (WN > 1) {
            // every warp's sums to the first of its row slice, which adds them in order
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                constexpr int kHalf = OT / 2;
                float *buf = red + wm * (WN - 1) * (16 * DP / 2);
                if (wn > 0) {
#pragma unroll
                    for (int j = 0; j < kHalf; ++j) {
                        const float(&x)[4] = o[part * kHalf + j];
                        *reinterpret_cast<float4 *>(buf + (wn - 1) * (16 * DP / 2) + (j * 32 + lane) * 4) = make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
                compute_barrier();
                if (wn == 0) {
#pragma unroll
                    for (int i = 0; i < WN - 1; ++i)
#pragma unroll
                        for (int j = 0; j < kHalf; ++j) {
                            const float4 x = *reinterpret_cast<const float4 *>(buf + i * (16 * DP / 2) + (j * 32 + lane) * 4);
                            float(&y)[4] = o[part * kHalf + j];
                            y[0] += x.x, y[1] += x.y, y[2] += x.z, y[3] += x.w;
                        }
                }
                if (part == 0) compute_barrier();
            }
        }
        if (wn == 0) {
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.from == 0 ? 1 : 0);
            float *part = a.parts + slot * attn_part_floats(S::kBlock, chunks);
            const int width = kChunk * chunks;
#pragma unroll
            for (int up = 0; up < 2; ++up) {
                const int r = wm * 16 + g + 8 * up, row = w.b * S::kBlock + r;
                if (row >= w.q.rows) continue;
                const int i = row / a.group, head = w.h * a.group + row - i * a.group;
                const int64_t out = (static_cast<int64_t>(w.q.start) + i) * a.ldo + static_cast<int64_t>(head) * a.c.d;
                if constexpr (KIND == kI8) {
                    // a lane has dims 8 (2 c + x) .. + 7 of a chunk
#pragma unroll
                    for (int ch = 0; ch < S::kMaxChunks; ++ch) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int dim = ch * kChunk + 8 * (2 * c + x);
                            float v[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[j] = o[ch * 8 + j][2 * up + x];
                            if (ch < chunks) {
                                if (!whole) {
                                    float4 *dst = reinterpret_cast<float4 *>(part + r * width + dim);
                                    dst[0] = make_float4(v[0], v[1], v[2], v[3]), dst[1] = make_float4(v[4], v[5], v[6], v[7]);
                                } else if (dim < a.c.d) {
                                    store8_out(a, out + dim, v);
                                }
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < OT; ++j) {
                        const int dim = 8 * j + 2 * c;
                        const float v0 = o[j][2 * up], v1 = o[j][2 * up + 1];
                        if (j / 8 < chunks) {
                            if (!whole) *reinterpret_cast<float2 *>(part + r * width + dim) = make_float2(v0, v1);
                            else if (dim < a.c.d) store2_out(a, out + dim, v0, v1);
                        }
                    }
                }
                if (!whole && c == 0) {
                    part[S::kBlock * width + r] = up ? m1 : m0;
                    part[S::kBlock * width + S::kBlock + r] = up ? l1 : l0;
                }
            }
            if (!whole && w.from == 0 && lane == 0 && wm == 0) put_meta(a, w);
        }
    }
}

template <int KIND, int TERMS, int WM, int DP> cudaError_t launch_shape(AttnArgs a, int sm_count, cudaStream_t s, int *ctas)
{
    using S = WarpShape<KIND, TERMS, WM, DP>;
    const int stage = warp_stage_bytes(a.c.chunks, a.c.type);
    // several CTAs an SM where rings of two tiles fit: their waits cover each other
    int per_sm = S::kPerSM;
    const auto stages = [&] { return ((per_sm > 1 ? static_cast<int>(kSmemPerSM) / per_sm - 1024 : static_cast<int>(kSmemOptIn)) - S::kFixed) / stage; };
    while (per_sm > 1 && stages() < 2) --per_sm;
    a.stages = std::min(8, stages());
    const size_t smem = S::kFixed + static_cast<size_t>(a.stages) * stage;
    const void *f = reinterpret_cast<const void *>(&attn_warp_kernel<KIND, TERMS, WM, DP>);
    cudaError_t e = set_max_smem(f, kSmemOptIn);
    if (e != cudaSuccess) return e;
    *ctas = std::min(kAttnMaxCtas, per_sm * sm_count);
    void *args[] = {&a};
    return launch_pdl(f, dim3(static_cast<unsigned>(*ctas)), dim3(kAttnThreads), smem, s, args);
}
template <int KIND, int TERMS> cudaError_t launch_kind(const AttnArgs &a, int sm_count, cudaStream_t s, int *ctas)
{
    const int dp = a.c.chunks <= 2 ? a.c.chunks * kChunk : 256;
#define Q4_SHAPE(wm) (dp == 64 ? launch_shape<KIND, TERMS, wm, 64>(a, sm_count, s, ctas) \
                      : dp == 128 ? launch_shape<KIND, TERMS, wm, 128>(a, sm_count, s, ctas) : launch_shape<KIND, TERMS, wm, 256>(a, sm_count, s, ctas))
    return a.block == 16 ? Q4_SHAPE(1) : a.block == 32 ? Q4_SHAPE(2) : Q4_SHAPE(4);
#undef Q4_SHAPE
}

} // namespace
} // namespace q4
