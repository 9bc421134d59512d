// q4mm_attn_tensor.cu -- attention of many query rows over the paged cache, on
// the 5th-generation tensor cores, for 16-bit queries and heads of up to 128 dims.
//
// A CTA takes 256 query rows of a sequence and cached head (an item), as two
// halves of 128, and walks over tiles of 128 tokens:
//     S = Q K^T      operands in shared memory, S in tensor memory (128 columns)
//     P = 2^(S - m)  a thread a row, out of and back into tensor memory, as 16-bit
//                    numbers in the place of S
//     O += P V       P from tensor memory, V from shared memory, O in tensor memory
// While one half's scores are turned into terms the other half's products run:
// products of a tile of both halves take 4 x 512 clocks, a half's softmax has 1024
// of them. The maximum m is raised, and O scaled, only where a row's scores pass it
// by 2^8; the softmax threads scale O themselves (S of a tile is committed after
// the products of the tile before, so O rests).
//   Warps: 0-3 and 4-7 the halves' softmax (a row a thread: no shuffles), 8 issues the
// products, 9 copies. Over codes 8-11 turn them into fp16 tiles and 12 issues; where the
// scales go, Bounds says.
//   What bounds it (clocks of a tile of 128 tokens, both halves): the products' 2048 and
// what the waits between them add. A test of a barrier that is already there answers
// after some 190 while products read shared memory, and the queue of products holds
// about three of 64: a loop takes 3300. 2048 new tokens over 16384, 32 heads on 8 of
// 128: 418 us, 1230 TFLOP/s (64 % of the measured bf16 rate); over codes the converting
// warps' 3000 a tile of K or V bound it (540 over 8100: 153 us; 140 to 148 bytes a thread
// are spilled); short items (prompts of up to 2000, a window of 1024, 64 dims: 63 us) their
// start and end, 8000 to 10000 an item. Tried and
// slower: two issuing warps (the halves fall into step), 16 softmax warps with half a
// row each, scores held in registers between the maximum and the terms (spills), eight
// converting warps, four for keys and four for values (150 to 188 us by the registers'
// split: what the ninth to sixteenth warp gain, spills lose).
//   K and V lie in the pages as the tensor cores read them, 64 dims a row of 128
// bytes, swizzled: K as a K-major operand, V (dims contiguous) as an N-major one.
//   Places before a block's first visible token and past its last are never copied: what
// is in their place may be another sequence's, of a page that was never written at
// that, so their values are set to 0 beside the copies of a tile that has some.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "q4mm_attn.cuh"

namespace q4 {
namespace {

constexpr int kHalf = 128, kTile = kTensorTile;
constexpr int kSoftmaxWarps = 8;                        // four a half
constexpr uint32_t kFirst = 1, kLast = 2, kTwo = 4, kEnd = 8;   // of a tile: where it stands in its item, whether that has a second half, and no tile comes after it
constexpr uint32_t kAtomRows = kTile * 128;              // bytes of 64 dims of a tile

template <int KIND, int DP> struct TensorShape {
    static constexpr bool kCodes = KIND == 2;
    static constexpr int kChunks = DP / kChunk;
    // Warps 8 and 9: products and copies; codes: 8-11 convert, 12 products, and the
    // warpgroups share the registers out.
    static constexpr int kThreads = kCodes ? 512 : 320;
    static constexpr int kConvertWarp0 = 8, kMmaWarp = kCodes ? 12 : 8, kCopyWarp = 9;
    static constexpr int kLaunchRegs = 128, kSoftmaxRegs = 144, kConvertRegs = 128, kMmaRegs = 96;   // codes (kLaunchRegs: build.py checks it)
    static constexpr int kTileBytes = kChunks * static_cast<int>(kAtomRows);
    // 16-bit: rings of K and of V tiles. Codes: one ring of fp16 tiles, K and V in turn.
    static constexpr int kK = kCodes || DP == 64 ? 4 : 2, kV = kCodes ? 0 : DP == 64 ? 4 : 3;
    static constexpr int kScaleSlots = 4;                // tiles whose scales are held
    static constexpr size_t kSmem = 2 * kHalf * DP * 2 + static_cast<size_t>(kK + kV) * kTileBytes +
                                    (kCodes ? kScaleSlots * (2 * kTile + 4) * 4 + 4 * kTile * 4 : 0) + 2 * kHalf * 4 + 512 + 1024;
};

struct Bars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], scales_full[4], scales_empty[4];
    uint64_t q_full[2], s_full[2], p_full[2][2], done;
    uint32_t flags[4];                                   // of the K tile in each slot
    uint32_t tmem;
    int abort;
};

// Waits with one outcome for the warp. A suspended wait (try_wait) resumes some 170
// ns late, a third of a half's softmax; tests without a pause take shared memory's
// time from the products' operands. NAP: nanoseconds between two tests.
template <int NAP> __device__ __forceinline__ bool spin_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        for (int i = 0; i < 16; ++i) {
            if (NAP > 0) __nanosleep(NAP);
            if (mbar_test_wait(bar, parity)) return true;
        }
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}
template <int NAP = 40> __device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, spin_wait<NAP>(bar, parity, limit_ns)) != 0;
}

struct Turn {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int depth)
    {
        if (++slot == depth) slot = 0, phase ^= 1u;
    }
};

// Over codes: whether a tile's scales are applied by columns, to scores and terms,
// exactly. They are for fp16 queries, and where some row of the block does not see
// all of the tile. For bf16 outputs the operands of other tiles carry them, rounded to
// fp16 (2^-12, far below the output's 2^-9) next to a power of two a tile: reading 256
// scales a row and tile from shared memory, which the products' operands keep busy,
// took the softmax 7000 clocks of a tile's 2048 (540 tokens over 8100: 205 us).
struct Bounds {
    int begin = 0, from = 0, upto = 0;   // (begin: first_seen())
    __device__ __forceinline__ Bounds() {}
    __device__ __forceinline__ Bounds(const AttnArgs &a, const Walk &w)
    {
        int x;
        row_range(a, w.q, w.b * a.block, begin, upto);
        row_range(a, w.q, min((w.b + 1) * a.block, w.q.rows) - 1, from, x);
    }
    __device__ __forceinline__ bool exact(const AttnArgs &a, int t0) const { return a.type != Q4_TYPE_BF16 || t0 + kTile > upto || t0 < from; }
};
// Descriptor of an N-major operand of 64-element rows of 128 bytes, swizzled: the
// next 64 of N `lead` bytes on, the next 8 of K 1024.
__device__ __forceinline__ uint64_t desc_n_major(uint32_t saddr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
constexpr uint32_t kNMajorB = 1u << 16;

// A warpgroup's registers a thread from FROM, the launch's, to TO.
template <int FROM, int TO> __device__ __forceinline__ void set_regs()
{
    if constexpr (TO > FROM) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(TO));
    else if constexpr (TO < FROM) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(TO));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// KIND: 0 fp16, 1 bf16, 2 codes (operands fp16).
template <int KIND, int DP>
__global__ void __launch_bounds__(TensorShape<KIND, DP>::kThreads, 1) attn_tensor_kernel(const AttnArgs a)
{
    using S = TensorShape<KIND, DP>;
    constexpr bool BF = KIND == 1, CODES = S::kCodes;
    constexpr int CH = S::kChunks;
    extern __shared__ uint8_t smem[];
    uint8_t *const qs = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));                                          // [half][chunk][128 rows][128 bytes]
    uint8_t *const ks = qs + 2 * kHalf * DP * 2;
    uint8_t *const vs = ks + S::kK * S::kTileBytes;
    float *const scales = reinterpret_cast<float *>(vs + S::kV * S::kTileBytes);   // [slot][keys, values][tile], then [slot][4]: the largest value scale, the exponents
    uint32_t *const factors = reinterpret_cast<uint32_t *>(scales + (CODES ? S::kScaleSlots * (2 * kTile + 4) : 0));   // [converting warp][token]
    float *const row_factor = reinterpret_cast<float *>(factors + (CODES ? 4 * kTile : 0));
    Bars *const bars = reinterpret_cast<Bars *>(row_factor + 2 * kHalf);
    // (a warp's number from one lane: what follows from it stays in uniform registers)
    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    static_assert(sizeof(Bars) <= 512, "barriers");
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bars->k_full[i], CODES ? 4 : 1);
            mbar_init(&bars->k_empty[i], 1);
            mbar_init(&bars->v_full[i], 1);
            mbar_init(&bars->v_empty[i], 1);
            mbar_init(&bars->scales_full[i], 4);
            mbar_init(&bars->scales_empty[i], kSoftmaxWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->q_full[i], 4);
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->p_full[i][0], 4);
            mbar_init(&bars->p_full[i][1], 4);
        }
        mbar_init(&bars->done, 1);
        bars->abort = 0;
        fence_barrier_init();
    }
    if (warp == S::kMmaWarp) {
        tmem_alloc(&bars->tmem, 512u);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    Walk w;
    w.begin(a, reinterpret_cast<long long *>(qs));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) a.meta[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    const uint32_t tmem = bars->tmem;
    const auto aborted = [&] { return *reinterpret_cast<volatile int *>(&bars->abort) != 0; };
    const auto fail = [&] {
        *reinterpret_cast<volatile int *>(&bars->abort) = 1;
        record_status(a.status, kErrTimeout);
    };
    const auto both = [&] { return w.q.rows - w.b * kTensorRows > kHalf; };   // whether the item has a second half

    if (warp < kSoftmaxWarps) {
        // ---------------------------------------------------------- softmax
        if constexpr (CODES) set_regs<S::kLaunchRegs, S::kSoftmaxRegs>();
        const int half = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + 128u * half, o_at = tmem + lanes + 256u + 128u * half;
        const int r_in = half * kHalf + (warp & 3) * 32 + lane;        // the thread's row in the block
        uint32_t s_phase = 0;
        Turn sc;                                                       // the tile's scales
        bool ok = true;
        for (; ok && w.valid(); w.next(a)) {
            if (half && !both()) {
                // the half is not there: it gives the scales back as they come
                for (int t = w.from; CODES && ok && t < w.upto; ++t) {
                    ok = warp_wait(&bars->scales_full[sc.slot], sc.phase, a.wait_ns);
                    if (ok && lane == 0) mbar_arrive(&bars->scales_empty[sc.slot]);
                    sc.step(S::kScaleSlots);
                }
                if (!ok) fail();
                continue;
            }
            const int first_row = w.b * kTensorRows + half * kHalf + (warp & 3) * 32;
            // the warp's 32 rows of Q, two or four an access, eight accesses in flight, into
            // the operand's image
            constexpr int kLanes = DP / 8, kRows = 32 / kLanes, kBatch = 8;
            const int x = lane % kLanes;
#pragma unroll 1
            for (int r0 = lane / kLanes; r0 < 32; r0 += kBatch * kRows) {
                uint32_t raw[kBatch][4];
                const auto fetch = [&](auto vec) {
#pragma unroll
                    for (int p = 0; p < kBatch; ++p) {
                        const int row = first_row + r0 + p * kRows;
#pragma unroll
                        for (int i = 0; i < 4; ++i) raw[p][i] = 0u;
                        if (row < w.q.rows && 8 * x < a.c.d) {
                            const int i = row / a.group, head = w.h * a.group + row - i * a.group;
                            load_raw<decltype(vec)::value>(a.Q, (static_cast<int64_t>(w.q.start) + i) * a.ldq + static_cast<int64_t>(head) * a.c.d + 8 * x, raw[p]);
                        }
                    }
                };
                if (a.vec) fetch(std::true_type{});
                else fetch(std::false_type{});
#pragma unroll
                for (int p = 0; p < kBatch; ++p) {
                    const int r = (warp & 3) * 32 + r0 + p * kRows;
                    if constexpr (CODES) {
                        // to fp16's range by a power of two: the largest in 2^12 .. 2^13
                        float f[8];
                        uint32_t mb = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t u = raw[p][i / 2] >> (16 * (i & 1));
                            f[i] = a.type == Q4_TYPE_BF16 ? __uint_as_float(u << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
                            mb = max(mb, abs_bits(f[i]));
                        }
#pragma unroll
                        for (int o = kLanes / 2; o > 0; o /= 2) mb = max(mb, __shfl_xor_sync(0xFFFFFFFFu, mb, o));
                        float factor = a.scale_log2, up = 1.0f;
                        if (mb >= 0x7F800000u) {
                            factor = __uint_as_float(0x7FC00000u);
                        } else if (mb != 0u) {
                            const int e = min(max(139 - static_cast<int>(mb >> 23), -126), 126);
                            up = pow2(e);
                            factor *= pow2(-e);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) raw[p][i] = mb >= 0x7F800000u ? 0u : pack_f16x2_rn(f[2 * i] * up, f[2 * i + 1] * up);
                        if (x == 0) row_factor[half * kHalf + r] = factor;
                    }
                    sts128(qs + (half * CH + x / 8) * kAtomRows + r * 128 + (((x & 7) ^ (r & 7)) << 4), make_uint4(raw[p][0], raw[p][1], raw[p][2], raw[p][3]));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full[half]);
            const int my_row = first_row + lane;
            float rf = CODES ? row_factor[half * kHalf + (warp & 3) * 32 + lane] : a.scale_log2;
            int lo, hi, full_from, full_upto, other;
            row_range(a, w.q, min(my_row, w.q.rows - 1), lo, hi);
            row_range(a, w.q, min(first_row, w.q.rows - 1), other, full_upto);
            row_range(a, w.q, min(first_row + 31, w.q.rows - 1), full_from, other);
            // A column that a row does not see has a score of -infinity, and is multiplied by the row's
            // factor: not by 0, and where the row sees nothing not by that of a query that is not finite.
            if (CODES && (rf == 0.0f || lo >= hi)) rf = 1.401298464324817e-45f;
            float m = neg_inf(), l = 0.0f;
            int E = -118;                                              // of the sums' unit, over codes
            const Bounds bounds(a, w);
            for (int t = w.from; t < w.upto; ++t) {
                const int t0 = (w.first + t) * kTile;
                if (!warp_wait(&bars->s_full[half], s_phase, a.wait_ns) ||
                    (CODES && !warp_wait(&bars->scales_full[sc.slot], sc.phase, a.wait_ns))) {
                    fail();
                    ok = false;
                    break;
                }
                s_phase ^= 1u;
                tc_fence_after();
                const float *sk = scales + sc.slot * (2 * kTile), *sv = sk + kTile;
                const bool masked = t0 + kTile > full_upto || t0 < full_from;   // some row does not see all of the tile
                // Scales by columns; or in the operands already, but for two powers of two. (The
                // two are apart, and loops over codes are not unrolled: the warps' code together
                // has to stay in the instruction caches.)
                const auto tile = [&](auto by_column) {
                constexpr bool exact = decltype(by_column)::value;     // (only such a tile is not seen whole)
                const bool hidden = (!CODES || exact) && masked;
                const float4 tail = CODES ? *reinterpret_cast<const float4 *>(scales + S::kScaleSlots * 2 * kTile + sc.slot * 4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const float rft = CODES && !exact ? rf * pow2(__float_as_int(tail.y)) : rf;
                // 32 columns of scores: their keys' scales, and what the row does not see
                const auto scored = [&](int i0, uint32_t *r) {
                    if constexpr (exact) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(sk + i0 + i);
                            const float s4[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) r[i + j] = __float_as_uint(__uint_as_float(r[i + j]) * s4[j]);
                        }
                    }
                    if (hidden) {
                        // bits of the columns that the row sees
                        const int from = min(max(lo - t0 - i0, 0), 32), upto = min(max(hi - t0 - i0, 0), 32);
                        const uint32_t sees = static_cast<uint32_t>(((1ull << upto) - 1ull) & ~((1ull << from) - 1ull));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(sees >> i & 1u)) r[i] = 0xFF800000u;
                    }
                };
                float mx[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
                const auto largest = [&](const uint32_t *r) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], fmaxf(__uint_as_float(r[i + 2 * j]), __uint_as_float(r[i + 2 * j + 1])));
                };
                // The scores are read twice, 32 columns at a time: held in registers (208 a softmax
                // thread, of the other warps') they took longer, by what the others then spilled.
                uint32_t r[64];
                tmem_ld_32x32b_x32(s_at, r);
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    tmem_wait_ld();
                    tmem_ld_32x32b_x32(s_at + 32 * c + 32, r + 32);
                    scored(32 * c, r);
                    largest(r);
                    tmem_wait_ld();
                    // the next columns, and after the last ones the first again
                    tmem_ld_32x32b_x32(s_at + (32 * c + 64) % kTile, r);
                    scored(32 * c + 32, r + 32);
                    largest(r + 32);
                }
                tmem_wait_ld();
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * rft;
                float vmax = tail.x;                                   // value scales that the row sees are at most this
                if (CODES && hidden) {
                    vmax = 0.0f;
#pragma unroll 1
                    for (int i = max(lo - t0, 0); i < min(hi - t0, kTile); ++i) vmax = fmaxf(vmax, sv[i]);
                }
                const bool wide = CODES && vmax >= pow2(E);
                if (__any_sync(0xFFFFFFFFu, top > m + kSlack || wide)) {
                    const float n = fmaxf(m, top);
                    float scale = m == neg_inf() ? 0.0f : exp2_fast(m - n);
                    m = n;
                    l *= scale;
                    if (wide) {
                        const int to = min(((__float_as_int(vmax) >> 23) & 255) - 126, 126);
                        scale *= to - E > 126 ? 0.0f : pow2(E - to);
                        E = to;
                    }
                    if (t > w.from) {
#pragma unroll 1
                        for (int i = 0; i < DP; i += 16) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_at + i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * scale);
                            tmem_st_32x32b_x16(o_at + i, o);
                        }
                    }
                }
                // terms in the sums' unit: of a tile whose values carry their scales 2^shift times p.
                // Below 2^-40 they are 0 in fp16 (terms are below 2^15, its smallest step is 2^-24), so a
                // smaller shift changes no product; but the denominator adds them up before that
                // rounding, and fp32 still holds them down to 2^-93 of the largest.
                const int shift = CODES && !exact ? max(__float_as_int(tail.z) - E, -40) : 0;
                const float u = (m == neg_inf() ? 0.0f : m - kLift) - static_cast<float>(shift);
                const F2 rf2 = f2(rft, rft), u2 = f2(-u, -u);
                [[maybe_unused]] const float down = CODES ? pow2(-E) : 1.0f;
                F2 sum = f2(0.0f, 0.0f), sum2 = sum;
                // 32 columns' terms into the 16 words at p, which may be r's own
                const auto terms = [&](auto columns, int i0, const uint32_t *r, uint32_t *p) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float e0, e1;
                        f2_split(f2_fma(f2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), rf2, u2), e0, e1);
                        e0 = exp2_fast(e0), e1 = exp2_fast(e1);
                        if (i & 1) sum2 = f2_add(sum2, f2(e0, e1));
                        else sum = f2_add(sum, f2(e0, e1));
                        if constexpr (decltype(columns)::value) {
                            // (below 1 where the row sees the token; finite times 0 where not)
                            const float2 v2 = *reinterpret_cast<const float2 *>(sv + i0 + 2 * i);
                            e0 *= fminf(v2.x * down, 1.0f), e1 *= fminf(v2.y * down, 1.0f);
                        }
                        p[i] = BF ? pack_bf16x2_rn(e0, e1) : pack_f16x2_rn(e0, e1);
                    }
                };
                // they go in the place of scores, in two parts: products start on the first
                const auto part_done = [&](int h) {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->p_full[half][h]);
                };
#pragma unroll 1
                for (int c = 0; c < 4; c += 2) {
                    uint32_t p[16];
                    // (terms of some columns take places that have been read)
                    tmem_ld_32x32b_x32(s_at + 32 * c + 32, r + 32);
                    scored(32 * c, r);
                    terms(by_column, 32 * c, r, p);
                    tmem_st_32x32b_x16(s_at + 16 * c, p);
                    tmem_wait_ld();
                    if (c == 0) tmem_ld_32x32b_x32(s_at + 64, r);
                    scored(32 * c + 32, r + 32);
                    terms(by_column, 32 * c + 32, r + 32, p);
                    tmem_st_32x32b_x16(s_at + 16 * c + 16, p);
                    if (c == 0) tmem_wait_ld();
                    part_done(c / 2);
                }
                l += f2_sum(f2_add(sum, sum2)) * (CODES ? pow2(-shift) : 1.0f);
                };
                if constexpr (CODES) {
                    if (bounds.exact(a, t0)) tile(std::true_type{});
                    else tile(std::false_type{});
                } else {
                    tile(std::false_type{});
                }
                if constexpr (CODES) {
                    if (lane == 0) mbar_arrive(&bars->scales_empty[sc.slot]);
                    sc.step(S::kScaleSlots);
                }
            }
            if (!ok) break;
            // ------------------------------------------------ the item's end
            if (!warp_wait(&bars->s_full[half], s_phase, a.wait_ns)) {
                fail();
                ok = false;
                break;
            }
            s_phase ^= 1u;
            tc_fence_after();
            const bool whole = w.whole();
            const int slot = 2 * static_cast<int>(blockIdx.x) + (w.from == 0 ? 1 : 0);
            float *part = a.parts + slot * attn_part_floats(kTensorRows, CH);
            const float back = CODES ? pow2(E) : 1.0f;
            const float mul = whole ? (l == 0.0f ? 0.0f : back / l) : back;
            const int i = my_row / a.group, head = w.h * a.group + my_row - i * a.group;
            const int64_t out = (static_cast<int64_t>(w.q.start) + i) * a.ldo + static_cast<int64_t>(head) * a.c.d;
            if (whole && !a.vec) {
#pragma unroll 1
                for (int c0 = 0; c0 < DP; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld_32x32b_x16(o_at + c0, o);
                    tmem_wait_ld();
                    if (my_row < w.q.rows) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
                            if (c0 + j < a.c.d) store2_out(a, out + c0 + j, __uint_as_float(o[j]) * mul, __uint_as_float(o[j + 1]) * mul);
                    }
                    __syncwarp();
                }
            } else {
                // 128 bytes of each of the warp's rows at a time, through the place of its
                // rows of Q, so that a row's bytes leave together (a thread's 16 bytes by
                // themselves made an item's end 16 us)
                uint8_t *const stage = qs + half * CH * kAtomRows + (warp & 3) * 4096;
                const bool bf = a.type == Q4_TYPE_BF16;
                const int left = w.q.rows - first_row;                 // rows of the warp that exist
#pragma unroll 1
                for (int c0 = 0; c0 < DP; c0 += whole ? 64 : 32) {
                    uint32_t u[32];
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(o_at + c0 + 32 * i, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const float y0 = __uint_as_float(o[2 * j]) * mul, y1 = __uint_as_float(o[2 * j + 1]) * mul;
                                u[16 * i + j] = bf ? pack_bf16x2_rn(y0, y1) : pack_f16x2_rn(y0, y1);
                            }
                        }
                    } else {
                        tmem_ld_32x32b_x32(o_at + c0, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * mul);
                    }
                    __syncwarp();                                      // what was staged before is out
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sts128(stage + lane * 128 + ((i ^ (lane & 7)) << 4), make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]));
                    __syncwarp();
                    const int unit = lane & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = 4 * i + (lane >> 3);
                        const uint4 v = lds128(stage + row * 128 + ((unit ^ (row & 7)) << 4));
                        const long long to = __shfl_sync(0xFFFFFFFFu, static_cast<long long>(out), row);
                        if (row < left) {
                            if (!whole) *reinterpret_cast<uint4 *>(part + (half * kHalf + (warp & 3) * 32 + row) * DP + c0 + 4 * unit) = v;
                            else if (c0 + 8 * unit < a.c.d) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.O) + to + c0 + 8 * unit) = v;
                        }
                    }
                }
                __syncwarp();
            }
            if (!whole && my_row < w.q.rows) {
                part[kTensorRows * DP + r_in] = m;
                part[kTensorRows * DP + kTensorRows + r_in] = l;
            }
            if (!whole && w.from == 0 && tid == 0) put_meta(a, w);
            tc_fence_before();
        }
    } else if (warp >= (CODES ? S::kMmaWarp : 8)) {
        if constexpr (CODES) set_regs<S::kLaunchRegs, S::kMmaRegs>();
        if (warp == S::kMmaWarp) {
            // ----------------------------------------------------- products
            constexpr uint32_t type = BF ? idesc_bf16_f32(0, 0) : idesc_f16_f32(0, 0);
            constexpr uint32_t id_s = type | idesc_f16_f32(kHalf, kTile), id_o = type | idesc_f16_f32(kHalf, DP) | kNMajorB;
            const uint32_t d = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint64_t q0 = smem_desc_sw128(smem_u32(qs)), k0 = smem_desc_sw128(smem_u32(ks));
            const uint64_t v0 = desc_n_major(smem_u32(CODES ? ks : vs), kAtomRows);
            uint64_t *const v_full = CODES ? bars->k_full : bars->v_full, *const v_empty = CODES ? bars->k_empty : bars->v_empty;
            Turn kt, vt;                                               // K and V tiles in turn
            if (CODES) vt.step(S::kK);                                 // ... of one ring
            uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            const auto wait = [&](uint64_t *bar, uint32_t phase) {
                if (ok && !warp_wait<0>(bar, phase, a.wait_ns)) {
                    fail();
                    ok = false;
                }
                return ok;
            };
            // The MMA queue holds some 170 clocks of work, less than a wait and what follows
            // it take: what the next group waits for is tested in the middle of a group, and
            // waited for after it only if it was not there.
            bool there = false;
            const auto test = [&](uint64_t *bar, uint32_t phase) { return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, phase)) != 0; };
            const auto wait_unless = [&](uint64_t *bar, uint32_t phase) { return there || wait(bar, phase); };
            const auto scores = [&](int half, bool last_use, auto next) {   // of the K tile in turn
                const uint64_t kd = k0 + static_cast<uint64_t>(static_cast<uint32_t>(kt.slot) * (S::kTileBytes >> 4));
                const uint64_t qd = q0 + static_cast<uint64_t>(half * CH * (kAtomRows >> 4));
                uint64_t *const freed = &bars->k_empty[kt.slot];
                constexpr int kSteps = CH * 4;
                tc_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (elect_one()) {
#pragma unroll
                        for (int i = part * kSteps / 2; i < (part + 1) * kSteps / 2; ++i)
                            tc_mma_f16(d + 128u * half, qd + i / 4 * (kAtomRows >> 4) + 2 * (i % 4), kd + i / 4 * (kAtomRows >> 4) + 2 * (i % 4), id_s,
                                       i > 0 ? 1u : 0u);
                        if (part == 1) {
                            tc_commit(&bars->s_full[half]);
                            if (last_use) tc_commit(freed);
                        }
                    }
                    __syncwarp();
                    if (part == 0) there = next();
                }
                if (last_use) {
                    kt.step(S::kK);
                    if (CODES) kt.step(S::kK);
                }
            };
            const auto sums = [&](int half, bool add, bool last, bool last_use, auto next) {   // with the V tile in turn
                const uint64_t vd = v0 + static_cast<uint64_t>(static_cast<uint32_t>(vt.slot) * (S::kTileBytes >> 4));
                uint64_t *const freed = &v_empty[vt.slot];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 0 ? !wait_unless(&bars->p_full[half][0], p_phase[half]) : !wait(&bars->p_full[half][1], p_phase[half])) return;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 4 * h; i < 4 * h + 4; ++i)
                            tc_mma_f16_ts(d + 256u + 128u * half, d + 128u * half + 8u * i, vd + i * (2048 >> 4), id_o, add || i > 0 ? 1u : 0u);
                        if (h == 1) {
                            if (last) tc_commit(&bars->s_full[half]);
                            if (last_use) tc_commit(freed);
                        }
                    }
                    __syncwarp();
                    if (h == 0) there = next();
                }
                p_phase[half] ^= 1u;
                if (last_use) {
                    vt.step(CODES ? S::kK : S::kV);
                    if (CODES) vt.step(S::kK);
                }
            };
            const auto terms_there = [&] { return test(&v_full[vt.slot], vt.phase) && test(&bars->p_full[0][0], p_phase[0]); };
            uint32_t flags = 0;                                        // of the tile
            bool start = true;
            bool work = w.valid();
            while (ok && work) {
                if (start) {
                    // an item's first scores
                    if (!wait(&bars->k_full[kt.slot], kt.phase)) break;
                    flags = bars->flags[kt.slot];
                    if (!wait(&bars->q_full[0], q_phase[0])) break;
                    q_phase[0] ^= 1u;
                    const bool two = (flags & kTwo) != 0;
                    scores(0, !two, terms_there);
                    if (two) {
                        if (!wait(&bars->q_full[1], q_phase[1])) break;
                        q_phase[1] ^= 1u;
                        scores(1, true, terms_there);
                    }
                }
                const bool more = (flags & kLast) == 0, two = (flags & kTwo) != 0, add = (flags & kFirst) == 0;
                work = (flags & kEnd) == 0;
                if (!there && !wait(&v_full[vt.slot], vt.phase)) break;
                sums(0, add, !more, !two, [&] { return more ? test(&bars->k_full[kt.slot], kt.phase) : two && test(&bars->p_full[1][0], p_phase[1]); });
                if (more) {
                    if (!ok || !wait_unless(&bars->k_full[kt.slot], kt.phase)) break;
                    flags = bars->flags[kt.slot];
                    scores(0, !two, [&] { return two ? test(&bars->p_full[1][0], p_phase[1]) : terms_there(); });
                }
                if (two) {
                    if (!ok) break;
                    sums(1, add, !more, true, [&] { return false; });
                    if (ok && more) scores(1, true, terms_there);
                }
                start = !more;
            }
            // what was issued is done before tensor memory is given back
            if (elect_one()) tc_commit(&bars->done);
            __syncwarp();
            if (!warp_wait(&bars->done, 0u, landing_limit(a.wait_ns))) fail();
        } else if (!CODES && warp == S::kCopyWarp) {
            // ------------------------------------------------------- copies
            Turn kt, vt;
            long long issued = 0, landing_k = 0, landing_v = 0;        // tiles; those of keys and of values that copies were issued for
            bool ok = true;
            const int in_page = a.c.page_tokens;
            for (; ok && w.valid(); w.next(a)) {
                const int32_t *table = a.c.table + w.s * a.c.ldt;
                const int64_t head = static_cast<int64_t>(w.h) * a.c.head_bytes;
                const int begin = first_seen(a, w), end = w.hi, pages = (end + in_page - 1) >> a.c.log_page;
                int held = -32, page = 0;                              // lane l holds page held + l of the sequence
                for (int t = w.from; ok && t < w.upto; ++t, ++issued) {
                    // tokens lo .. lo + tokens - 1 of the tile are there
                    const int t0 = (w.first + t) * kTile, lo = max(t0, begin), tokens = max(min(end, t0 + kTile) - lo, 0);
                    const int p0 = lo >> a.c.log_page, np = tokens > 0 ? ((lo + tokens - 1) >> a.c.log_page) - p0 + 1 : 0;
                    if (np > 0 && p0 + np > held + 32) {
                        held = p0;
                        page = page_of(a, table, held + lane, p0, pages);
                    }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {                   // keys, then values
                        Turn &tn = kv == 0 ? kt : vt;
                        constexpr int kDepth[2] = {S::kK, S::kV};
                        uint64_t *full = kv == 0 ? &bars->k_full[tn.slot] : &bars->v_full[tn.slot];
                        uint64_t *empty = kv == 0 ? &bars->k_empty[tn.slot] : &bars->v_empty[tn.slot];
                        uint8_t *dst = (kv == 0 ? ks : vs) + tn.slot * S::kTileBytes;
                        bool go = !aborted();
                        if (go && issued >= kDepth[kv] && !mbar_wait(empty, tn.phase ^ 1u, a.wait_ns)) {
                            fail();
                            go = false;
                        }
                        ok = __all_sync(0xFFFFFFFFu, go) != 0;
                        if (!ok) break;
                        // a lane copies 64 dims of a page's tokens: n from row `at` of the tile on
                        static_assert(kTile / 16 * CH <= 32, "a lane a piece");
                        const int j = lane / CH, y = lane % CH, pg = __shfl_sync(0xFFFFFFFFu, page, min(p0 + j - held, 31));
                        const int in = max(lo - ((p0 + j) << a.c.log_page), 0), at = ((p0 + j) << a.c.log_page) + in - t0;
                        const int n = j < np ? min(in_page - in, lo - t0 + tokens - at) : 0;
                        if (kv == 1) {
                            // no values where no token is, and none of a page that the cache does not have
                            const auto clear = [&](int from, int upto, int chunk) {
                                for (int i = 8 * from + lane; i < 8 * upto; i += 32) sts128(dst + chunk * kAtomRows + 16 * i, make_uint4(0u, 0u, 0u, 0u));
                            };
                            unsigned bad = __ballot_sync(0xFFFFFFFFu, n > 0 && pg < 0);
                            if (tokens < kTile || bad != 0) {
                                for (int i = 0; i < CH; ++i) clear(0, lo - t0, i), clear(lo - t0 + tokens, kTile, i);
                                for (; bad != 0; bad &= bad - 1) {
                                    const int l = __ffs(bad) - 1, from = __shfl_sync(0xFFFFFFFFu, at, l);
                                    clear(from, from + __shfl_sync(0xFFFFFFFFu, n, l), l % CH);
                                }
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                        }
                        const int bytes = pg >= 0 ? n * 128 : 0;
                        const uint32_t all = __reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(bytes));
                        if (lane == 0) {
                            if (kv == 0) {
                                uint32_t flags = (both() ? kTwo : 0u) | (t == w.from ? kFirst : 0u);
                                if (t + 1 == w.upto) {
                                    Walk after = w;
                                    after.next(a);
                                    flags |= kLast | (after.valid() ? 0u : kEnd);
                                }
                                bars->flags[tn.slot] = flags;
                            }
                            mbar_arrive_expect_tx(full, all);
                        }
                        __syncwarp();
                        if (bytes > 0)
                            bulk_g2s(dst + y * kAtomRows + at * 128, a.c.pages + pg * a.c.page_bytes + head + ((kv * CH + y) * in_page + in) * 128,
                                     static_cast<uint32_t>(bytes), full);
                        landing_k = kv == 0 ? issued + 1 : landing_k;
                        landing_v = kv == 1 ? issued + 1 : landing_v;
                        tn.step(kDepth[kv]);
                    }
                }
            }
            // no copy may be landing when the CTA leaves
            const auto land = [&](uint64_t *full, long long n, int depth) {
                for (long long i = n > depth ? n - depth : 0; i < n; ++i)
                    if (!mbar_wait(&full[i % depth], static_cast<uint32_t>(i / depth) & 1u, landing_limit(a.wait_ns))) fail();
            };
            land(bars->k_full, landing_k, S::kK);
            land(bars->v_full, landing_v, S::kV);
        }
    } else {
        if constexpr (CODES) {
            // ---------------------------------------------- codes to fp16
            set_regs<S::kLaunchRegs, S::kConvertRegs>();
            // Four warps; a thread has a 16-byte unit of four tokens' rows in each 64 dims,
            // fetched a tile of keys or values ahead of its conversion: tokens me / 4 + 32 i.
            // A lane has the scales of tokens 4 lane .. + 3.
            constexpr int kUnits = CH * 4;
            const int me = tid - S::kConvertWarp0 * 32, in_page = a.c.page_tokens, log_page = a.c.log_page;
            const int unit = me & 3;
            const int to_values = CH * in_page * 64;                   // from a key's unit to its value's
            // The walk is where the fetches are, a tile ahead: `fresh` says that it has come to
            // another item. Of the tile that was fetched:
            int at = w.from, held = 0, page = 0, ahead = 0;            // lane l holds page held + l, and the one 32 further on
            bool fresh = true;
            uint32_t mark = 0;
            bool exact = false;
            Bounds bounds;
            uint4 codes[kUnits];
            float4 scale;
            // where the fetched tile's keys are (nullptr: not held) and their scales
            const uint8_t *src[4];
            const float4 *scale_src;
            int scale_there;                                           // bits of its four tokens that are there
            const auto aim = [&] {
                if (!w.valid()) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) src[i] = nullptr;
                    scale_src = nullptr, scale_there = 0;
                    return;
                }
                const int end = w.hi, t0 = (w.first + at) * kTile, tokens = min(max(end - t0, 0), kTile);
                const int32_t *table = a.c.table + w.s * a.c.ldt;
                const int p0 = t0 >> log_page, pages = (end + in_page - 1) >> log_page;
                if (fresh) {
                    bounds = Bounds(a, w);
                    held = p0;
                    page = page_of(a, table, held + lane, bounds.begin >> log_page, pages);
                    ahead = page_of(a, table, held + 32 + lane, bounds.begin >> log_page, pages);
                } else if (p0 >= held + 32) {                          // (a tile's pages never straddle: 32 is a multiple of their number)
                    held += 32;
                    page = ahead;
                    ahead = page_of(a, table, held + 32 + lane, bounds.begin >> log_page, pages);
                }
                const uint8_t *head = a.c.pages + static_cast<int64_t>(w.h) * a.c.head_bytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int tok = i * 32 + me / 4, x = t0 + tok;
                    const int pg = __shfl_sync(0xFFFFFFFFu, page, (x >> log_page) - held);
                    src[i] = tok < tokens && x >= bounds.begin && pg >= 0 ? head + pg * a.c.page_bytes + (x & (in_page - 1)) * 64 + 16 * unit : nullptr;
                }
                const int x = t0 + 4 * lane, pg = __shfl_sync(0xFFFFFFFFu, page, (x >> log_page) - held);
                scale_there = (15 >> (4 - min(max(tokens - 4 * lane, 0), 4))) & (15 << min(max(bounds.begin - x, 0), 4));
                if (pg < 0) scale_there = 0;                           // a page that the cache does not have
                scale_src = scale_there != 0 ? reinterpret_cast<const float4 *>(head + pg * a.c.page_bytes + 2 * to_values + (x & (in_page - 1)) * 4) : nullptr;
                exact = bounds.exact(a, t0);
                mark = (both() ? kTwo : 0u) | (fresh ? kFirst : 0u);
                fresh = false;
                if (++at >= w.upto) {
                    w.next(a);
                    at = w.from;
                    fresh = true;
                    mark |= kLast | (w.valid() ? 0u : kEnd);
                }
            };
            const auto load = [&](int j, int kv) {
                // (past L1: the little of it that is left beside shared memory holds the threads' own)
                return src[j % 4] ? __ldcg(reinterpret_cast<const uint4 *>(src[j % 4] + kv * to_values + j / 4 * (in_page * 64))) : make_uint4(0u, 0u, 0u, 0u);
            };
            const auto load_scales = [&](int kv) {
                float4 s = scale_src ? __ldcg(scale_src + kv * (in_page / 4)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!(scale_there & 1)) s.x = 0.0f;
                if (!(scale_there & 2)) s.y = 0.0f;
                if (!(scale_there & 4)) s.z = 0.0f;
                if (!(scale_there & 8)) s.w = 0.0f;
                return s;
            };
            aim();
#pragma unroll
            for (int j = 0; j < kUnits; ++j) codes[j] = load(j, 0);
            scale = load_scales(0);
            uint32_t *const mine = factors + (warp - S::kConvertWarp0) * kTile;
            Turn kt, sc;
            long long done = 0;
            bool ok = true;
            bool work = mark != 0u;                                    // (a tile is kFirst, or there is none)
            {
                while (ok && work) {
                    const uint32_t flags = mark;                       // of this tile
                    const bool by_column = exact;
                    work = (flags & kEnd) == 0;
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        // (tested here, looked at after the factors are made)
                        uint64_t *const room = &bars->k_empty[kt.slot], *const scales_room = &bars->scales_empty[sc.slot];
                        const bool need_room = done >= S::kK, need_scales = kv == 0 && done >= 2 * S::kScaleSlots;
                        const bool there = mbar_test_wait2(room, kt.phase ^ 1u, need_scales ? scales_room : room, need_scales ? sc.phase ^ 1u : kt.phase ^ 1u);
                        const float4 was = scale;
                        const float s[4] = {was.x, was.y, was.z, was.w};
                        if (kv == 1) aim();                            // keys of the next tile come next
                        scale = load_scales(kv ^ 1);
                        uint32_t top = 0;                              // the largest that is a number
#pragma unroll
                        for (int i = 0; i < 4; ++i) top = max(top, abs_bits(s[i]) < 0x7F800000u ? abs_bits(s[i]) : 0u);
                        top = __reduce_max_sync(0xFFFFFFFFu, top);
                        const int e = max(static_cast<int>(top >> 23) - 126, -118);   // scales are below 2^e
                        const float down = pow2(-e);
                        uint32_t factor[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = by_column ? 1.0f : s[i] * down;
                            factor[i] = pack_f16x2_rn(y, y);
                        }
                        __syncwarp();                                  // the factors before have been read
                        sts128(mine + 4 * lane, make_uint4(factor[0], factor[1], factor[2], factor[3]));
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) factor[i] = mine[i * 32 + me / 4];
                        if (!__all_sync(0xFFFFFFFFu, there)) {
                            if (need_scales && !warp_wait(scales_room, sc.phase ^ 1u, a.wait_ns)) ok = false;
                            if (ok && need_room && !warp_wait(room, kt.phase ^ 1u, a.wait_ns)) ok = false;
                        }
                        if (!ok) break;
                        uint8_t *dst = ks + kt.slot * S::kTileBytes;
#pragma unroll
                        for (int j = 0; j < kUnits; ++j) {
                            const uint4 v = codes[j];
                            codes[j] = load(j, kv ^ 1);
                            const int tok = j % 4 * 32 + me / 4, u = unit ^ ((tok >> 1) & 3);   // which of the row's units this is
                            uint32_t o[8];
                            codes_f16(v.x, o[0], o[1]), codes_f16(v.y, o[2], o[3]);
                            codes_f16(v.z, o[4], o[5]), codes_f16(v.w, o[6], o[7]);
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = hmul2_bits(o[i], factor[j % 4]);
                            uint8_t *row = dst + j / 4 * kAtomRows + tok * 128;
                            sts128(row + (((2 * u) ^ (tok & 7)) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                            sts128(row + (((2 * u + 1) ^ (tok & 7)) << 4), make_uint4(o[4], o[5], o[6], o[7]));
                        }
                        if (warp == S::kConvertWarp0) {
                            *reinterpret_cast<float4 *>(scales + sc.slot * (2 * kTile) + kv * kTile + 4 * lane) = was;
                            if (lane == 0) {
                                float *tail = scales + S::kScaleSlots * 2 * kTile + sc.slot * 4;
                                tail[1 + kv] = __int_as_float(e);
                                if (kv == 1) tail[0] = __uint_as_float(top);
                            }
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            if (kv == 0 && me == 0) bars->flags[kt.slot] = flags;
                            mbar_arrive(&bars->k_full[kt.slot]);
                            if (kv == 1) mbar_arrive(&bars->scales_full[sc.slot]);
                        }
                        kt.step(S::kK);
                        ++done;
                    }
                    sc.step(S::kScaleSlots);
                }
            }
            if (!ok) fail();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == S::kMmaWarp) tmem_dealloc(tmem, 512u);
}

template <int KIND, int DP> cudaError_t launch(const AttnArgs &args, int sm_count, cudaStream_t s, int *ctas)
{
    AttnArgs a = args;
    const void *f = reinterpret_cast<const void *>(&attn_tensor_kernel<KIND, DP>);
    static_assert(TensorShape<KIND, DP>::kSmem <= kSmemOptIn, "shared memory");
    cudaError_t e = set_max_smem(f, TensorShape<KIND, DP>::kSmem);
    if (e != cudaSuccess) return e;
    if constexpr (TensorShape<KIND, DP>::kCodes) {
        // The warpgroups' registers have to add up to what the launch has: a share that is not
        // there is waited for without end. The build refuses another count; looked at until it
        // is known, so that a query that fails once is asked again.
        using S = TensorShape<KIND, DP>;
        static_assert(4 * S::kLaunchRegs >= 2 * S::kSoftmaxRegs + S::kConvertRegs + S::kMmaRegs, "the warpgroups' shares");
        static std::atomic<bool> enough{false};
        if (!enough.load(std::memory_order_relaxed)) {
            cudaFuncAttributes fa{};
            e = cudaFuncGetAttributes(&fa, f);
            if (e != cudaSuccess) return e;
            if (fa.numRegs != S::kLaunchRegs) return cudaErrorLaunchOutOfResources;
            enough.store(true, std::memory_order_relaxed);
        }
    }
    *ctas = std::min(kTensorMaxCtas, sm_count);
    void *p[] = {&a};
    return launch_pdl(f, dim3(static_cast<unsigned>(*ctas)), dim3(TensorShape<KIND, DP>::kThreads), TensorShape<KIND, DP>::kSmem, s, p);
}

} // namespace

cudaError_t launch_attn_tensor(AttnArgs a, int sm_count, cudaStream_t s)
{
    a.tile = kTensorTile, a.block = kTensorRows;
    a.item_cost = 2;
    int ctas = 0;
    const bool small = a.c.chunks == 1;
    cudaError_t e;
    switch (a.c.type) {
    case Q4_TYPE_F16: e = small ? launch<0, 64>(a, sm_count, s, &ctas) : launch<0, 128>(a, sm_count, s, &ctas); break;
    case Q4_TYPE_BF16: e = small ? launch<1, 64>(a, sm_count, s, &ctas) : launch<1, 128>(a, sm_count, s, &ctas); break;
    default: e = small ? launch<2, 64>(a, sm_count, s, &ctas) : launch<2, 128>(a, sm_count, s, &ctas); break;
    }
    return e != cudaSuccess ? e : launch_attn_join(a, ctas, s);
}

} // namespace q4
