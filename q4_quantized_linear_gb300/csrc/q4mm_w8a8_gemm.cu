// q4mm_w8a8_gemm.cu -- the int8 product for many tokens, on the 5th-generation
// tensor cores: Y[t][j] = sx[t] * s_j * sum_c xq[t][c] * code[j][c].
//
// sm_103a has no fast integer MMA; an int8 code is exact in fp16, so a product
// of codes is exact in the MMA and their sum is exact while it stays below
// 2^24 (fp32 accumulation). Past that each step of 16 columns cuts the running sum
// to fp32: up to 8e-6 of the terms' sizes at k = 14336 and 3e-5 at 131072 for codes
// of one sign, nothing for codes of mixed sign. The MMA is bound by the fp16 rate: 2 m n k
// operations at the dense fp16 peak.
//
// A pair of CTAs (cta_group::2) takes a tile of 256 weight rows by N tokens:
// A = the weights, 128 rows in each CTA's tensor memory; B = the tokens, half
// of them in each CTA's shared memory; D = 128 rows x N fp32 in each CTA's
// tensor memory. The pair halves what each SM reads of B from L2 and from
// shared memory: with a CTA of its own (128 x N) an SM would need 80 bytes a
// clock of L2 at N = 256 to keep the MMA busy, a pair needs 48.
//   The weights stay int8 in memory, L2 and shared memory: dequantising warps
// turn a record's 64 codes of a row into fp16 (one byte permute and one
// subtraction for two) and store them to tensor memory as the A operand.
//   The tokens are laid out once per call as fp16 tiles in the swizzled image
// the MMA reads, so that a K step's half tile is one bulk copy.
//
// Warps of a CTA:
//   0      B producer: bulk copies of its half of the token tile
//   1      tensor memory; in the even CTA one thread issues the MMAs
//   2      weight-record producer
//   3      tells the even CTA when a step's operands are in place here: waits
//          for the weights in tensor memory and for the B tile, then arrives on
//          the even CTA's `ready` barrier, one arrival a CTA and step (by the
//          dequantising warps themselves it took a third of their time)
//   4-11   dequantise: four warps take a step's first record, four its second
//   12-19  epilogue: two warps per 32 rows, half of the token columns each.
// The MMA's commits release a stage (A and B) in both CTAs. A pair runs
// through tiles in turn: the rings carry on into the next tile while the
// epilogue reads D; only D's own read keeps the MMA waiting.
// Where tiles are too few for the device, K is cut into slices, each a tile of its
// own that writes its raw sums (whole numbers in fp32) to the workspace; a second
// kernel adds them in slice order and scales.
//   GB300, us a call with the coding (floor at the measured bf16 rate): 4096 x
// 14336 x 4096 bf16 274 (248); 4096 x 9728 x 2560 fp32 144 (105), its stores; 540 x
// 9728 x 2560 fp32 30.5 (14), the dequantising warps (a step of 128 columns takes
// them 0.4 us whatever the tokens); 540 x 2560 x 9728 bf16 35 (14), 64 x 9728 x
// 2560 15.4 (3.7), the latencies of a step and of the launches.
// Every wait is bounded; after a timeout all roles leave their loops, the
// MMAs and copies in flight are waited for and the CTAs of the pair leave
// together.
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_rows.cuh"
#include "q4mm_w8a8.h"

namespace q4 {
namespace {

constexpr int kErrTimeout = 5;
constexpr int kDequantWarp0 = 4, kDequantWarps = 8;
constexpr int kEpilogueWarp0 = 12, kEpilogueWarps = 8;
constexpr int kThreads = (kEpilogueWarp0 + kEpilogueWarps) * 32;
// A step of the K loop takes two records' columns (128): every barrier is
// touched half as often as with one, and a step's fixed latencies (two waits,
// a store to tensor memory, two arrivals, a commit), some 0.35 us, bounded the
// loop at 0.36 us a record with one.
constexpr int kStepRecords = 2;
constexpr uint32_t kSlotBytes = kStepRecords * kW8RecordBytes;
constexpr int kMaxAStages = 8, kMaxBStages = 10, kWRing = 4;
constexpr uint32_t kAColumns = kStepRecords * 32;                 // tensor-memory columns of a step's weights
constexpr int kStageTokens = 16;                                  // token columns an epilogue warp stages at once
constexpr size_t kWarpStaging = kStageTokens * 32 * 4;
constexpr size_t kStagingBytes = kEpilogueWarps * (kWarpStaging + 128 * 4);   // and its tokens' scales

// Codes to fp16 tiles: [half tile of H = N / 2 tokens][64 columns][H rows of
// 128 bytes], 16-byte chunk c of row r at c ^ (r & 7). Rows past m and columns
// past k are zeros.
__global__ void __launch_bounds__(256) tile_kernel(const int8_t *Xq, uint8_t *ximg, int m, int64_t k, int np, int H,
                                                   int halves)
{
    // the product starts its set-up once this kernel has its input: its bounded
    // waits then never span an earlier kernel
    pdl_wait();
    pdl_launch_dependents();
    const int64_t total = static_cast<int64_t>(halves) * np * H * 4;
    for (int64_t it = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; it < total;
         it += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int c = static_cast<int>(it & 3);              // 16 codes
        const int64_t rowid = it >> 2;                       // (j * np + p) * H + r
        const int r = static_cast<int>(rowid % H);
        const int64_t jp = rowid / H;
        const int p = static_cast<int>(jp % np);
        const int64_t tok = (jp / np) * H + r;
        const int64_t col = static_cast<int64_t>(p) * kPairK + 16 * c;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (tok < m && col < k) v = __ldg(reinterpret_cast<const uint4 *>(Xq + tok * k + col));
        const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = hsub2_bits(__byte_perm(w[i], 0x64646464u, 0x4140), 0x64806480u);
            o[2 * i + 1] = hsub2_bits(__byte_perm(w[i], 0x64646464u, 0x4342), 0x64806480u);
        }
        uint8_t *dst = ximg + rowid * 128;
        *reinterpret_cast<uint4 *>(dst + (((2 * c) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(dst + (((2 * c + 1) ^ (r & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

struct SliceSumArgs {
    const float *partials;     // [slices][m][ld]
    int64_t ld, stride;
    int slices;
    const float *sx, *row_scale;
    void *Y;
    int64_t ldy, n;
};

struct CodeTileArgs {
    const void *X;
    int64_t ldx;
    uint8_t *ximg;
    float *sx;
    int m, rows;       // tokens, and with the last tile's padding
    int64_t k;
    int np, H;
};

// Tokens to codes and straight into the tiles: a row per CTA in turn, read
// once (its first NV vectors a thread stay in registers; what is past them is
// read again from L2). Rows m .. rows - 1 and columns past k are zeros. The
// codes and scales are q4_a8_quantize's.
template <typename T, int V> __global__ void __launch_bounds__(512) code_tile_kernel(const CodeTileArgs a)
{
    constexpr int NV = V >= 4 ? 2 : 4;
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    const int G = blockDim.x, t = threadIdx.x, k = static_cast<int>(a.k), kp = a.np * kPairK;
    RowReducer red{rbuf, G / 32, false};
    red.clear(G);
    __syncthreads();
    for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *xr = static_cast<const T *>(a.X) + row * a.ldx;
        const int kr = row < a.m ? k : 0;
        Pack<T, V> x[NV];
        uint32_t mb = 0u;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * G + t) * V;
            x[i] = c < kr ? load_pack<T, V>(xr, c, kr) : zero_pack<T, V>();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) mb = max(mb, abs_bits(elem(x[i], j)));
        for (int c = (NV * G + t) * V; c < kr; c += G * V) {
            const Pack<T, V> v = load_pack<T, V>(xr, c, kr);
#pragma unroll
            for (int j = 0; j < V; ++j) mb = max(mb, abs_bits(elem(v, j)));
        }
        const CodeScale cs = code_scale(red.max_bits(mb));
        if (t == 0 && row < a.m) a.sx[row] = cs.scale;
        const int j2 = row / a.H, r = row - j2 * a.H;
        uint8_t *out = a.ximg + (static_cast<int64_t>(j2) * a.np * a.H + r) * 128;
        auto put = [&](int c, const Pack<T, V> &v) {
            float f[V];
#pragma unroll
            for (int j = 0; j < V; ++j) f[j] = static_cast<float>(code_of(elem(v, j), cs.factor));
            const int p = c / kPairK, e = c - p * kPairK;   // V divides 8: inside one 16-byte chunk
            store_pack<__half, V>(reinterpret_cast<__half *>(out + static_cast<int64_t>(p) * a.H * 128 +
                                                             (((e >> 3) ^ (r & 7)) << 4)) + (e & 7), 0, V, pack_of<__half, V>(f));
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * G + t) * V;
            if (c < kp) put(c, x[i]);
        }
        for (int c = (NV * G + t) * V; c < kp; c += G * V) put(c, load_pack<T, V>(xr, c, kr));
    }
}

struct Smem {
    uint8_t *b, *w, *stage;
    uint64_t *full_b, *empty_b, *full_w, *empty_w, *stored, *ready, *empty_a, *d_full, *d_empty, *done;
    uint32_t *tmem_slot;
    int *abort;
};

__device__ __forceinline__ bool aborted(const Smem &sm) { return *reinterpret_cast<volatile int *>(sm.abort) != 0; }
__device__ __forceinline__ void fail(const Smem &sm, const W8a8GemmArgs &a)
{
    *reinterpret_cast<volatile int *>(sm.abort) = 1;
    record_status(a.status, kErrTimeout);
}
// A bounded wait with one outcome for the warp.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, limit_ns)) != 0;
}
// The MMA warp's waits: tests without suspending, since a warp resumes some
// 170 ns late from a suspended wait and the tensor cores would run dry (4096 x
// 14336 x 4096: 404 us a call with suspended waits, 364 with tests).
__device__ __forceinline__ bool warp_test(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)) != 0;
}
__device__ __forceinline__ bool warp_spin_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    for (uint32_t i = 0; i < 64; ++i)
        if (warp_test(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        for (uint32_t i = 0; i < 64; ++i)
            if (warp_test(bar, parity)) return true;
        if (__any_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > limit_ns)) return false;
    }
}

// A position in a ring of `depth` slots and its phase.
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step(int depth)
    {
        if (++slot == depth) slot = 0, phase ^= 1u;
    }
};

// A staged [16 tokens][32 rows] out to `tokens` rows of Y, B bytes a store; of the
// 32 weight rows `rows` exist.
template <typename T, int B>
__device__ __forceinline__ void store_staged(T *dst, int64_t ld, const uint8_t *stage, int rows, int tokens, int lane)
{
    using A = typename AccessOf<B>::type;
    constexpr int kVec = B / static_cast<int>(sizeof(T)), kLanes = 32 / kVec, kTokens = 32 / kLanes;
    const int c = lane % kLanes * kVec;
#pragma unroll
    for (int i = 0; i < kStageTokens; i += kTokens) {
        const int t = i + lane / kLanes;
        const T *src = reinterpret_cast<const T *>(stage) + t * 32 + c;
        if (t >= tokens) continue;
        T *out = dst + t * ld + c;
        if (c + kVec <= rows) {
            *reinterpret_cast<A *>(out) = *reinterpret_cast<const A *>(src);
        } else {
            using E = typename AccessOf<static_cast<int>(sizeof(T))>::type;
            for (int u = 0; u < kVec; ++u)
                if (c + u < rows) reinterpret_cast<E *>(out)[u] = reinterpret_cast<const E *>(src)[u];
        }
    }
}

// SLICED: K slices (T is float: raw sums).
template <typename T, bool SLICED> __global__ void __launch_bounds__(kThreads, 1) w8a8_gemm_kernel(const W8a8GemmArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
    const int N = a.N, H = N / 2, SA = a.astages, SB = a.bstages, RW = a.wring, np = a.np;
    const uint32_t brec = static_cast<uint32_t>(H) * 128u;    // a record's columns of the half tile
    const uint32_t bstage = kStepRecords * brec;
    // Steps of a tile: K slice `tile % KS` has `per` of them, the last slice what is
    // left; the last step of K may hold one record.
    const int all_steps = (np + kStepRecords - 1) / kStepRecords, KS = SLICED ? a.kslices : 1;
    const int per = SLICED ? (all_steps + KS - 1) / KS : all_steps;
    const auto first_step = [&](int tile) { return tile % KS * per; };
    const auto end_step = [&](int tile) { return min(all_steps, first_step(tile) + per); };
    const uint32_t acol0 = static_cast<uint32_t>(N);   // first A column after D (N is a multiple of 32)

    Smem sm;
    sm.b = base;
    sm.w = sm.b + static_cast<size_t>(SB) * bstage;
    sm.stage = sm.w + static_cast<size_t>(RW) * kSlotBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm.stage + kStagingBytes);
    sm.full_b = bars;
    sm.ready = sm.full_b + SB;
    sm.empty_a = sm.ready + SA;
    // rings of one depth turn together: one commit releases both
    sm.empty_b = SB == SA ? sm.empty_a : sm.empty_a + SA;
    sm.full_w = sm.empty_a + SA + (SB == SA ? 0 : SB);
    sm.empty_w = sm.full_w + RW;
    sm.stored = sm.empty_w + RW;
    sm.d_full = sm.stored + SA;
    sm.d_empty = sm.d_full + 1;
    sm.done = sm.d_empty + 1;
    sm.tmem_slot = reinterpret_cast<uint32_t *>(sm.done + 1);
    sm.abort = reinterpret_cast<int *>(sm.tmem_slot + 1);
    if (tid == 0) {
        for (int i = 0; i < SB; ++i) mbar_init(&sm.full_b[i], 1);
        if (SB != SA)
            for (int i = 0; i < SB; ++i) mbar_init(&sm.empty_b[i], 1);
        for (int i = 0; i < SA; ++i) {
            mbar_init(&sm.stored[i], kDequantWarps);
            mbar_init(&sm.ready[i], 2);                    // both CTAs
            mbar_init(&sm.empty_a[i], 1);
        }
        for (int i = 0; i < RW; ++i) mbar_init(&sm.full_w[i], 1), mbar_init(&sm.empty_w[i], kDequantWarps);
        mbar_init(sm.d_full, 1);
        mbar_init(sm.d_empty, 2 * kEpilogueWarps);
        mbar_init(sm.done, 1);
        *sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(sm.tmem_slot, 512u);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // the other CTA's barriers are initialised before anything arrives there
    tc_fence_after();
    const uint32_t tmem = *sm.tmem_slot;
    const bool dequant = warp >= kDequantWarp0 && warp < kDequantWarp0 + kDequantWarps;

    if (warp == 0) {
        // ----------------------------------------------------- B producer
        pdl_wait();
        if (lane == 0) {
            Ring b;
            int64_t issued = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
                const int jt = tile / KS % a.ts;
                const uint8_t *src = a.ximg + (static_cast<size_t>(2 * jt) + rank) * np * brec;
                const int end = end_step(tile);
                for (int st = first_step(tile); st < end; ++st) {
                    if (aborted(sm)) { ok = false; break; }
                    if (issued >= SB && !mbar_wait(&sm.empty_b[b.slot], b.phase ^ 1u, a.wait_ns)) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    const uint32_t bytes = static_cast<uint32_t>(min(kStepRecords, np - st * kStepRecords)) * brec;
                    mbar_arrive_expect_tx(&sm.full_b[b.slot], bytes);
                    bulk_g2s(sm.b + static_cast<size_t>(b.slot) * bstage, src + static_cast<size_t>(st) * bstage, bytes,
                             &sm.full_b[b.slot]);
                    ++issued;
                    b.step(SB);
                }
            }
            // no copy may be landing when the CTA leaves, also if another role gave up
            for (int64_t i = issued > SB ? issued - SB : 0; i < issued; ++i)
                if (!mbar_wait(&sm.full_b[i % SB], static_cast<uint32_t>(i / SB) & 1u, landing_limit(a.wait_ns))) fail(sm, a);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ record producer
        // What the kernels in front wrote is visible only past the wait: the
        // weights stream before it only where the caller declared them read-only.
        if (!a.prefetch_w) pdl_wait();
        if (lane == 0) {
            Ring w;
            int64_t issued = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
                // the last pair of an odd number of groups: its second CTA
                // reads the last group again and writes nothing
                const int G = min(2 * (tile / KS / a.ts) + static_cast<int>(rank), a.groups - 1);
                const uint8_t *src = a.W + static_cast<size_t>(G) * np * kW8RecordBytes;
                const int end = end_step(tile);
                for (int st = first_step(tile); st < end; ++st) {
                    if (aborted(sm)) { ok = false; break; }
                    if (issued >= RW && !mbar_wait(&sm.empty_w[w.slot], w.phase ^ 1u, a.wait_ns)) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    const uint32_t bytes = static_cast<uint32_t>(min(kStepRecords, np - st * kStepRecords)) * kW8RecordBytes;
                    mbar_arrive_expect_tx(&sm.full_w[w.slot], bytes);
                    bulk_g2s(sm.w + static_cast<size_t>(w.slot) * kSlotBytes, src + static_cast<size_t>(st) * kSlotBytes, bytes,
                             &sm.full_w[w.slot]);
                    ++issued;
                    w.step(RW);
                }
            }
            for (int64_t i = issued > RW ? issued - RW : 0; i < issued; ++i)
                if (!mbar_wait(&sm.full_w[i % RW], static_cast<uint32_t>(i / RW) & 1u, landing_limit(a.wait_ns))) fail(sm, a);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        // The whole warp runs the loop, one elected lane issues.
        if (rank == 0) {
            const uint32_t idesc = idesc_f16_f32(256, static_cast<uint32_t>(N));
            const uint64_t bdesc0 = smem_desc_sw128(smem_u32(sm.b));
            const uint32_t d = __shfl_sync(0xFFFFFFFFu, tmem, 0), a0 = d + acol0;
            Ring r, b;
            bool ok = true;
            uint32_t seq = 0;
            for (int tile = pair; ok && tile < a.tiles; tile += pairs, ++seq) {
                // D has been read out of both CTAs' tensor memory
                if (seq > 0 && !warp_spin_wait(sm.d_empty, (seq - 1) & 1u, a.wait_ns)) {
                    ok = false;
                    break;
                }
                bool ready = warp_test(&sm.ready[r.slot], r.phase);
                const int begin = first_step(tile), end = end_step(tile);
                for (int st = begin; st < end; ++st) {
                    if (!ready && !warp_spin_wait(&sm.ready[r.slot], r.phase, a.wait_ns)) {
                        ok = false;
                        break;
                    }
                    const uint64_t bd = bdesc0 + static_cast<uint64_t>(static_cast<uint32_t>(b.slot) * (bstage >> 4));
                    const uint64_t bd2 = bd + (brec >> 4);
                    const uint32_t at = a0 + kAColumns * static_cast<uint32_t>(r.slot);
                    const bool whole = (st + 1) * kStepRecords <= np;
                    uint64_t *const done_a = &sm.empty_a[r.slot], *const done_b = &sm.empty_b[b.slot];
                    r.step(SA);
                    b.step(SB);
                    tc_fence_after();
                    if (elect_one()) {
                        tc_mma_f16_ts_pair(d, at, bd, idesc, st > begin ? 1u : 0u);
#pragma unroll
                        for (uint32_t i = 1; i < 4; ++i) tc_mma_f16_ts_pair(d, at + 8u * i, bd + 2u * i, idesc, 1u);
                        if (whole) {
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i) tc_mma_f16_ts_pair(d, at + 32u + 8u * i, bd2 + 2u * i, idesc, 1u);
                        }
                        tc_commit_pair(done_a, 3);
                        if (SB != SA) tc_commit_pair(done_b, 3);
                    }
                    __syncwarp();
                    ready = st + 1 < end && warp_test(&sm.ready[r.slot], r.phase);
                }
                if (ok && elect_one()) tc_commit_pair(sm.d_full, 3);
                __syncwarp();
            }
            if (!ok && lane == 0) fail(sm, a);
            __syncwarp();
            if (elect_one()) tc_commit_pair(sm.done, 3);   // also after a timeout
        }
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------- operands in place here
        if (lane == 0) {
            Ring r, b;
            bool ok = true;
            const uint32_t ready0 = mapa_shared(smem_u32(sm.ready), 0u);
            for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
                const int end = end_step(tile);
                for (int st = first_step(tile); st < end; ++st, r.step(SA), b.step(SB)) {
                    if (!mbar_test_wait2(&sm.full_b[b.slot], b.phase, &sm.stored[r.slot], r.phase) &&
                        (!mbar_wait(&sm.full_b[b.slot], b.phase, a.wait_ns) || !mbar_wait(&sm.stored[r.slot], r.phase, a.wait_ns))) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    mbar_arrive_remote_async(ready0 + 8u * static_cast<uint32_t>(r.slot));
                }
            }
        }
        __syncwarp();
    } else if (dequant) {
        // --------------------------------------------------- dequantise W
        const int q = warp & 3, rec = (warp - kDequantWarp0) >> 2;
        const int row = q * 32 + lane;
        const uint32_t at0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + acol0 + 32u * static_cast<uint32_t>(rec);
        const uint8_t *const src0 = sm.w + rec * kW8RecordBytes + row * kPairK;
        // A row is four 16-byte chunks, rows 64 bytes apart: lanes reading the same
        // chunk would share two bank groups, four lanes each. So lane l starts at
        // chunk (l / 2) % 4, and the chunks are put back in order by selects
        // (registers take no index).
        const int rot = (lane >> 1) & 3;
        Ring w, r;
        bool ok = true;
        for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
            const int end = end_step(tile);
            for (int st = first_step(tile); st < end; ++st, w.step(RW), r.step(SA)) {
                // (a barrier's first phase counts as complete where it has none before)
                if (!__all_sync(0xFFFFFFFFu, mbar_test_wait2(&sm.full_w[w.slot], w.phase, &sm.empty_a[r.slot], r.phase ^ 1u)) &&
                    (!warp_wait(&sm.full_w[w.slot], w.phase, a.wait_ns) ||
                     !warp_wait(&sm.empty_a[r.slot], r.phase ^ 1u, a.wait_ns))) {
                    fail(sm, a);
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (st * kStepRecords + rec < np) {
                    const uint8_t *src = src0 + static_cast<uint32_t>(w.slot) * kSlotBytes;
                    uint32_t u[16], out[32];
                    {
                        uint32_t v[16];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint4 x = lds128(src + 16 * ((c + rot) & 3));
                            v[4 * c] = x.x, v[4 * c + 1] = x.y, v[4 * c + 2] = x.z, v[4 * c + 3] = x.w;
                        }
                        uint32_t t[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) t[i] = (rot & 1) ? v[(i + 12) & 15] : v[i];
#pragma unroll
                        for (int i = 0; i < 16; ++i) u[i] = (rot & 2) ? t[(i + 8) & 15] : t[i];
                    }
                    // a byte is 128 + c: as the low mantissa byte of 1024 it is the fp16
                    // 1152 + c, less 1152 exactly c
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        out[2 * i] = hsub2_bits(__byte_perm(u[i], 0x64646464u, 0x4140), 0x64806480u);
                        out[2 * i + 1] = hsub2_bits(__byte_perm(u[i], 0x64646464u, 0x4342), 0x64806480u);
                    }
                    tmem_st_32x32b_x32(at0 + static_cast<uint32_t>(r.slot) * kAColumns, out);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty_w[w.slot]);   // read into registers
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.stored[r.slot]);
            }
        }
    } else if (warp >= kEpilogueWarp0) {
        // ------------------------------------------------------- epilogue
        // A lane holds one weight row; Y's rows are tokens. Sixteen tokens at a
        // time go through the warp's staging area and out as 16 bytes a lane, or
        // 8 or 4 where Y's rows are aligned to no more (with 2- or 4-byte stores
        // straight from the registers the epilogue of a 256 x 256 tile took 3.7 us).
        pdl_wait();
        const int q = warp & 3, half = (warp - kEpilogueWarp0) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        uint8_t *stage = sm.stage + (warp - kEpilogueWarp0) * (kWarpStaging + 128 * 4);
        float *const sxs = reinterpret_cast<float *>(stage + kWarpStaging);
        T *Y = static_cast<T *>(a.Y);
        const uintptr_t ybits = reinterpret_cast<uintptr_t>(Y) | static_cast<uintptr_t>(a.ldy * sizeof(T));
        uint32_t seq = 0;
        for (int tile = pair; tile < a.tiles; tile += pairs, ++seq) {
            const int G = 2 * (tile / KS / a.ts) + static_cast<int>(rank);
            const int64_t row0 = static_cast<int64_t>(G) * kW8GroupRows + q * 32;
            const int rows = G < a.groups ? static_cast<int>(max(int64_t(0), min(int64_t(32), a.n - row0))) : 0;
            const float sw = SLICED ? 1.0f : lane < rows ? __ldg(a.row_scale + row0 + lane) : 0.0f;
            const int t0 = (tile / KS % a.ts) * N + half * H;   // this warp's tokens: t0 .. t0 + H - 1
            T *const Yt = SLICED ? Y + tile % KS * a.slice_stride : Y;
            for (int i = lane; i < H; i += 32) sxs[i] = SLICED ? 1.0f : t0 + i < a.m ? __ldg(a.sx + t0 + i) : 0.0f;
            __syncwarp();
            const F2 sw2 = f2(sw, sw);
            if (!warp_wait(sm.d_full, seq & 1u, a.wait_ns)) {
                fail(sm, a);
                break;
            }
            tc_fence_after();
            const uint32_t d0 = tmem + lane_base + static_cast<uint32_t>(half * H);
            // Sixteen columns at a time; D is given back when the last have been read.
            // (Held in registers, all of them before the first store, D came back
            // sooner, but the registers spilled: 31.9 us instead of 30.7 at 540 x 9728
            // x 2560 fp32, 152 instead of 138 at 3332 x 17044 x 1472.)
#pragma unroll 1
            for (int ch = 0; ch * 16 < H; ++ch) {
                uint32_t c[16];
                tmem_ld_32x32b_x16(d0 + static_cast<uint32_t>(ch * 16), c);
                tmem_wait_ld();
                if ((ch + 1) * 16 >= H) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_async(mapa_shared(smem_u32(sm.d_empty), 0u));
                }
                using Bits = typename AccessOf<static_cast<int>(sizeof(T))>::type;
                Bits *const st = reinterpret_cast<Bits *>(stage);
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 sx = *reinterpret_cast<const float4 *>(sxs + ch * 16 + i);
                    const F2 y[2] = {f2_mul(f2(__uint_as_float(c[i]), __uint_as_float(c[i + 1])), f2_mul(f2(sx.x, sx.y), sw2)),
                                     f2_mul(f2(__uint_as_float(c[i + 2]), __uint_as_float(c[i + 3])), f2_mul(f2(sx.z, sx.w), sw2))};
                    const Pack<T, 4> o = pack_pairs<T, 4>(y);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if constexpr (sizeof(T) == 4) st[(i + u) * 32 + lane] = o.w[u];
                        else st[(i + u) * 32 + lane] = static_cast<Bits>(o.w[u / 2] >> (16 * (u & 1)));
                    }
                }
                __syncwarp();
                const int tc = t0 + ch * 16;
                T *const dst = Yt + tc * a.ldy + row0;
                const int tokens = min(kStageTokens, a.m - tc);
                if ((ybits & 15u) == 0) store_staged<T, 16>(dst, a.ldy, stage, rows, tokens, lane);
                else if ((ybits & 7u) == 0) store_staged<T, 8>(dst, a.ldy, stage, rows, tokens, lane);
                else if ((ybits & 3u) == 0) store_staged<T, 4>(dst, a.ldy, stage, rows, tokens, lane);
                else store_staged<T, static_cast<int>(sizeof(T))>(dst, a.ldy, stage, rows, tokens, lane);
                __syncwarp();
            }
        }
    }

    // No MMA of the pair and none of its arrivals is in flight past this.
    __syncthreads();
    if (tid == 0 && !mbar_wait(sm.done, 0, landing_limit(a.wait_ns))) fail(sm, a);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA's memory is used by the other past this
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512u);
}

// Y = sx s_j times the slices' sums, four weight rows a thread where Y's rows
// allow it.
template <typename T, int V> __global__ void __launch_bounds__(256) slice_sum_kernel(const SliceSumArgs a)
{
    pdl_wait();
    const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
    const int64_t t = blockIdx.y;
    if (c >= a.n) return;
    const float *p = a.partials + t * a.ld + c;   // the partials' rows are whole groups of 128
    float s[V] = {};
    for (int k = 0; k < a.slices; ++k) {
        const Pack<float, V> v = load_pack<float, V>(p + k * a.stride, 0, V);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += elem(v, i);
    }
    const float sx = a.sx[t];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = s[i] * (sx * a.row_scale[c + i]);
    store_pack<T, V>(static_cast<T *>(a.Y) + t * a.ldy, c, a.n, pack_of<T, V>(s));
}

const void *kernel_of(int ytype, bool sliced)
{
    return sliced                 ? reinterpret_cast<const void *>(&w8a8_gemm_kernel<float, true>)
           : ytype == Q4_TYPE_F32 ? reinterpret_cast<const void *>(&w8a8_gemm_kernel<float, false>)
           : ytype == Q4_TYPE_F16 ? reinterpret_cast<const void *>(&w8a8_gemm_kernel<__half, false>)
                                  : reinterpret_cast<const void *>(&w8a8_gemm_kernel<__nv_bfloat16, false>);
}

size_t smem_bytes(int N, int astages, int bstages, int wring)
{
    return 1024 + static_cast<size_t>(bstages) * kStepRecords * (N / 2) * 128 + static_cast<size_t>(wring) * kSlotBytes + kStagingBytes +
           static_cast<size_t>(2 * bstages + 3 * astages + 2 * wring + 3) * 8 + 16;
}

} // namespace

// K is cut where a slice has three steps at least, and where the slices' sums stay
// small: a bound of their own, so that the workspace's size does not follow the
// plans up and down. (By the costs below slices past these bounds gain 8 % at most,
// on layers of 30000 columns and more; layers past 131072 rows fill the device.)
constexpr int64_t kMaxSlices = 16, kMinSliceSteps = 3;
constexpr int64_t kMaxSlicedRowTiles = 512, kMaxSliceBytes = int64_t(64) << 20;
constexpr int64_t kMaxSlicedTokens = 65535;   // a grid dimension of the second kernel
static int64_t slice_bytes(int64_t slices, int64_t m, int64_t n) { return slices * m * round_up(n, kW8GroupRows) * 4; }

size_t w8a8_gemm_bytes(int64_t m, int64_t k, int64_t n)
{
    const int64_t np = ceil_div(k, kPairK), steps = ceil_div(np, kStepRecords);
    // tokens of the tiles: a multiple of 32, less than a tile of at most 256 (or of
    // the tokens, rounded up) past m
    const int64_t tokens = std::min(2 * round_up(m, 32), (m + 255) / 32 * 32);
    const int64_t slices = std::min(kMaxSlices, ceil_div(steps, kMinSliceSteps));
    const bool sliced = slices > 1 && ceil_div(n, 2 * kW8GroupRows) <= kMaxSlicedRowTiles;
    const int64_t sums = sliced ? std::min(kMaxSliceBytes, slice_bytes(slices, std::min(m, kMaxSlicedTokens), n)) : 0;
    return static_cast<size_t>(tokens * np * 128 + sums);
}

// Tokens a tile and K slices: the fewest clocks over the pairs' turns. A step takes
// 4 N clocks of MMA (256 x N x 128 at 8192 products a clock and pair), but not
// under the 700 or so in which its operands are prepared; a tile adds its first
// step's latency and D's way out; slices add a kernel and their sums' traffic.
bool plan_w8a8_gemm(int64_t m, int64_t k, int64_t n, int sm_count, W8a8GemmPlan *plan)
{
    const int64_t np = ceil_div(k, kPairK), groups = ceil_div(n, kW8GroupRows), rt = ceil_div(groups, 2);
    const int64_t steps = ceil_div(np, kStepRecords);
    // pairs on the device at once: a CTA takes an SM (where it holds fewer the others
    // follow: no pair waits on another)
    const int held = std::max(1, sm_count / 2);
    double best = 1e300;
    W8a8GemmPlan out;
    const int widest = static_cast<int>(std::min<int64_t>(256, round_up(m, 32)));
    for (int N = 32; N <= widest; N += 32) {
        W8a8GemmPlan c;
        c.N = N;
        c.astages = std::min<int>(kMaxAStages, (512 - N) / kAColumns);
        c.wring = kWRing;
        c.bstages = kMaxBStages;
        while (c.bstages > 2 && smem_bytes(N, c.astages, c.bstages, c.wring) > kSmemOptIn) --c.bstages;
        if (c.bstages <= c.astages + 1) c.bstages = std::min(c.bstages, c.astages);   // one commit a step
        c.smem = std::max<size_t>(smem_bytes(N, c.astages, c.bstages, c.wring), kSmemPerSM / 2 + 1024);   // one CTA per SM
        if (c.smem > kSmemOptIn) continue;
        c.ts = static_cast<int>(ceil_div(m, N));
        if (rt * c.ts > (int64_t(1) << 24)) continue;
        c.image_bytes = static_cast<size_t>(2) * c.ts * np * (N / 2) * 128;
        for (int ks = 1; ks <= kMaxSlices; ++ks) {
            const int64_t per = ceil_div(steps, ks), sums = ks > 1 ? slice_bytes(ks, m, n) : 0;
            if (ks > 1 && (per < kMinSliceSteps || ceil_div(steps, per) != ks ||   // every slice has steps
                           m > kMaxSlicedTokens || rt > kMaxSlicedRowTiles || sums > kMaxSliceBytes))
                continue;
            c.kslices = ks;
            c.tiles = static_cast<int>(rt * c.ts * ks);
            c.pairs = std::min(held, c.tiles);
            const double turns = static_cast<double>(ceil_div(c.tiles, c.pairs));
            const double cost = turns * (static_cast<double>(per) * std::max(4.0 * N, 700.0) + 2500.0 + 8.0 * N) +
                                (ks > 1 ? 4000.0 + static_cast<double>(sums) / 1500.0 : 0.0);
            if (cost < best) {
                best = cost;
                out = c;
            }
        }
    }
    if (out.N == 0) return false;
    *plan = out;
    return true;
}

namespace {
template <typename T> cudaError_t launch_code_tiles(CodeTileArgs a, int vec, int sm_count, cudaStream_t s)
{
    const void *fn = reinterpret_cast<const void *>(&code_tile_kernel<T, 1>);
    if (vec * sizeof(T) == 16) fn = reinterpret_cast<const void *>(&code_tile_kernel<T, 16 / sizeof(T)>);
    else if constexpr (sizeof(T) == 2) {
        if (vec == 2) fn = reinterpret_cast<const void *>(&code_tile_kernel<T, 2>);
    }
    const int64_t vecs = ceil_div(static_cast<int64_t>(a.np) * kPairK, vec);
    const int threads = static_cast<int>(std::min<int64_t>(512, round_up(ceil_div(vecs, vec >= 4 ? 2 : 4), 32)));
    const int64_t grid = std::min<int64_t>(a.rows, static_cast<int64_t>(sm_count) * (2048 / std::max(threads, 128)));
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(threads)), 0, s, args);
}
} // namespace

cudaError_t launch_w8a8_gemm(const W8a8GemmPlan &plan, const W8a8GemmArgs &args, const W8a8Tokens &tok, int64_t k,
                             uint8_t *ximg, int sm_count, cudaStream_t s)
{
    int m = args.m, np = args.np, H = plan.N / 2, halves = 2 * plan.ts;
    cudaError_t e;
    if (tok.Xq) {
        const int8_t *Xq = tok.Xq;
        void *kargs[] = {&Xq, &ximg, &m, &k, &np, &H, &halves};
        const int64_t blocks = ceil_div(static_cast<int64_t>(halves) * np * H * 4, 256);
        e = launch_pdl(reinterpret_cast<const void *>(&tile_kernel),
                       dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 8 * static_cast<int64_t>(sm_count)))), dim3(256),
                       0, s, kargs);
    } else {
        CodeTileArgs c{};
        c.X = tok.X;
        c.ldx = tok.ldx;
        c.ximg = ximg;
        c.sx = tok.sx;
        c.m = m;
        c.rows = halves * H;
        c.k = k;
        c.np = np;
        c.H = H;
        e = tok.xtype == Q4_TYPE_F32   ? launch_code_tiles<float>(c, tok.vec, sm_count, s)
            : tok.xtype == Q4_TYPE_F16 ? launch_code_tiles<__half>(c, tok.vec, sm_count, s)
                                       : launch_code_tiles<__nv_bfloat16>(c, tok.vec, sm_count, s);
    }
    if (e != cudaSuccess) return e;
    W8a8GemmArgs a = args;
    a.ximg = ximg;
    a.N = plan.N;
    a.ts = plan.ts;
    a.tiles = plan.tiles;
    a.kslices = plan.kslices;
    a.astages = plan.astages;
    a.bstages = plan.bstages;
    a.wring = plan.wring;
    const bool sliced = plan.kslices > 1;
    const int64_t rows = static_cast<int64_t>(a.groups) * kW8GroupRows;
    if (sliced) {
        a.Y = ximg + plan.image_bytes;
        a.ldy = rows;
        a.n = static_cast<int>(rows);
        a.ytype = Q4_TYPE_F32;
        a.slice_stride = static_cast<int64_t>(m) * rows;
    }
    const void *fn = kernel_of(a.ytype, sliced);
    e = set_max_smem(fn, plan.smem);
    if (e != cudaSuccess) return e;
    void *kargs[] = {&a};
    e = launch_pdl(fn, dim3(static_cast<unsigned>(2 * plan.pairs)), dim3(kThreads), plan.smem, s, kargs, 2);
    if (e != cudaSuccess || !sliced) return e;
    SliceSumArgs r{};
    r.partials = static_cast<const float *>(a.Y);
    r.ld = rows;
    r.stride = a.slice_stride;
    r.slices = plan.kslices;
    r.sx = args.sx;
    r.row_scale = args.row_scale;
    r.Y = args.Y;
    r.ldy = args.ldy;
    r.n = args.n;
    const int size = type_size(args.ytype);
    RowAlign al;
    al.add(args.Y, args.ldy * size);
    const bool wide = al.bytes() >= 4 * size;
    fn = args.ytype == Q4_TYPE_F32   ? wide ? reinterpret_cast<const void *>(&slice_sum_kernel<float, 4>) : reinterpret_cast<const void *>(&slice_sum_kernel<float, 1>)
         : args.ytype == Q4_TYPE_F16 ? wide ? reinterpret_cast<const void *>(&slice_sum_kernel<__half, 4>) : reinterpret_cast<const void *>(&slice_sum_kernel<__half, 1>)
         : wide                      ? reinterpret_cast<const void *>(&slice_sum_kernel<__nv_bfloat16, 4>)
                                     : reinterpret_cast<const void *>(&slice_sum_kernel<__nv_bfloat16, 1>);
    void *rargs[] = {&r};
    return launch_pdl(fn, dim3(static_cast<unsigned>(ceil_div(args.n, 256 * (wide ? 4 : 1))), static_cast<unsigned>(m)), dim3(256), 0,
                      s, rargs);
}

} // namespace q4
