// q4mm_w8a8_gemm.cu -- the int8 product for many tokens, on the 5th-generation
// tensor cores: Y[t][j] = sx[t] * s_j * sum_c xq[t][c] * code[j][c].
//
// sm_103a has no fast integer MMA; an int8 code is exact in fp16, so a product
// of codes is exact in the MMA and their sum is exact while it stays below
// 2^24 (fp32 accumulation). The MMA is bound by the fp16 rate: 2 m n k
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
//   4-11   dequantise, two sets of four warps on alternating K steps. A warp
//          that has stored its rows also waits for the step's B tile, then
//          arrives on the even CTA's `ready` barrier: one barrier covers both
//          operands of both CTAs.
//   12-19  epilogue: two warps per 32 rows, half of the token columns each.
// The MMA's commits release a stage (A and B) in both CTAs. A pair runs
// through tiles in turn: the rings carry on into the next tile while the
// epilogue reads D; only D's own read keeps the MMA waiting.
// Every wait is bounded; after a timeout all roles leave their loops, the
// MMAs and copies in flight are waited for and the CTAs of the pair leave
// together.
#include <algorithm>
#include <cuda_runtime.h>
#include <map>
#include <mutex>
#include <utility>

#include "q4mm_rows.cuh"
#include "q4mm_w8a8.h"

namespace q4 {
namespace {

constexpr int kErrTimeout = 5;
constexpr int kDequantWarp0 = 4, kDequantWarps = 8;
constexpr int kEpilogueWarp0 = 12, kEpilogueWarps = 8;
constexpr int kThreads = (kEpilogueWarp0 + kEpilogueWarps) * 32;
constexpr int kMaxStages = 8, kWRing = 8;

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

struct Smem {
    uint8_t *b, *w;
    uint64_t *full_b, *full_w, *empty_w, *ready, *empty, *d_full, *d_empty, *done;
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
__device__ __forceinline__ bool warp_wait_cluster(uint64_t *bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait_cluster(bar, parity, limit_ns)) != 0;
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

template <typename T> __global__ void __launch_bounds__(kThreads, 1) w8a8_gemm_kernel(const W8a8GemmArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = static_cast<int>(blockIdx.x) >> 1, pairs = static_cast<int>(gridDim.x) >> 1;
    const int N = a.N, H = N / 2, S = a.stages, RW = a.wring, np = a.np;
    const uint32_t bstage = static_cast<uint32_t>(H) * 128u;
    const uint32_t acol0 = static_cast<uint32_t>(N);   // first A column after D (N is a multiple of 32)

    Smem sm;
    sm.b = base;
    sm.w = sm.b + static_cast<size_t>(S) * bstage;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm.w + static_cast<size_t>(RW) * kW8RecordBytes);
    sm.full_b = bars;
    sm.ready = sm.full_b + S;
    sm.empty = sm.ready + S;
    sm.full_w = sm.empty + S;
    sm.empty_w = sm.full_w + RW;
    sm.d_full = sm.empty_w + RW;
    sm.d_empty = sm.d_full + 1;
    sm.done = sm.d_empty + 1;
    sm.tmem_slot = reinterpret_cast<uint32_t *>(sm.done + 1);
    sm.abort = reinterpret_cast<int *>(sm.tmem_slot + 1);
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&sm.full_b[i], 1);
            mbar_init(&sm.ready[i], kDequantWarps);     // a set's four warps in each CTA
            mbar_init(&sm.empty[i], 1);
        }
        for (int i = 0; i < RW; ++i) mbar_init(&sm.full_w[i], 1), mbar_init(&sm.empty_w[i], kDequantWarps / 2);
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
                const int jt = tile % a.ts;
                const uint8_t *src = a.ximg + (static_cast<size_t>(2 * jt) + rank) * np * bstage;
                for (int p = 0; p < np; ++p) {
                    if (aborted(sm)) { ok = false; break; }
                    if (issued >= S && !mbar_wait_cluster(&sm.empty[b.slot], b.phase ^ 1u, a.wait_ns)) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full_b[b.slot], bstage);
                    bulk_g2s(sm.b + static_cast<size_t>(b.slot) * bstage, src + static_cast<size_t>(p) * bstage, bstage,
                             &sm.full_b[b.slot]);
                    ++issued;
                    b.step(S);
                }
            }
            // after a timeout: what is still landing (all has been read otherwise)
            if (!ok)
                for (int64_t i = issued > S ? issued - S : 0; i < issued; ++i)
                    if (!mbar_wait(&sm.full_b[i % S], static_cast<uint32_t>(i / S) & 1u, a.wait_ns)) fail(sm, a);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------ record producer
        if (!a.prefetch_w) pdl_wait();
        if (lane == 0) {
            Ring w;
            int64_t issued = 0;
            bool ok = true;
            for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
                // the last pair of an odd number of groups: its second CTA
                // reads the last group again and writes nothing
                const int G = min(2 * (tile / a.ts) + static_cast<int>(rank), a.groups - 1);
                const uint8_t *src = a.W + static_cast<size_t>(G) * np * kW8RecordBytes;
                for (int p = 0; p < np; ++p) {
                    if (aborted(sm)) { ok = false; break; }
                    if (issued >= RW && !mbar_wait(&sm.empty_w[w.slot], w.phase ^ 1u, a.wait_ns)) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&sm.full_w[w.slot], kW8RecordBytes);
                    bulk_g2s(sm.w + static_cast<size_t>(w.slot) * kW8RecordBytes, src + static_cast<size_t>(p) * kW8RecordBytes,
                             kW8RecordBytes, &sm.full_w[w.slot]);
                    ++issued;
                    w.step(RW);
                }
            }
            if (!ok)
                for (int64_t i = issued > RW ? issued - RW : 0; i < issued; ++i)
                    if (!mbar_wait(&sm.full_w[i % RW], static_cast<uint32_t>(i / RW) & 1u, a.wait_ns)) fail(sm, a);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = idesc_f16_f32(256, static_cast<uint32_t>(N));
            const uint64_t bdesc0 = smem_desc_sw128(smem_u32(sm.b));
            const uint64_t bstep = static_cast<uint64_t>(bstage >> 4);
            Ring r;
            bool ok = true;
            uint32_t seq = 0;
            for (int tile = pair; ok && tile < a.tiles; tile += pairs, ++seq) {
                // D has been read out of both CTAs' tensor memory
                if (seq > 0 && !mbar_wait_cluster(sm.d_empty, (seq - 1) & 1u, a.wait_ns)) {
                    fail(sm, a);
                    break;
                }
                for (int p = 0; p < np; ++p) {
                    if (!mbar_wait_cluster(&sm.ready[r.slot], r.phase, a.wait_ns)) {
                        fail(sm, a);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t bd = bdesc0 + static_cast<uint64_t>(r.slot) * bstep;
                    const uint32_t at = tmem + acol0 + 32u * static_cast<uint32_t>(r.slot);
                    tc_mma_f16_ts_pair(tmem, at, bd, idesc, p > 0 ? 1u : 0u);
                    tc_mma_f16_ts_pair(tmem, at + 8u, bd + 2u, idesc, 1u);
                    tc_mma_f16_ts_pair(tmem, at + 16u, bd + 4u, idesc, 1u);
                    tc_mma_f16_ts_pair(tmem, at + 24u, bd + 6u, idesc, 1u);
                    tc_commit_pair(&sm.empty[r.slot], 3);
                    r.step(S);
                }
                if (ok) tc_commit_pair(sm.d_full, 3);
            }
            tc_commit_pair(sm.done, 3);   // also after a timeout
        }
        __syncwarp();
    } else if (dequant) {
        // --------------------------------------------------- dequantise W
        const int q = warp & 3, set = (warp - kDequantWarp0) >> 2;
        const int row = q * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        Ring w, r;
        uint32_t step = 0;
        bool ok = true;
        for (int tile = pair; ok && tile < a.tiles; tile += pairs) {
            for (int p = 0; p < np; ++p, ++step, w.step(RW), r.step(S)) {
                if (static_cast<int>(step & 1u) != set) continue;   // both rings are even: a slot has one set
                if (__any_sync(0xFFFFFFFFu, aborted(sm))) { ok = false; break; }
                if (!warp_wait(&sm.full_w[w.slot], w.phase, a.wait_ns) ||
                    (step >= static_cast<uint32_t>(S) && !warp_wait_cluster(&sm.empty[r.slot], r.phase ^ 1u, a.wait_ns))) {
                    fail(sm, a);
                    ok = false;
                    break;
                }
                // A row is four 16-byte chunks, rows 64 bytes apart: lanes reading
                // the same chunk would share two bank groups, four lanes each. So
                // lane l starts at chunk (l / 2) % 4, and the chunks are put back in
                // order by selects (registers take no index).
                const uint8_t *rec = sm.w + static_cast<size_t>(w.slot) * kW8RecordBytes + row * kPairK;
                const int rot = (lane >> 1) & 3;
                uint32_t u[16], out[32];
                {
                    uint32_t v[16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint4 x = lds128(rec + 16 * ((c + rot) & 3));
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
                tc_fence_after();
                tmem_st_32x32b_x32(tmem + lane_base + acol0 + static_cast<uint32_t>(r.slot) * 32u, out);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                bool landed = true;
                if (lane == 0) {
                    mbar_arrive(&sm.empty_w[w.slot]);
                    landed = mbar_wait(&sm.full_b[r.slot], r.phase, a.wait_ns);
                    if (landed) {
                        fence_proxy_async_smem();
                        mbar_arrive_remote(mapa_shared(smem_u32(&sm.ready[r.slot]), 0u));
                    }
                }
                if (!__shfl_sync(0xFFFFFFFFu, landed ? 1 : 0, 0)) {
                    fail(sm, a);
                    ok = false;
                    break;
                }
            }
        }
    } else if (warp >= kEpilogueWarp0) {
        // ------------------------------------------------------- epilogue
        pdl_wait();
        const int q = warp & 3, half = (warp - kEpilogueWarp0) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
        T *Y = static_cast<T *>(a.Y);
        uint32_t seq = 0;
        for (int tile = pair; tile < a.tiles; tile += pairs, ++seq) {
            const int G = 2 * (tile / a.ts) + static_cast<int>(rank);
            const int64_t row = static_cast<int64_t>(G) * kW8GroupRows + q * 32 + lane;
            const bool live = G < a.groups && row < a.n;
            const float sw = live ? __ldg(a.row_scale + row) : 0.0f;
            if (!warp_wait_cluster(sm.d_full, seq & 1u, a.wait_ns)) {
                fail(sm, a);
                break;
            }
            tc_fence_after();
            const int t0 = (tile % a.ts) * N;
            for (int c0 = half * H; c0 < half * H + H; c0 += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + lane_base + static_cast<uint32_t>(c0), v);
                tmem_wait_ld();
                if (c0 + 16 == half * H + H) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(sm.d_empty), 0u));
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = t0 + c0 + i;
                    if (t < a.m && live)
                        Y[t * a.ldy + row] = from_f32<T>(__uint_as_float(v[i]) * (__ldg(a.sx + t) * sw));
                }
            }
        }
    }

    // No MMA of the pair and none of its arrivals is in flight past this.
    __syncthreads();
    if (tid == 0 && !mbar_wait_cluster(sm.done, 0, a.wait_ns)) fail(sm, a);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // neither CTA's memory is used by the other past this
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512u);
}

const void *kernel_of(int ytype)
{
    return ytype == Q4_TYPE_F32   ? reinterpret_cast<const void *>(&w8a8_gemm_kernel<float>)
           : ytype == Q4_TYPE_F16 ? reinterpret_cast<const void *>(&w8a8_gemm_kernel<__half>)
                                  : reinterpret_cast<const void *>(&w8a8_gemm_kernel<__nv_bfloat16>);
}

size_t smem_bytes(int N, int stages, int wring)
{
    return 1024 + static_cast<size_t>(stages) * (N / 2) * 128 + static_cast<size_t>(wring) * kW8RecordBytes +
           static_cast<size_t>(3 * stages + 2 * wring + 3) * 8 + 16;
}

// CTA pairs that the current device holds at once; 0 when it cannot be asked.
int max_pairs(size_t smem)
{
    static std::mutex mu;
    static std::map<std::pair<int, size_t>, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    std::lock_guard<std::mutex> lock(mu);
    const auto it = cache.find({dev, smem});
    if (it != cache.end()) return it->second;
    int n = 0;
    const void *fn = kernel_of(Q4_TYPE_F32);
    if (set_max_smem(fn, smem) == cudaSuccess) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) n = 0;
    }
    cudaGetLastError();
    cache.emplace(std::make_pair(dev, smem), n);
    return n;
}

} // namespace

// Tokens a tile: the fewest clocks over the pairs' turns. A K step takes 2 N
// clocks of MMA (256 x N x 64 at 8192 products a clock and pair), but not
// under the 300 or so in which a step's operands are prepared; a tile adds
// its first step's latency and D's read.
bool plan_w8a8_gemm(int64_t m, int64_t k, int64_t n, W8a8GemmPlan *plan)
{
    const int64_t np = ceil_div(k, kPairK), rt = ceil_div(ceil_div(n, kW8GroupRows), 2);
    double best = 1e300;
    W8a8GemmPlan out;
    for (int N = 32; N <= 256; N += 32) {
        W8a8GemmPlan c;
        c.N = N;
        c.stages = std::min(kMaxStages, (512 - N) / 32) & ~1;
        c.wring = kWRing;
        c.smem = std::max<size_t>(smem_bytes(N, c.stages, c.wring), kSmemPerSM / 2 + 1024);   // one CTA per SM
        if (c.smem > kSmemOptIn) continue;
        c.ts = static_cast<int>(ceil_div(m, N));
        if (rt * c.ts > (int64_t(1) << 30)) continue;
        c.tiles = static_cast<int>(rt * c.ts);
        const int held = max_pairs(c.smem);
        if (held < 1) continue;
        c.pairs = std::min(held, c.tiles);
        c.image_bytes = static_cast<size_t>(2) * c.ts * np * (N / 2) * 128;
        const double turns = static_cast<double>(ceil_div(c.tiles, c.pairs));
        const double cost = turns * (static_cast<double>(np) * std::max(2.0 * N, 300.0) + 1000.0 + 4.0 * N);
        if (cost < best) {
            best = cost;
            out = c;
        }
    }
    if (out.N == 0) return false;
    *plan = out;
    return true;
}

cudaError_t launch_w8a8_gemm(const W8a8GemmPlan &plan, const W8a8GemmArgs &args, const int8_t *Xq, int64_t k,
                             uint8_t *ximg, int sm_count, cudaStream_t s)
{
    int m = args.m, np = args.np, H = plan.N / 2, halves = 2 * plan.ts;
    {
        void *kargs[] = {&Xq, &ximg, &m, &k, &np, &H, &halves};
        const int64_t blocks = ceil_div(static_cast<int64_t>(halves) * np * H * 4, 256);
        const cudaError_t e = launch_pdl(reinterpret_cast<const void *>(&tile_kernel),
                                         dim3(static_cast<unsigned>(std::min<int64_t>(blocks, 8 * static_cast<int64_t>(sm_count)))),
                                         dim3(256), 0, s, kargs);
        if (e != cudaSuccess) return e;
    }
    W8a8GemmArgs a = args;
    a.ximg = ximg;
    a.N = plan.N;
    a.ts = plan.ts;
    a.tiles = plan.tiles;
    a.stages = plan.stages;
    a.wring = plan.wring;
    const void *fn = kernel_of(a.ytype);
    const cudaError_t e = set_max_smem(fn, plan.smem);
    if (e != cudaSuccess) return e;
    void *kargs[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(2 * plan.pairs)), dim3(kThreads), plan.smem, s, kargs, 2);
}

} // namespace q4
