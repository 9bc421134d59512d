// q4mm_norm_stream.cu -- the norms over many rows of whole 16-byte vectors (the
// mathematics is in q4mm_norm.cu). A CTA takes rows in turn. Its first thread
// keeps bulk copies of the rows to come in flight, into a ring in shared memory,
// so the memory is busy while a row's sums meet at a barrier; loads into
// registers leave it idle then, and there are not enough registers to load far
// ahead. Both passes over a row, its sums and its results, read it from shared
// memory; past the barrier of a row's first sum every thread is done with the
// row before, whose slot is then refilled. The channels' weights, and backward
// their sums, stay in registers over the rows.
//   Every wait is bounded: after one that ran out the status word says so, the
// CTA goes through its rows without waiting (its results are void) and leaves
// when the copies in flight have landed.
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_norm.cuh"

namespace q4 {
namespace {

constexpr int kErrTimeout = 5;
constexpr int kMatrices = 3;

// The rows first, first + step, ... of up to three matrices.
struct RowStream {
    uint8_t *buf;
    uint64_t *full;
    int stages, used;
    uint32_t bytes;                  // of a row
    const uint8_t *src[kMatrices];
    int64_t ld[kMatrices];           // bytes
    int64_t m;
    int *status;
    uint64_t wait_ns;
    bool dead;

    __device__ __forceinline__ void issue(int64_t row, int slot)
    {
        mbar_arrive_expect_tx(&full[slot], bytes * used);
        uint8_t *dst = buf + static_cast<size_t>(slot) * used * bytes;
        for (int i = 0; i < used; ++i) bulk_g2s(dst + static_cast<size_t>(i) * bytes, src[i] + row * ld[i], bytes, &full[slot]);
    }
    __device__ __forceinline__ void start()
    {
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
            fence_barrier_init();
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < stages; ++i) {
                const int64_t row = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
                if (row < m) issue(row, i);
            }
    }
    __device__ __forceinline__ void wait(int slot, uint32_t phase)
    {
        if (!dead && !mbar_wait(&full[slot], phase, wait_ns)) {
            dead = true;
            record_status(status, kErrTimeout);
        }
    }
    // past the barrier of `row`'s first sum: refill the slot of the row before
    __device__ __forceinline__ void refill_before(int64_t row, int slot)
    {
        const int64_t next = row + static_cast<int64_t>(stages - 1) * gridDim.x;
        if (threadIdx.x == 0 && row >= static_cast<int64_t>(gridDim.x) && next < m && !dead)
            issue(next, slot == 0 ? stages - 1 : slot - 1);
    }
    // after a timeout: what is still landing
    __device__ __forceinline__ void finish(int slot, uint32_t phase)
    {
        if (!__syncthreads_or(dead ? 1 : 0) || threadIdx.x != 0) return;
        for (int i = 0; i < stages; ++i) {
            // a slot's last copy completes the phase that its wait would have been for
            mbar_wait(&full[slot], phase, wait_ns);
            if (++slot == stages) slot = 0, phase ^= 1u;
        }
    }
    // the vector at element c
    template <typename T, int V> __device__ __forceinline__ Pack<T, V> get(int slot, int matrix, int c) const
    {
        const uint4 v = lds128(buf + (static_cast<size_t>(slot) * used + matrix) * bytes + static_cast<size_t>(c) * sizeof(T));
        Pack<T, V> p;
        p.w[0] = v.x, p.w[1] = v.y, p.w[2] = v.z, p.w[3] = v.w;
        return p;
    }
};

template <typename T>
__device__ __forceinline__ RowStream make_stream(uint8_t *smem, int64_t m, int64_t d, int stages, int used, int *status,
                                                 uint64_t wait_ns)
{
    RowStream r{};
    r.bytes = static_cast<uint32_t>(d * sizeof(T));
    r.stages = stages;
    r.used = used;
    r.buf = smem;
    r.full = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(stages) * used * r.bytes);
    r.m = m;
    r.status = status;
    r.wait_ns = wait_ns;
    return r;
}

// Slot and phase of the row being worked on.
struct Turn {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++slot == stages) slot = 0, phase ^= 1u;
    }
};

// Up to 256 threads three CTAs fit on an SM's registers, else one of 512.
#define Q4_STREAM_BOUNDS __launch_bounds__(BIG ? 512 : 256, BIG ? 1 : 3)

template <typename T, int NV, bool BIG>
__global__ void Q4_STREAM_BOUNDS norm_after_stream_kernel(const NormAfterArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const bool full = a.gate_kind == Q4_GATE_FULL;
    const int d = static_cast<int>(a.d);
    RowStream rs = make_stream<T>(smem, a.m, a.d, stages, full ? 3 : 2, a.status, a.wait_ns);
    rs.src[0] = static_cast<const uint8_t *>(a.B), rs.ld[0] = a.ldb * sizeof(T);
    rs.src[1] = static_cast<const uint8_t *>(a.R), rs.ld[1] = a.ldr * sizeof(T);
    rs.src[2] = static_cast<const uint8_t *>(a.gate), rs.ld[2] = a.ldg * sizeof(T);
    rs.start();
    const RowGroup g = row_group(static_cast<int>(blockDim.x));
    RowReducer red{rbuf, static_cast<int>(blockDim.x) / 32};
    const auto after_at = [&](int c, float (&w)[V]) {
        channel_weights<V>(a.w, a.w_off, c, d, w);
        if (a.gate_kind == Q4_GATE_CHANNEL) {
            float gc[V];
            load_params<V>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    Channels<V, NV, true> wa, wo;
    wa.fill(g, after_at);
    if (a.out.H) wo.fill(g, [&](int c, float (&w)[V]) { channel_weights<V>(a.out.w, a.out.w_off, c, d, w); });
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        rs.wait(turn.slot, turn.phase);
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c < d) s[0] = square_sum<T, V>(rs.get<T, V>(turn.slot, 0, c), s[0]);
        }
        red.sum(s);
        rs.refill_before(row, turn.slot);
        float q = a.scale / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        if (a.gate_kind == Q4_GATE_TOKEN) q *= static_cast<const float *>(a.gate)[row];
        T *yr = static_cast<T *>(a.Y) + row * a.ldy;
        s[0] = 0.0f;
        Pack<T, V> r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), rv = rs.get<T, V>(turn.slot, 1, c);
            float w[V], y[V];
            wa.get(i, c, after_at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = elem(bv, j) * q * w[j];
            if (full) {
                const Pack<T, V> gv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] *= elem(gv, j);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] += elem(rv, j);
            r[i] = pack_of<T, V>(y);
            store_pack<T, V>(yr, c, d, r[i]);
            s[0] = square_sum<T, V>(r[i], s[0]);
        }
        if (a.out.H) {
            red.sum(s);
            const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.out_eps);
            write_normed<T, V, NV, true>(r, [&](int c) { return load_pack<T, V>(yr, c, d); }, rho, a.out, wo, row, g, d, red);
        }
    }
    rs.finish(turn.slot, turn.phase);
}

template <typename T, int NV, bool BIG>
__global__ void Q4_STREAM_BOUNDS norm_before_bwd_stream_kernel(const NormBeforeBwdArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const bool residual = a.dR != nullptr;
    const int d = static_cast<int>(a.d);
    RowStream rs = make_stream<T>(smem, a.m, a.d, stages, residual ? 3 : 2, a.status, a.wait_ns);
    rs.src[0] = static_cast<const uint8_t *>(a.X), rs.ld[0] = a.ldx * sizeof(T);
    rs.src[1] = static_cast<const uint8_t *>(a.dH), rs.ld[1] = a.lddh * sizeof(T);
    rs.src[2] = static_cast<const uint8_t *>(a.dR), rs.ld[2] = a.lddr * sizeof(T);
    rs.start();
    const RowGroup g = row_group(static_cast<int>(blockDim.x));
    RowReducer red{rbuf, static_cast<int>(blockDim.x) / 32};
    const auto at = [&](int c, float (&w)[V]) { channel_weights<V>(a.w, a.w_off, c, d, w); };
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    float acc[NV][V] = {};
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        rs.wait(turn.slot, turn.phase);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            const Pack<T, V> xv = rs.get<T, V>(turn.slot, 0, c), hv = rs.get<T, V>(turn.slot, 1, c);
            float w[V];
            wc.get(i, c, at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = elem(xv, j);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(elem(hv, j) * w[j], f, s[1]);
            }
        }
        red.sum(s);
        rs.refill_before(row, turn.slot);
        const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        const float mean = rho * s[1] / static_cast<float>(d);
        T *out = static_cast<T *>(a.dX) + row * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            const Pack<T, V> xv = rs.get<T, V>(turn.slot, 0, c), hv = rs.get<T, V>(turn.slot, 1, c);
            float w[V], o[V];
            wc.get(i, c, at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = elem(xv, j) * rho, h = elem(hv, j);
                acc[i][j] = fmaf(h, u, acc[i][j]);
                o[j] = rho * (h * w[j] - u * mean);
            }
            if (residual) {
                const Pack<T, V> rv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += elem(rv, j);
            }
            store_pack<T, V>(out, c, d, pack_of<T, V>(o));
        }
    }
    rs.finish(turn.slot, turn.phase);
    if (a.partials) write_partials<V, NV>(acc, a.partials, g, d, nullptr);
}

template <typename T, int NV, bool BIG>
__global__ void Q4_STREAM_BOUNDS norm_after_bwd_stream_kernel(const NormAfterBwdArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const bool full = a.gate_kind == Q4_GATE_FULL, token = a.gate_kind == Q4_GATE_TOKEN;
    const int d = static_cast<int>(a.d);
    RowStream rs = make_stream<T>(smem, a.m, a.d, stages, full ? 3 : 2, a.status, a.wait_ns);
    rs.src[0] = static_cast<const uint8_t *>(a.B), rs.ld[0] = a.ldb * sizeof(T);
    rs.src[1] = static_cast<const uint8_t *>(a.dY), rs.ld[1] = a.lddy * sizeof(T);
    rs.src[2] = static_cast<const uint8_t *>(a.gate), rs.ld[2] = a.ldg * sizeof(T);
    rs.start();
    const RowGroup g = row_group(static_cast<int>(blockDim.x));
    RowReducer red{rbuf, static_cast<int>(blockDim.x) / 32};
    // (o + w), times the channel's gate
    const auto at = [&](int c, float (&w)[V]) {
        channel_weights<V>(a.w, a.w_off, c, d, w);
        if (a.gate_kind == Q4_GATE_CHANNEL) {
            float gc[V];
            load_params<V>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    float acc[NV][V] = {};
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        const float gtok = token ? static_cast<const float *>(a.gate)[row] : 1.0f;
        rs.wait(turn.slot, turn.phase);
        // sums of b^2 and of g w dy b (a token's gate is taken out: its gradient is
        // that sum)
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), yv = rs.get<T, V>(turn.slot, 1, c);
            float w[V];
            wc.get(i, c, at, w);
            if (full) {
                const Pack<T, V> gv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V; ++j) w[j] *= elem(gv, j);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = elem(bv, j);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(elem(yv, j) * w[j], f, s[1]);
            }
        }
        red.sum(s);
        rs.refill_before(row, turn.slot);
        const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        if (token && a.dgate && g.t == 0) static_cast<float *>(a.dgate)[row] = a.scale * rho * s[1];
        const float mean = gtok * rho * s[1] / static_cast<float>(d), q = a.scale * rho;
        T *out = static_cast<T *>(a.dB) + row * a.lddb;
        T *dgr = full && a.dgate ? static_cast<T *>(a.dgate) + row * a.lddg : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), yv = rs.get<T, V>(turn.slot, 1, c);
            float w[V], o[V];
            wc.get(i, c, at, w);
            if (dgr) {
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] = a.scale * elem(yv, j) * (elem(bv, j) * rho) * w[j];
                store_pack<T, V>(dgr, c, d, pack_of<T, V>(o));
            }
            Pack<T, V> gv = zero_pack<T, V>();
            if (full) gv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = elem(bv, j) * rho, gy = elem(yv, j) * (full ? elem(gv, j) : gtok);
                // the channel's gate, like s, is a factor of the whole column
                acc[i][j] = fmaf(gy, u, acc[i][j]);
                o[j] = q * (gy * w[j] - u * mean);
            }
            store_pack<T, V>(out, c, d, pack_of<T, V>(o));
        }
    }
    rs.finish(turn.slot, turn.phase);
    if (a.partials) write_partials<V, NV>(acc, a.partials, g, d, nullptr);
}

template <typename T, int NV, bool BIG> struct AfterStream {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_stream_kernel<T, NV, BIG>); }
};
template <typename T, int NV, bool BIG> struct BeforeBwdStream {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_before_bwd_stream_kernel<T, NV, BIG>); }
};
template <typename T, int NV, bool BIG> struct AfterBwdStream {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_bwd_stream_kernel<T, NV, BIG>); }
};

template <template <typename, int, bool> class K, typename T> const void *stream_fn(const NormStreamPlan &p)
{
    if (p.G > 256) return p.NV == 2 ? K<T, 2, true>::fn() : K<T, 4, true>::fn();
    return p.NV == 1 ? K<T, 1, false>::fn() : p.NV == 2 ? K<T, 2, false>::fn() : K<T, 4, false>::fn();
}
template <template <typename, int, bool> class K, typename Args>
cudaError_t launch_stream(const NormStreamPlan &p, Args a, int type, cudaStream_t s)
{
    const void *fn = type == Q4_TYPE_F32   ? stream_fn<K, float>(p)
                     : type == Q4_TYPE_F16 ? stream_fn<K, __half>(p)
                                           : stream_fn<K, __nv_bfloat16>(p);
    const cudaError_t e = set_max_smem(fn, p.smem);
    if (e != cudaSuccess) return e;
    a.G = p.G;
    int stages = p.stages;
    void *args[] = {&a, &stages};
    return launch_pdl(fn, dim3(static_cast<unsigned>(p.ctas)), dim3(static_cast<unsigned>(p.G)), p.smem, s, args);
}

} // namespace

bool plan_norm_stream(int64_t m, int64_t d, int type, int matrices, int sm_count, NormStreamPlan *plan)
{
    const int size = type_size(type), V = 16 / size;
    const int64_t bytes = d * size, vecs = d / V;
    // a row under 1 KB is a warp's; with fewer rows than CTAs nothing is read ahead
    if (bytes % 16 != 0 || bytes < 1024 || vecs > 2048 || m <= 2 * sm_count) return false;
    NormStreamPlan p;
    const int most = size == 2 ? 2 : 4;   // vectors whose weights stay in registers
    p.NV = vecs <= 256 ? 1 : vecs <= 512 ? 2 : vecs <= 1024 ? most : 4;
    p.G = static_cast<int>(round_up(ceil_div(vecs, p.NV), 32));
    const size_t stage = static_cast<size_t>(matrices) * bytes + 8;
    int per_sm = p.G > 256 ? 1 : 3;
    for (; per_sm > 0; --per_sm) {
        p.stages = static_cast<int>(std::min<size_t>(4, (kSmemPerSM / per_sm - 2048) / stage));
        if (p.stages >= 3) break;
    }
    if (per_sm == 0) return false;
    p.smem = stage * p.stages;
    if (p.smem > kSmemOptIn - 1024) return false;
    p.ctas = std::min<int64_t>(m, std::min<int64_t>(kNormPartials, static_cast<int64_t>(sm_count) * per_sm));
    *plan = p;
    return true;
}

cudaError_t launch_norm_after_stream(const NormStreamPlan &p, const NormAfterArgs &a, int type, cudaStream_t s)
{
    return launch_stream<AfterStream>(p, a, type, s);
}
cudaError_t launch_norm_before_bwd_stream(const NormStreamPlan &p, const NormBeforeBwdArgs &a, int type, cudaStream_t s)
{
    return launch_stream<BeforeBwdStream>(p, a, type, s);
}
cudaError_t launch_norm_after_bwd_stream(const NormStreamPlan &p, const NormAfterBwdArgs &a, int type, cudaStream_t s)
{
    return launch_stream<AfterBwdStream>(p, a, type, s);
}

} // namespace q4
