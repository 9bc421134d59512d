// q4mm_norm_stream.cuh -- the norms over many rows (the mathematics is in
// q4mm_norm.cu); q4mm_norm_stream.cu has those whose rows start on 16 bytes,
// q4mm_norm_stream_any.cu the others. A CTA takes rows in turn. A warp of its own
// keeps bulk copies of the rows to come in flight, into a ring in shared memory,
// so the memory is busy while a row's sums meet at a barrier; loads into
// registers leave it idle then, and there are not enough registers to load far
// ahead. (Issued by one of the row's threads, the copies held up the others at
// each row's barrier.)
//   Both passes over a row, its sums and its results, read it from shared memory;
// then the row's warps release its slot. The channels' weights, and backward
// their sums, stay in registers over the rows. What bounds a CTA then is the way
// of a row (sums, barrier, root, results) and its instructions, two CTAs an SM
// side by side; packed fp32 arithmetic took a fifth off them. Two rows at once a
// CTA, three CTAs an SM with the weights in shared memory, and more rows ahead
// measured no faster.
//   GB300, us a call (floor at the measured copy rate): join 4096 x 4096 bf16 with
// a gate for each value 30 (25), fp32 52 (40); gradient before 8192 x 4096 bf16 47
// (40), 2049 x 2560 fp32 20 (12); after 8192 x 4096 bf16, channel gate 45 (30), a
// gate for each value 58 (50). On odd boundaries: join 4000 x 4097 bf16 36 (19), fp32
// 51 (39), gradients before 4000 x 4097 bf16 33 (19), after 3000 x 2561 fp32 24 (14).
//   Every wait is bounded: after one that ran out the status word says so and the
// thread goes through its rows without waiting (the call's results are void) and
// without giving slots back, so the copying warp's own wait runs out too; the CTA
// leaves when the copies in flight have landed.
#pragma once

#include "q4mm_norm.cuh"

namespace q4 {
namespace {

constexpr int kErrTimeout = 5;
constexpr int kMatrices = 3;

// The rows blockIdx.x, + gridDim.x, ... of up to three matrices.
struct RowStream {
    uint8_t *buf;
    uint64_t *full, *empty;          // [stages] each
    int stages, used;
    uint32_t bytes, copied;          // a row's place in a slot; what is copied to it
    int skew;                        // bytes of a place before its row
    const uint8_t *src[kMatrices];
    int64_t ld[kMatrices];           // bytes
    int64_t m;
    int *status;
    uint64_t wait_ns;
    bool dead;

    // the whole CTA, once
    __device__ __forceinline__ void start(int row_warps)
    {
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], row_warps);
            fence_barrier_init();
        }
        __syncthreads();
    }
    // the copying warp's one thread: every row of the CTA, until all have landed
    __device__ __forceinline__ void copy_rows()
    {
        int slot = 0;
        uint32_t phase = 0;
        int64_t issued = 0;
        for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
            if (issued >= stages && !mbar_wait(&empty[slot], phase ^ 1u, wait_ns)) {
                record_status(status, kErrTimeout);
                break;
            }
            mbar_arrive_expect_tx(&full[slot], copied * used);
            uint8_t *dst = buf + static_cast<size_t>(slot) * used * bytes;
            for (int i = 0; i < used; ++i) bulk_g2s(dst + static_cast<size_t>(i) * bytes, src[i] + row * ld[i], copied, &full[slot]);
            ++issued;
            if (++slot == stages) slot = 0, phase ^= 1u;
        }
        for (int64_t k = issued > stages ? issued - stages : 0; k < issued; ++k)
            mbar_wait(&full[k % stages], static_cast<uint32_t>(k / stages) & 1u, landing_limit(wait_ns));
    }
    __device__ __forceinline__ void wait(int slot, uint32_t phase)
    {
        if (!dead && !mbar_wait(&full[slot], phase, wait_ns)) {
            dead = true;
            record_status(status, kErrTimeout);
        }
    }
    // A row's warp has read the slot for the last time. Only a lane that saw the
    // slot's copies land gives it back: a slot given back before that would be armed
    // for another row while the first is still on its way.
    __device__ __forceinline__ void release(int slot)
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0 && !dead) mbar_arrive(&empty[slot]);
    }
    __device__ __forceinline__ const uint8_t *place(int slot, int matrix) const
    {
        return buf + (static_cast<size_t>(slot) * used + matrix) * bytes + skew;
    }
    // the vector at element c, and an element
    template <typename T, int V> __device__ __forceinline__ Pack<T, V> get(int slot, int matrix, int c) const
    {
        const uint4 v = lds128(place(slot, matrix) + static_cast<size_t>(c) * sizeof(T));
        Pack<T, V> p;
        p.w[0] = v.x, p.w[1] = v.y, p.w[2] = v.z, p.w[3] = v.w;
        return p;
    }
    template <typename T> __device__ __forceinline__ float one(int slot, int matrix, int c) const
    {
        return load_elem(reinterpret_cast<const T *>(place(slot, matrix)), c);
    }
};

// A matrix that is streamed.
struct StreamSource {
    const void *p;
    int64_t ld;   // elements
};
// A CTA's rows start alike (its step is a multiple of kRowStep), in every matrix.
// Where that is not at 16 bytes, the aligned words that hold some of a row are
// copied: each lies in the row's allocation.
template <typename T, bool ANY>
__device__ __forceinline__ RowStream make_stream(uint8_t *smem, const StreamSource (&in)[kMatrices], int64_t m, int d,
                                                 int stages, int used, int *status, uint64_t wait_ns)
{
    RowStream r{};
    r.skew = ANY ? static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T *>(in[0].p) + blockIdx.x * in[0].ld) & 15) : 0;
    r.copied = static_cast<uint32_t>(d * sizeof(T) + r.skew + (ANY ? 15 : 0)) & ~15u;
    r.bytes = ANY ? static_cast<uint32_t>(d * sizeof(T) + 30 - sizeof(T)) / 16 * 16 : r.copied;
    r.stages = stages;
    r.used = used;
    r.buf = smem;
    r.full = reinterpret_cast<uint64_t *>(smem + static_cast<size_t>(stages) * used * r.bytes);
    r.empty = r.full + stages;
    for (int i = 0; i < kMatrices; ++i) {
        r.src[i] = static_cast<const uint8_t *>(in[i].p) - r.skew;
        r.ld[i] = in[i].ld * static_cast<int64_t>(sizeof(T));
    }
    r.m = m;
    r.status = status;
    r.wait_ns = wait_ns;
    return r;
}

// The weights of vector i as pairs.
template <int V, int NV, typename F>
__device__ __forceinline__ void weight_pairs(const Channels<V, NV, true> &ch, int i, int c, F at, F2 (&w)[V / 2])
{
    float f[V];
    ch.get(i, c, at, f);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) w[j] = f2(f[2 * j], f[2 * j + 1]);
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

// Threads of rows and a warp that copies; two CTAs of up to 256 fit on an SM's
// registers, or one of 512.
#define Q4_STREAM_BOUNDS __launch_bounds__((BIG ? 512 : 256) + 32, BIG ? 1 : 2)

template <typename T, int NV, bool BIG, bool ANY, bool full>
__global__ void Q4_STREAM_BOUNDS norm_after_stream_kernel(const NormAfterArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const StreamSource in[kMatrices] = {{a.B, a.ldb}, {a.R, a.ldr}, {a.gate, a.ldg}};
    RowStream rs = make_stream<T, ANY>(smem, in, a.m, d, stages, full ? 3 : 2, a.status, a.wait_ns);
    RowReducer red{rbuf, a.G / 32, true};
    red.clear(static_cast<int>(blockDim.x));
    rs.start(a.G / 32);
    if (static_cast<int>(threadIdx.x) >= a.G) {
        if (static_cast<int>(threadIdx.x) == a.G) rs.copy_rows();
        return;
    }
    RowGroup g{static_cast<int>(threadIdx.x), a.G, blockIdx.x, gridDim.x};
    g.begin<ANY>(static_cast<const T *>(in[0].p) + g.row * in[0].ld, d);   // the same in all of its rows
    const auto after_at = [&](int c, float (&w)[V]) {
        channel_weights<V, ANY>(a.w, a.w_off, c, d, w);
        if (a.gate_kind == Q4_GATE_CHANNEL) {
            float gc[V];
            load_params<V, ANY>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    float wl = 0.0f;   // of the element outside the vectors
    if (g.loose >= 0) {
        wl = channel_weight(a.w, a.w_off, g.loose);
        if (a.gate_kind == Q4_GATE_CHANNEL) wl *= static_cast<const float *>(a.gate)[g.loose];
    }
    Channels<V, NV, true> wa, wo;
    wa.fill(g, after_at);
    if (a.out.H) wo.fill(g, [&](int c, float (&w)[V]) { channel_weights<V, ANY>(a.out.w, a.out.w_off, c, d, w); });
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        rs.wait(turn.slot, turn.phase);
        F2 sq = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) sq = f2_fma(pair(bv, j), pair(bv, j), sq);
        }
        float alone = g.loose >= 0 ? rs.one<T>(turn.slot, 0, g.loose) : 0.0f;
        float s[1] = {fmaf(alone, alone, f2_sum(sq))};
        red.sum(s);
        Pack<T, V> r[NV];
        float f = a.scale * rms_factor(s[0], inv_d, a.eps);
        if (a.gate_kind == Q4_GATE_TOKEN) f *= static_cast<const float *>(a.gate)[row];
        T *yr = static_cast<T *>(a.Y) + row * a.ldy;
        const F2 ff = f2(f, f);
        sq = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), rv = rs.get<T, V>(turn.slot, 1, c);
            F2 w[V / 2], y[V / 2];
            weight_pairs<V, NV>(wa, i, c, after_at, w);
            if constexpr (full) {
                const Pack<T, V> gv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) w[j] = f2_mul(w[j], pair(gv, j));
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) y[j] = f2_fma(f2_mul(pair(bv, j), ff), w[j], pair(rv, j));
            r[i] = pack_pairs<T, V>(y);
            store_pack<T, V>(yr, c, d, r[i]);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) sq = f2_fma(pair(r[i], j), pair(r[i], j), sq);
        }
        s[0] = f2_sum(sq);
        if (g.loose >= 0) {
            alone = alone * f * wl;
            if constexpr (full) alone *= rs.one<T>(turn.slot, 2, g.loose);
            alone = store_elem(yr, g.loose, rs.one<T>(turn.slot, 1, g.loose) + alone);
            s[0] = fmaf(alone, alone, s[0]);
        }
        rs.release(turn.slot);
        if (!a.out.H) continue;
        red.sum(s);
        write_normed<T, V, NV, true, ANY>(r, [&](int c) { return load_pack<T, V>(yr, c, d); }, alone, rms_factor(s[0], inv_d, a.out_eps),
                                     a.out, wo, row, g, d, red);
    }
}

template <typename T, int NV, bool BIG, bool ANY>
__global__ void Q4_STREAM_BOUNDS norm_before_bwd_stream_kernel(const NormBeforeBwdArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    const bool residual = a.dR != nullptr;
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const StreamSource in[kMatrices] = {{a.X, a.ldx}, {a.dH, a.lddh}, {a.dR, a.lddr}};
    RowStream rs = make_stream<T, ANY>(smem, in, a.m, d, stages, residual ? 3 : 2, a.status, a.wait_ns);
    RowReducer red{rbuf, a.G / 32, true};
    red.clear(static_cast<int>(blockDim.x));
    rs.start(a.G / 32);
    if (static_cast<int>(threadIdx.x) >= a.G) {
        if (static_cast<int>(threadIdx.x) == a.G) rs.copy_rows();
        return;
    }
    RowGroup g{static_cast<int>(threadIdx.x), a.G, blockIdx.x, gridDim.x};
    g.begin<ANY>(static_cast<const T *>(in[0].p) + g.row * in[0].ld, d);   // the same in all of its rows
    const auto at = [&](int c, float (&w)[V]) { channel_weights<V, ANY>(a.w, a.w_off, c, d, w); };
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    // of the element outside the vectors
    const float wl = g.loose >= 0 ? channel_weight(a.w, a.w_off, g.loose) : 0.0f;
    float alone = 0.0f;
    F2 acc[NV][V / 2] = {};
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        float s[2];   // of x^2 and of dn x
        rs.wait(turn.slot, turn.phase);
        F2 sq = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> xv = rs.get<T, V>(turn.slot, 0, c), hv = rs.get<T, V>(turn.slot, 1, c);
            F2 w[V / 2];
            weight_pairs<V, NV>(wc, i, c, at, w);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 f = pair(xv, j);
                sq = f2_fma(f, f, sq);
                dot = f2_fma(f2_mul(pair(hv, j), w[j]), f, dot);
            }
        }
        s[0] = f2_sum(sq), s[1] = f2_sum(dot);
        float xa = 0.0f, ha = 0.0f;
        if (g.loose >= 0) {
            xa = rs.one<T>(turn.slot, 0, g.loose), ha = rs.one<T>(turn.slot, 1, g.loose);
            s[0] = fmaf(xa, xa, s[0]), s[1] = fmaf(ha * wl, xa, s[1]);
        }
        red.sum(s);
        // dx = rho dn - x rho^2 mean [+ dr], mean = rho sum(dn x) / d
        const float rho = rms_factor(s[0], inv_d, a.eps), mean = rho * s[1] * inv_d;
        const F2 rho2 = f2(rho, rho), back = f2(-rho * mean * rho, -rho * mean * rho);
        T *out = static_cast<T *>(a.dX) + row * a.lddx;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> xv = rs.get<T, V>(turn.slot, 0, c), hv = rs.get<T, V>(turn.slot, 1, c);
            F2 w[V / 2], o[V / 2];
            weight_pairs<V, NV>(wc, i, c, at, w);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 x = pair(xv, j), h = f2_mul(pair(hv, j), rho2);
                acc[i][j] = f2_fma(h, x, acc[i][j]);
                o[j] = f2_fma(h, w[j], f2_mul(x, back));
            }
            if (residual) {
                const Pack<T, V> rv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) o[j] = f2_fma(o[j], f2(1.0f, 1.0f), pair(rv, j));
            }
            store_pack<T, V>(out, c, d, pack_pairs<T, V>(o));
        }
        if (g.loose >= 0) {
            const float h = ha * rho;
            alone = fmaf(h, xa, alone);
            const float o = h * wl - xa * (rho * mean * rho);
            store_elem(out, g.loose, residual ? o + rs.one<T>(turn.slot, 2, g.loose) : o);
        }
        rs.release(turn.slot);
    }
    if (a.partials) {
        float sums[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) f2_split(acc[i][j], sums[i][2 * j], sums[i][2 * j + 1]);
        write_partials<V, NV, ANY>(sums, alone, a.partials, g, d, nullptr);
    }
}

template <typename T, int NV, bool BIG, bool ANY, bool full>
__global__ void Q4_STREAM_BOUNDS norm_after_bwd_stream_kernel(const NormAfterBwdArgs a, int stages)
{
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    const bool token = a.gate_kind == Q4_GATE_TOKEN;
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const StreamSource in[kMatrices] = {{a.B, a.ldb}, {a.dY, a.lddy}, {a.gate, a.ldg}};
    RowStream rs = make_stream<T, ANY>(smem, in, a.m, d, stages, full ? 3 : 2, a.status, a.wait_ns);
    RowReducer red{rbuf, a.G / 32, true};
    red.clear(static_cast<int>(blockDim.x));
    rs.start(a.G / 32);
    if (static_cast<int>(threadIdx.x) >= a.G) {
        if (static_cast<int>(threadIdx.x) == a.G) rs.copy_rows();
        return;
    }
    RowGroup g{static_cast<int>(threadIdx.x), a.G, blockIdx.x, gridDim.x};
    g.begin<ANY>(static_cast<const T *>(in[0].p) + g.row * in[0].ld, d);   // the same in all of its rows
    // s (o + w), times the channel's gate
    const auto at = [&](int c, float (&w)[V]) {
        channel_weights<V, ANY>(a.w, a.w_off, c, d, w);
#pragma unroll
        for (int j = 0; j < V; ++j) w[j] *= a.scale;
        if (a.gate_kind == Q4_GATE_CHANNEL) {
            float gc[V];
            load_params<V, ANY>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    float wl = 0.0f, alone = 0.0f;   // of the element outside the vectors
    if (g.loose >= 0) {
        wl = channel_weight(a.w, a.w_off, g.loose) * a.scale;
        if (a.gate_kind == Q4_GATE_CHANNEL) wl *= static_cast<const float *>(a.gate)[g.loose];
    }
    F2 acc[NV][V / 2] = {};
    Turn turn;
    for (int64_t row = g.row; row < a.m; row += g.step, turn.next(stages)) {
        // sums of b^2 and of s g w dy b (a token's gate is taken out: its
        // gradient is that sum)
        float s[2];
        rs.wait(turn.slot, turn.phase);
        F2 sq = 0, dot = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), yv = rs.get<T, V>(turn.slot, 1, c);
            F2 w[V / 2];
            weight_pairs<V, NV>(wc, i, c, at, w);
            if constexpr (full) {
                const Pack<T, V> gv = rs.get<T, V>(turn.slot, 2, c);
#pragma unroll
                for (int j = 0; j < V / 2; ++j) w[j] = f2_mul(w[j], pair(gv, j));
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 f = pair(bv, j);
                sq = f2_fma(f, f, sq);
                dot = f2_fma(f2_mul(pair(yv, j), w[j]), f, dot);
            }
        }
        s[0] = f2_sum(sq), s[1] = f2_sum(dot);
        float ba = 0.0f, ya = 0.0f, ga = 1.0f;
        if (g.loose >= 0) {
            ba = rs.one<T>(turn.slot, 0, g.loose), ya = rs.one<T>(turn.slot, 1, g.loose);
            if constexpr (full) ga = rs.one<T>(turn.slot, 2, g.loose);
            s[0] = fmaf(ba, ba, s[0]), s[1] = fmaf(ya * wl * ga, ba, s[1]);
        }
        red.sum(s);
        const float gtok = token ? static_cast<const float *>(a.gate)[row] : 1.0f;
        const float rho = rms_factor(s[0], inv_d, a.eps);
        if (token && a.dgate && g.t == 0) static_cast<float *>(a.dgate)[row] = rho * s[1];
        // db = rho (s g dy w - u mean), u = b rho
        const float mean = gtok * rho * s[1] * inv_d, k = -rho * mean * rho;
        const F2 rho2 = f2(gtok * rho, gtok * rho), back = f2(k, k);
        T *out = static_cast<T *>(a.dB) + row * a.lddb;
        T *dgr = full && a.dgate ? static_cast<T *>(a.dgate) + row * a.lddg : nullptr;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            const Pack<T, V> bv = rs.get<T, V>(turn.slot, 0, c), yv = rs.get<T, V>(turn.slot, 1, c);
            Pack<T, V> gv;
            F2 w[V / 2], o[V / 2];
            weight_pairs<V, NV>(wc, i, c, at, w);
            if constexpr (full) {
                gv = rs.get<T, V>(turn.slot, 2, c);
                if (dgr) {
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) o[j] = f2_mul(f2_mul(pair(yv, j), rho2), f2_mul(pair(bv, j), w[j]));
                    store_pack<T, V>(dgr, c, d, pack_pairs<T, V>(o));
                }
            }
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 b = pair(bv, j);
                F2 y = f2_mul(pair(yv, j), rho2);
                if constexpr (full) y = f2_mul(y, pair(gv, j));
                // the channel's gate, like s, is a factor of the whole column
                acc[i][j] = f2_fma(y, b, acc[i][j]);
                o[j] = f2_fma(y, w[j], f2_mul(b, back));
            }
            store_pack<T, V>(out, c, d, pack_pairs<T, V>(o));
        }
        if (g.loose >= 0) {
            float y = ya * (gtok * rho);
            if constexpr (full) {
                if (dgr) store_elem(dgr, g.loose, y * ba * wl);
                y *= ga;
            }
            alone = fmaf(y, ba, alone);
            store_elem(out, g.loose, y * wl + ba * k);
        }
        rs.release(turn.slot);
    }
    if (a.partials) {
        float sums[NV][V];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V / 2; ++j) f2_split(acc[i][j], sums[i][2 * j], sums[i][2 * j + 1]);
        write_partials<V, NV, ANY>(sums, alone, a.partials, g, d, nullptr);
    }
}

template <typename T, int NV, bool BIG, bool ANY> struct AfterStream {
    static const void *fn(const NormAfterArgs &a)
    {
        return a.gate_kind == Q4_GATE_FULL ? reinterpret_cast<const void *>(&norm_after_stream_kernel<T, NV, BIG, ANY, true>)
                                           : reinterpret_cast<const void *>(&norm_after_stream_kernel<T, NV, BIG, ANY, false>);
    }
};
template <typename T, int NV, bool BIG, bool ANY> struct BeforeBwdStream {
    static const void *fn(const NormBeforeBwdArgs &) { return reinterpret_cast<const void *>(&norm_before_bwd_stream_kernel<T, NV, BIG, ANY>); }
};
template <typename T, int NV, bool BIG, bool ANY> struct AfterBwdStream {
    static const void *fn(const NormAfterBwdArgs &a)
    {
        return a.gate_kind == Q4_GATE_FULL ? reinterpret_cast<const void *>(&norm_after_bwd_stream_kernel<T, NV, BIG, ANY, true>)
                                           : reinterpret_cast<const void *>(&norm_after_bwd_stream_kernel<T, NV, BIG, ANY, false>);
    }
};

template <template <typename, int, bool, bool> class K, typename T, bool ANY, typename Args>
const void *stream_fn(const NormStreamPlan &p, const Args &a)
{
    if (p.G > 256) return p.NV == 2 ? K<T, 2, true, ANY>::fn(a) : K<T, 4, true, ANY>::fn(a);
    return p.NV == 1 ? K<T, 1, false, ANY>::fn(a) : p.NV == 2 ? K<T, 2, false, ANY>::fn(a) : K<T, 4, false, ANY>::fn(a);
}
template <template <typename, int, bool, bool> class K, bool ANY, typename Args>
cudaError_t launch_stream(const NormStreamPlan &p, Args a, int type, cudaStream_t s)
{
    const void *fn = type == Q4_TYPE_F32   ? stream_fn<K, float, ANY>(p, a)
                     : type == Q4_TYPE_F16 ? stream_fn<K, __half, ANY>(p, a)
                                           : stream_fn<K, __nv_bfloat16, ANY>(p, a);
    const cudaError_t e = set_max_smem(fn, p.smem);
    if (e != cudaSuccess) return e;
    a.G = p.G;
    int stages = p.stages;
    void *args[] = {&a, &stages};
    return launch_pdl(fn, dim3(static_cast<unsigned>(p.ctas)), dim3(static_cast<unsigned>(p.G + 32)), p.smem, s, args);
}

} // namespace
} // namespace q4
