// q4mm_norm.cu -- the norms before and after a block of linear layers.
//
//   N(x) = x / sqrt(mean(x^2) + eps)                      (per row of d values)
//   before:  h = N(x) * (o + w)             as values, or as int8 codes and a
//                                           scale for the int8 product
//   after:   y = r + s * g * N(b) * (o + w) the residual stream r, the residual
//                                           scale s, the gate g (none, one per
//                                           channel, per token or per value)
//   both:    y as above, then h = N(y) * (o' + w') of y as it is stored
//
// Gradients (u = x * rho, rho = 1 / sqrt(mean(x^2) + eps)):
//   dx = rho * (dn - u * mean(dn * u))     with dn = dh * (o + w), and
//   dw = sum over tokens of dh * u         (dn = s * g * dy * (o + w) and
//                                           dw = sum of s * g * dy * u after)
//   dg = s * dy * u * (o + w), summed over what the gate is shared by.
// mean(dn * u) = rho * sum(dn * x) / d does not need rho inside its sum, so a
// row takes one reduction of all its sums and its values are read once; the
// statistics are recomputed rather than kept from the forward pass, which
// would cost a read of them and saves nothing here.
//
// All of it is bound by the memory traffic: each matrix is read or written
// once. Statistics and sums are fp32; a result is rounded to its type once.
// Column sums (dw, the channel gate's gradient) stay in registers over the
// rows of a CTA, go to the workspace as one row of partial sums per CTA and
// are added there in CTA order by a second kernel: the same bits every run.
//
// The kernels of this file take few rows, narrow ones and very long ones, and those
// of matrices whose rows start unlike one another. GB300, us a call (floor), join:
// 1 x 2560 fp32 3.8 (0.01; the launch, a load, two reductions); 16384 x 1000 bf16 39
// (19); 12000 x 601 bf16, rows on odd boundaries, 27 (9; 600 aligned 22); 2000 x 16384
// fp32 125 (77; values past the registers are read twice).
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_norm.cuh"

namespace q4 {
namespace {

// The largest CTA of a kernel with NV vectors a thread: its registers allow
// 1024 threads an SM.
__host__ __device__ constexpr int max_threads(int NV) { return NV == 1 ? 1024 : 512; }

template <typename T, int V, int NV, bool ANY>
__global__ void __launch_bounds__(max_threads(NV), 1024 / max_threads(NV)) norm_before_kernel(const NormBeforeArgs a)
{
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32, false};
    if (red.warps > 1) {
        red.clear(static_cast<int>(blockDim.x));
        __syncthreads();
    }
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    Channels<V, NV, false> wo;
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *xr = static_cast<const T *>(a.X) + row * a.ldx;
        g.begin<ANY>(xr, d);
        Pack<T, V> x[NV];
        load_row<T, V, NV>(x, xr, g, d);
        const float alone = g.loose >= 0 ? load_elem(xr, g.loose) : 0.0f;
        float r = 1.0f;   // x * 1 * 1 is x
        if (!a.plain) {
            float s[1] = {alone * alone};
#pragma unroll
            for (int i = 0; i < NV; ++i) s[0] = square_sum<T, V>(x[i], s[0]);
            for (int c = g.at<V>(NV); c < g.end; c += g.G * V) s[0] = square_sum<T, V>(load_pack<T, V>(xr, c, d), s[0]);
            red.sum(s);
            r = rms_factor(s[0], inv_d, a.eps);
        }
        write_normed<T, V, NV, false, ANY>(x, [&](int c) { return load_pack<T, V>(xr, c, d); }, alone, r, a.out, wo, row, g, d, red);
    }
}

template <typename T, int V, int NV, bool ANY>
__global__ void __launch_bounds__(max_threads(NV), 1024 / max_threads(NV)) norm_after_kernel(const NormAfterArgs a)
{
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32, false};
    if (red.warps > 1) {
        red.clear(static_cast<int>(blockDim.x));
        __syncthreads();
    }
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const bool full = a.gate_kind == Q4_GATE_FULL;
    const auto after_at = [&](int c, float (&w)[V]) {
        channel_weights<V, ANY>(a.w, a.w_off, c, d, w);
        if (a.gate_kind == Q4_GATE_CHANNEL) {
            float gc[V];
            load_params<V, ANY>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    Channels<V, NV, false> wa, wo;
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *br = static_cast<const T *>(a.B) + row * a.ldb, *rr = static_cast<const T *>(a.R) + row * a.ldr;
        const T *gr = full ? static_cast<const T *>(a.gate) + row * a.ldg : nullptr;
        T *yr = static_cast<T *>(a.Y) + row * a.ldy;
        g.begin<ANY>(br, d);
        const int rest = g.at<V>(NV);
        Pack<T, V> b[NV], r[NV], gt[NV];
        load_row<T, V, NV>(b, br, g, d);
        load_row<T, V, NV>(r, rr, g, d);
        if (full) load_row<T, V, NV>(gt, gr, g, d);
        float alone = g.loose >= 0 ? load_elem(br, g.loose) : 0.0f;
        float s[1] = {alone * alone};
#pragma unroll
        for (int i = 0; i < NV; ++i) s[0] = square_sum<T, V>(b[i], s[0]);
        for (int c = rest; c < g.end; c += g.G * V) s[0] = square_sum<T, V>(load_pack<T, V>(br, c, d), s[0]);
        red.sum(s);
        float q = a.scale * rms_factor(s[0], inv_d, a.eps);
        if (a.gate_kind == Q4_GATE_TOKEN) q *= static_cast<const float *>(a.gate)[row];
        // y = r + q g b (o + w), stored; the sum of its squares as stored
        s[0] = 0.0f;
        const auto join = [&](int i, const Pack<T, V> &rv, const Pack<T, V> &bv, const Pack<T, V> &gv, int c) {
            float w[V], y[V];
            if (i < 0) after_at(c, w);
            else wa.get(i, c, after_at, w);
            if constexpr (kPairs<T, V>) {
                if (full) {
#pragma unroll
                    for (int j = 0; j < V; ++j) w[j] *= elem(gv, j);
                }
                scaled_sum<T, V>(bv, q, w, rv, y);
                if (c + V > d) {   // nothing outside enters the sum
#pragma unroll
                    for (int j = 0; j < V; ++j) y[j] = c + j < d ? y[j] : 0.0f;
                }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float f = elem(bv, j) * q * w[j];
                    if (full) f *= elem(gv, j);
                    y[j] = c + j < d ? elem(rv, j) + f : 0.0f;
                }
            }
            const Pack<T, V> o = pack_of<T, V>(y);
            store_pack<T, V>(yr, c, d, o);
            s[0] = square_sum<T, V>(o, s[0]);
            return o;
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c < g.end) r[i] = join(i, r[i], b[i], gt[i], c);
        }
        for (int c = rest; c < g.end; c += g.G * V)
            join(-1, load_pack<T, V>(rr, c, d), load_pack<T, V>(br, c, d), full ? load_pack<T, V>(gr, c, d) : zero_pack<T, V>(), c);
        if (g.loose >= 0) {
            float w = channel_weight(a.w, a.w_off, g.loose);
            if (a.gate_kind == Q4_GATE_CHANNEL) w *= static_cast<const float *>(a.gate)[g.loose];
            if (full) w *= load_elem(gr, g.loose);
            alone = store_elem(yr, g.loose, load_elem(rr, g.loose) + alone * q * w);
            s[0] = fmaf(alone, alone, s[0]);
        }
        if (a.out.H) {
            red.sum(s);
            const float rho = rms_factor(s[0], inv_d, a.out_eps);
            write_normed<T, V, NV, false, ANY>(r, [&](int c) { return load_pack<T, V>(yr, c, d); }, alone, rho, a.out, wo, row, g, d, red);
        }
    }
}

// ---------------------------------------------------------------- backward --

template <typename T, int V, int NV, bool ANY> __global__ void __launch_bounds__(512) norm_before_bwd_kernel(const NormBeforeBwdArgs a)
{
    extern __shared__ float dsmem[];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32, false};
    if (red.warps > 1) {
        red.clear(static_cast<int>(blockDim.x));
        __syncthreads();
    }
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const T *X = static_cast<const T *>(a.X), *DH = static_cast<const T *>(a.dH), *DR = static_cast<const T *>(a.dR);
    float acc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
    float alone = 0.0f;   // the column sum outside the vectors
    float *tail = a.partials ? a.partials + static_cast<int64_t>(blockIdx.x) * d : nullptr;
    bool first = true;
    const auto at = [&](int c, float (&w)[V]) { channel_weights<V, ANY>(a.w, a.w_off, c, d, w); };
    g.begin<ANY>(X + g.row * a.ldx, d);   // the same in all of the group's rows
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *xr = X + row * a.ldx, *hr = DH + row * a.lddh, *rr = DR ? DR + row * a.lddr : nullptr;
        T *out = static_cast<T *>(a.dX) + row * a.lddx;
        Pack<T, V> x[NV], dh[NV], dr[NV];
        load_row<T, V, NV>(x, xr, g, d);
        load_row<T, V, NV>(dh, hr, g, d);
        if (rr) load_row<T, V, NV>(dr, rr, g, d);
        float xa = 0.0f, ha = 0.0f, wl = 0.0f;   // outside the vectors
        if (g.loose >= 0) xa = load_elem(xr, g.loose), ha = load_elem(hr, g.loose), wl = channel_weight(a.w, a.w_off, g.loose);
        float s[2] = {xa * xa, ha * wl * xa};
        const auto sums = [&](int i, const Pack<T, V> &xv, const Pack<T, V> &hv, int c) {
            float w[V];
            if (i < 0) at(c, w);
            else wc.get(i, c, at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = elem(xv, j);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(elem(hv, j) * w[j], f, s[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c < g.end) sums(i, x[i], dh[i], c);
        }
        for (int c = g.at<V>(NV); c < g.end; c += g.G * V) sums(-1, load_pack<T, V>(xr, c, d), load_pack<T, V>(hr, c, d), c);
        red.sum(s);
        const float rho = rms_factor(s[0], inv_d, a.eps);
        const float mean = rho * s[1] * inv_d;
        const auto one = [&](int i, int c, const Pack<T, V> &xv, const Pack<T, V> &hv, const Pack<T, V> &rv, float (&col)[V]) {
            float w[V];
            if (i < 0) at(c, w);
            else wc.get(i, c, at, w);
            float o[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = elem(xv, j) * rho, h = elem(hv, j);
                col[j] = fmaf(h, u, col[j]);
                o[j] = rho * (h * w[j] - u * mean);
                if (rr) o[j] += elem(rv, j);
            }
            store_pack<T, V>(out, c, d, pack_of<T, V>(o));
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c < g.end) one(i, c, x[i], dh[i], dr[i], acc[i]);
        }
        if (g.loose >= 0) {
            const float u = xa * rho;
            alone = fmaf(ha, u, alone);
            store_elem(out, g.loose, rho * (ha * wl - u * mean) + (rr ? load_elem(rr, g.loose) : 0.0f));
        }
        for (int c = g.at<V>(NV); c < g.end; c += g.G * V) {
            float col[V];
#pragma unroll
            for (int j = 0; j < V; ++j) col[j] = !first && tail && c + j < d ? tail[c + j] : 0.0f;
            const Pack<T, V> rv = rr ? load_pack<T, V>(rr, c, d) : zero_pack<T, V>();
            one(-1, c, load_pack<T, V>(xr, c, d), load_pack<T, V>(hr, c, d), rv, col);
            if (tail)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < d) tail[c + j] = col[j];
        }
        first = false;
    }
    if (a.partials) write_partials<V, NV, ANY>(acc, alone, a.partials, g, d, dsmem);
}

template <typename T, int V, int NV, bool ANY> __global__ void __launch_bounds__(512) norm_after_bwd_kernel(const NormAfterBwdArgs a)
{
    extern __shared__ float dsmem[];
    __shared__ __align__(16) float rbuf[kReduceFloats];
    pdl_wait();
    pdl_launch_dependents();
    RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32, false};
    if (red.warps > 1) {
        red.clear(static_cast<int>(blockDim.x));
        __syncthreads();
    }
    const int d = static_cast<int>(a.d);
    const float inv_d = 1.0f / static_cast<float>(d);
    const bool full = a.gate_kind == Q4_GATE_FULL, token = a.gate_kind == Q4_GATE_TOKEN;
    const bool channel = a.gate_kind == Q4_GATE_CHANNEL;
    const T *B = static_cast<const T *>(a.B), *DY = static_cast<const T *>(a.dY), *Gt = static_cast<const T *>(a.gate);
    float acc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
    float alone = 0.0f;   // the column sum outside the vectors
    float *tail = a.partials ? a.partials + static_cast<int64_t>(blockIdx.x) * d : nullptr;
    bool first = true;
    // (o + w), times the channel's gate
    const auto at = [&](int c, float (&w)[V]) {
        channel_weights<V, ANY>(a.w, a.w_off, c, d, w);
        if (channel) {
            float gc[V];
            load_params<V, ANY>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] *= gc[j];
        }
    };
    g.begin<ANY>(B + g.row * a.ldb, d);   // the same in all of the group's rows
    Channels<V, NV, true> wc;
    wc.fill(g, at);
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *br = B + row * a.ldb, *dyr = DY + row * a.lddy, *gr = full ? Gt + row * a.ldg : nullptr;
        T *out = static_cast<T *>(a.dB) + row * a.lddb;
        T *dgr = full && a.dgate ? static_cast<T *>(a.dgate) + row * a.lddg : nullptr;
        const float gtok = token ? static_cast<const float *>(a.gate)[row] : 1.0f;
        Pack<T, V> b[NV], dy[NV], gt[NV];
        load_row<T, V, NV>(b, br, g, d);
        load_row<T, V, NV>(dy, dyr, g, d);
        if (full) load_row<T, V, NV>(gt, gr, g, d);
        // sums of b^2 and of g w dy b (a token's gate is taken out: its gradient is
        // that sum)
        float ba = 0.0f, ya = 0.0f, ga = 1.0f, wl = 0.0f;   // outside the vectors
        if (g.loose >= 0) {
            ba = load_elem(br, g.loose), ya = load_elem(dyr, g.loose), wl = channel_weight(a.w, a.w_off, g.loose);
            if (channel) wl *= static_cast<const float *>(a.gate)[g.loose];
            if (full) ga = load_elem(gr, g.loose);
        }
        float s[2] = {ba * ba, ya * ga * wl * ba};
        const auto sums = [&](int i, int c, const Pack<T, V> &bv, const Pack<T, V> &yv, const Pack<T, V> &gv) {
            float w[V];
            if (i < 0) at(c, w);
            else wc.get(i, c, at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = elem(bv, j);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(elem(yv, j) * (full ? elem(gv, j) * w[j] : w[j]), f, s[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c < g.end) sums(i, c, b[i], dy[i], gt[i]);
        }
        for (int c = g.at<V>(NV); c < g.end; c += g.G * V)
            sums(-1, c, load_pack<T, V>(br, c, d), load_pack<T, V>(dyr, c, d), full ? load_pack<T, V>(gr, c, d) : zero_pack<T, V>());
        red.sum(s);
        const float rho = rms_factor(s[0], inv_d, a.eps);
        if (token && a.dgate && g.t == 0) static_cast<float *>(a.dgate)[row] = a.scale * rho * s[1];
        const float mean = gtok * rho * s[1] * inv_d;
        const float q = a.scale * rho;
        const auto one = [&](int i, int c, const Pack<T, V> &bv, const Pack<T, V> &yv, const Pack<T, V> &gv, float (&col)[V]) {
            float w[V], o[V], og[V];
            if (i < 0) at(c, w);
            else wc.get(i, c, at, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = elem(bv, j) * rho, y = elem(yv, j);
                const float gy = full ? elem(gv, j) * y : gtok * y;
                // the channel's gate, like s, is a factor of the whole column
                col[j] = fmaf(gy, u, col[j]);
                o[j] = q * (gy * w[j] - u * mean);
                og[j] = a.scale * y * u * w[j];
            }
            store_pack<T, V>(out, c, d, pack_of<T, V>(o));
            if (dgr) store_pack<T, V>(dgr, c, d, pack_of<T, V>(og));
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c < g.end) one(i, c, b[i], dy[i], gt[i], acc[i]);
        }
        if (g.loose >= 0) {
            const float u = ba * rho, gy = full ? ga * ya : gtok * ya;
            alone = fmaf(gy, u, alone);
            store_elem(out, g.loose, q * (gy * wl - u * mean));
            if (dgr) store_elem(dgr, g.loose, a.scale * ya * u * wl);
        }
        for (int c = g.at<V>(NV); c < g.end; c += g.G * V) {
            float col[V];
#pragma unroll
            for (int j = 0; j < V; ++j) col[j] = !first && tail && c + j < d ? tail[c + j] : 0.0f;
            const Pack<T, V> gv = full ? load_pack<T, V>(gr, c, d) : zero_pack<T, V>();
            one(-1, c, load_pack<T, V>(br, c, d), load_pack<T, V>(dyr, c, d), gv, col);
            if (tail)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < d) tail[c + j] = col[j];
        }
        first = false;
    }
    if (a.partials) write_partials<V, NV, ANY>(acc, alone, a.partials, g, d, dsmem);
}

// Column sums of the partials: 32 columns a CTA, the rows dealt to 32 warps
// and their sums added in warp order. dw = sum * scale [* gate];
// dgate = sum * scale * (o + w).
__global__ void __launch_bounds__(1024) column_sum_kernel(const NormColumnArgs a)
{
    __shared__ float part[32][33];
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float s = 0.0f;
    if (c < a.d)
        for (int p = warp; p < a.rows; p += 32 * 16) {   // sixteen loads in flight
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = p + 32 * i < a.rows ? a.partials[(p + 32 * i) * a.d + c] : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) s += v[i];
        }
    part[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= a.d) return;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += part[i][lane];
    s *= a.scale;
    if (a.dw) a.dw[c] = a.gate ? s * a.gate[c] : s;
    if (a.dgate) a.dgate[c] = s * (a.w ? a.w_off + a.w[c] : 1.0f);
}

// -------------------------------------------------------------- launching --

// How a row of d elements is held: vectors of V elements, NV of them a thread
// in registers, G threads a row, `threads` a CTA.
struct RowPlan {
    int V, NV, G, threads;
    int64_t ctas;
};

// Vectors a thread, threads a row and a CTA. With 16-byte vectors 1, 2 or 4 a
// thread, else 2, 4 or 8 elements. Few rows take many threads each; many take a
// warp each where that holds them, else CTAs of about 256 threads: their barriers
// stop fewer others, and several fit on an SM. A row longer than 512 threads hold
// is finished by the kernels' loops.
RowPlan plan_rows(const RowAccess &acc, int64_t m, int64_t d, bool backward, int64_t sm_count)
{
    RowPlan p;
    p.V = acc.vec;
    const int64_t vecs = acc.any ? std::max<int64_t>(1, d / acc.vec) : ceil_div(d, acc.vec);   // at most
    const bool wide = acc.vec > 1;
    const int n[3] = {wide ? 1 : 2, wide ? 2 : 4, wide ? 4 : 8};
    const bool few = m <= 304;
    p.NV = n[2];
    p.G = 32;
    if (vecs <= 32 * n[0]) {
        p.NV = n[0];
    } else if (!few && vecs <= 32 * n[2]) {
        p.NV = vecs <= 32 * n[1] ? n[1] : n[2];
    } else {
        const int limit = few && !backward ? 1024 : few ? 512 : 256;
        for (int i = 2; i >= 0; --i)
            if (ceil_div(vecs, n[i]) <= std::min(limit, n[i] == 1 && !backward ? 1024 : 512)) p.NV = n[i];
        p.G = static_cast<int>(std::min<int64_t>(512, round_up(ceil_div(vecs, p.NV), 32)));
        if (p.NV == 1 && !backward) p.G = static_cast<int>(round_up(vecs, 32));
    }
    p.threads = p.G == 32 ? (few ? 64 : 256) : p.G;
    // Forward a CTA takes its rows once and leaves: CTAs of other rows fill the
    // time that its loads take. Backward as many as the device holds at the least
    // (1024 threads an SM), for the column sums; a multiple of kRowStep, so that
    // a group's rows all start alike.
    p.ctas = std::min<int64_t>(ceil_div(m, p.threads / p.G),
                               backward ? round_row_step(std::min<int64_t>(kNormPartials, sm_count * (1024 / p.threads)))
                                        : (int64_t(1) << 30));
    return p;
}

template <template <typename, int, int, bool> class K, typename T, typename Args>
cudaError_t launch_rows_v(const RowPlan &p, bool any, Args a, size_t smem, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const void *fn = nullptr;
    if (any) fn = p.NV == 1 ? K<T, W, 1, true>::fn() : p.NV == 2 ? K<T, W, 2, true>::fn() : K<T, W, 4, true>::fn();
    else if (p.V == W) fn = p.NV == 1 ? K<T, W, 1, false>::fn() : p.NV == 2 ? K<T, W, 2, false>::fn() : K<T, W, 4, false>::fn();
    else fn = p.NV == 2 ? K<T, 1, 2, false>::fn() : p.NV == 4 ? K<T, 1, 4, false>::fn() : K<T, 1, 8, false>::fn();
    a.G = p.G;
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(p.ctas)), dim3(static_cast<unsigned>(p.threads)), smem, s, args);
}
template <template <typename, int, int, bool> class K, typename Args>
cudaError_t launch_rows(int type, const RowPlan &p, bool any, const Args &a, size_t smem, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_rows_v<K, float>(p, any, a, smem, s);
    case Q4_TYPE_F16: return launch_rows_v<K, __half>(p, any, a, smem, s);
    default: return launch_rows_v<K, __nv_bfloat16>(p, any, a, smem, s);
    }
}

template <typename T, int V, int NV, bool ANY> struct BeforeKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_before_kernel<T, V, NV, ANY>); }
};
template <typename T, int V, int NV, bool ANY> struct AfterKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_kernel<T, V, NV, ANY>); }
};
template <typename T, int V, int NV, bool ANY> struct BeforeBwdKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_before_bwd_kernel<T, V, NV, ANY>); }
};
template <typename T, int V, int NV, bool ANY> struct AfterBwdKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_bwd_kernel<T, V, NV, ANY>); }
};

// Shared memory in which the groups of a CTA meet (one group: none).
size_t partial_smem(const RowPlan &p, int64_t d) { return p.threads > p.G ? sizeof(float) * (p.threads / p.G) * d : 0; }

cudaError_t launch_columns(NormColumnArgs a, cudaStream_t s)
{
    void *args[] = {&a};
    return launch_pdl(reinterpret_cast<const void *>(&column_sum_kernel), dim3(static_cast<unsigned>(ceil_div(a.d, 32))),
                      dim3(1024), 0, s, args);
}

} // namespace

cudaError_t launch_norm_before(const NormBeforeArgs &a, int type, const RowAccess &acc, int sm_count, cudaStream_t s)
{
    const RowPlan p = plan_rows(acc, a.m, a.d, false, sm_count);
    return launch_rows<BeforeKernel>(type, p, acc.any, a, 0, s);
}

cudaError_t launch_norm_after(const NormAfterArgs &a, int type, const RowAccess &acc, int sm_count, cudaStream_t s)
{
    NormStreamPlan sp;
    if (acc.vec > 1 && plan_norm_stream(a.m, a.d, type, acc.any, a.gate_kind == Q4_GATE_FULL ? 3 : 2, sm_count, &sp))
        return launch_norm_after_stream(sp, a, type, s);
    const RowPlan p = plan_rows(acc, a.m, a.d, false, sm_count);
    return launch_rows<AfterKernel>(type, p, acc.any, a, 0, s);
}

cudaError_t launch_norm_before_bwd(const NormBeforeBwdArgs &a, float *dw, int type, const RowAccess &acc, int sm_count, cudaStream_t s)
{
    NormStreamPlan sp;
    cudaError_t e;
    int64_t ctas;
    if (acc.vec > 1 && plan_norm_stream(a.m, a.d, type, acc.any, a.dR ? 3 : 2, sm_count, &sp)) {
        e = launch_norm_before_bwd_stream(sp, a, type, s);
        ctas = sp.ctas;
    } else {
        const RowPlan p = plan_rows(acc, a.m, a.d, true, sm_count);
        e = launch_rows<BeforeBwdKernel>(type, p, acc.any, a, partial_smem(p, a.d), s);
        ctas = p.ctas;
    }
    if (e != cudaSuccess || !dw) return e;
    NormColumnArgs c{};
    c.partials = a.partials;
    c.rows = static_cast<int>(ctas);
    c.d = a.d;
    c.scale = 1.0f;
    c.dw = dw;
    return launch_columns(c, s);
}

cudaError_t launch_norm_after_bwd(const NormAfterBwdArgs &a, float *dw, int type, const RowAccess &acc, int sm_count, cudaStream_t s)
{
    NormStreamPlan sp;
    cudaError_t e;
    int64_t ctas;
    if (acc.vec > 1 && plan_norm_stream(a.m, a.d, type, acc.any, a.gate_kind == Q4_GATE_FULL ? 3 : 2, sm_count, &sp)) {
        e = launch_norm_after_bwd_stream(sp, a, type, s);
        ctas = sp.ctas;
    } else {
        const RowPlan p = plan_rows(acc, a.m, a.d, true, sm_count);
        e = launch_rows<AfterBwdKernel>(type, p, acc.any, a, partial_smem(p, a.d), s);
        ctas = p.ctas;
    }
    if (e != cudaSuccess || !a.partials) return e;
    NormColumnArgs c{};
    c.partials = a.partials;
    c.rows = static_cast<int>(ctas);
    c.d = a.d;
    c.scale = a.scale;
    c.dw = dw;
    if (a.gate_kind == Q4_GATE_CHANNEL) {
        c.gate = static_cast<const float *>(a.gate);
        c.dgate = static_cast<float *>(a.dgate);
        c.w = a.w;
        c.w_off = a.w_off;
    }
    return launch_columns(c, s);
}

} // namespace q4
