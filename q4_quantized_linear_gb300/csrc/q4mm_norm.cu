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
#include <algorithm>
#include <cuda_runtime.h>

#include "q4mm_norm.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

// Which rows this thread works on, and where in them.
struct RowGroup {
    int t, G;                 // thread of the row, threads of a row
    int64_t row, step;        // first row, rows between two of this group's
};
__device__ __forceinline__ RowGroup row_group(int G)
{
    RowGroup g;
    const int groups = static_cast<int>(blockDim.x) / G;
    g.G = G;
    g.t = static_cast<int>(threadIdx.x) % G;
    g.row = static_cast<int64_t>(blockIdx.x) * groups + static_cast<int>(threadIdx.x) / G;
    g.step = static_cast<int64_t>(gridDim.x) * groups;
    return g;
}

// Rows of the next iteration are loaded before this one's reductions where
// that doubles no more than 32 bytes a thread and matrix.
template <typename T, int V, int NV> constexpr bool kAhead = NV * V * sizeof(T) <= 32;
// The channels' weights stay in registers over the rows where they are few.
template <int V, int NV> constexpr bool kKeep = NV * V <= 8;

template <typename T, int V, int NV>
__device__ __forceinline__ void load_row(Pack<T, V> (&x)[NV], const T *row, int t, int G, int d)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * G + t) * V;
        if (c < d) x[i] = load_pack<T, V>(row, c, d);
        else
#pragma unroll
            for (int j = 0; j < V; ++j) x[i].e[j] = from_f32<T>(0.0f);
    }
}

template <int V> __device__ __forceinline__ void channel_weights(const float *w, float off, int c, int d, float out[V])
{
    if (w) {
        load_params<V>(w, c, d, out);
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] += off;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 1.0f;
    }
}

// h = x * r * w of one vector, for values or for the coding.
template <typename T, int V>
__device__ __forceinline__ void normed(const Pack<T, V> &x, float r, const float w[V], float h[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) h[j] = to_f32(x.e[j]) * r * w[j];
}

template <typename T, int V> __device__ __forceinline__ void store_values(T *row, int c, int d, const float h[V])
{
    Pack<T, V> o;
#pragma unroll
    for (int j = 0; j < V; ++j) o.e[j] = from_f32<T>(h[j]);
    store_pack<T, V>(row, c, d, o);
}
template <int V> __device__ __forceinline__ void store_codes(int8_t *row, int c, int d, const float h[V], float factor)
{
    Pack<int8_t, V> o;
#pragma unroll
    for (int j = 0; j < V; ++j) o.e[j] = code_of(h[j], factor);
    store_pack<int8_t, V>(row, c, d, o);
}

// The second half of a row that has been summed: h = x * r * (o + w), stored
// as values or coded. `x(i, c)` gives vector i at element c; vectors past NV
// are read again by `again(c)`.
template <typename T, int V, int NV, typename Again>
__device__ __forceinline__ void write_normed(const Pack<T, V> (&x)[NV], Again again, float r, const NormOut &o,
                                             int64_t row, const RowGroup &g, int d, RowReducer &red,
                                             const float (&wk)[kKeep<V, NV> ? NV : 1][V])
{
    float w[V], h[V];
    if (!o.codes) {
        T *out = static_cast<T *>(o.H) + row * o.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            if constexpr (kKeep<V, NV>) {
                normed<T, V>(x[i], r, wk[i], h);
            } else {
                channel_weights<V>(o.w, o.w_off, c, d, w);
                normed<T, V>(x[i], r, w, h);
            }
            store_values<T, V>(out, c, d, h);
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            channel_weights<V>(o.w, o.w_off, c, d, w);
            normed<T, V>(again(c), r, w, h);
            store_values<T, V>(out, c, d, h);
        }
        return;
    }
    uint32_t mb = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * g.G + g.t) * V;
        if (c >= d) continue;
        if constexpr (kKeep<V, NV>) {
            normed<T, V>(x[i], r, wk[i], h);
        } else {
            channel_weights<V>(o.w, o.w_off, c, d, w);
            normed<T, V>(x[i], r, w, h);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) mb = max(mb, c + j < d ? abs_bits(h[j]) : 0u);
    }
    for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
        channel_weights<V>(o.w, o.w_off, c, d, w);
        normed<T, V>(again(c), r, w, h);
#pragma unroll
        for (int j = 0; j < V; ++j) mb = max(mb, c + j < d ? abs_bits(h[j]) : 0u);
    }
    const CodeScale cs = code_scale(red.max_bits(mb));
    if (g.t == 0) o.h_scale[row] = cs.scale;
    int8_t *out = static_cast<int8_t *>(o.H) + row * o.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * g.G + g.t) * V;
        if (c >= d) continue;
        if constexpr (kKeep<V, NV>) {
            normed<T, V>(x[i], r, wk[i], h);
        } else {
            channel_weights<V>(o.w, o.w_off, c, d, w);
            normed<T, V>(x[i], r, w, h);
        }
        store_codes<V>(out, c, d, h, cs.factor);
    }
    for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
        channel_weights<V>(o.w, o.w_off, c, d, w);
        normed<T, V>(again(c), r, w, h);
        store_codes<V>(out, c, d, h, cs.factor);
    }
}

template <int V, int NV>
__device__ __forceinline__ void keep_weights(float (&wk)[kKeep<V, NV> ? NV : 1][V], const float *w, float off,
                                             const RowGroup &g, int d)
{
    if constexpr (kKeep<V, NV>) {
#pragma unroll
        for (int i = 0; i < NV; ++i) channel_weights<V>(w, off, (i * g.G + g.t) * V, d, wk[i]);
    }
}

template <typename T, int V, int NV> __global__ void __launch_bounds__(1024) norm_before_kernel(const NormBeforeArgs a)
{
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32};
    const int d = static_cast<int>(a.d);
    float wk[kKeep<V, NV> ? NV : 1][V];
    keep_weights<V, NV>(wk, a.out.w, a.out.w_off, g, d);
    Pack<T, V> next[NV];
    if (kAhead<T, V, NV> && g.row < a.m) load_row<T, V, NV>(next, static_cast<const T *>(a.X) + g.row * a.ldx, g.t, g.G, d);
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *xr = static_cast<const T *>(a.X) + row * a.ldx;
        Pack<T, V> x[NV];
        if constexpr (kAhead<T, V, NV>) {
#pragma unroll
            for (int i = 0; i < NV; ++i) x[i] = next[i];
            if (row + g.step < a.m) load_row<T, V, NV>(next, xr + g.step * a.ldx, g.t, g.G, d);
        } else {
            load_row<T, V, NV>(x, xr, g.t, g.G, d);
        }
        float r = 1.0f;   // x * 1 * 1 is x
        if (!a.plain) {
            float s[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float f = to_f32(x[i].e[j]);
                    s[0] = fmaf(f, f, s[0]);
                }
            for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
                const Pack<T, V> v = load_pack<T, V>(xr, c, d);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float f = to_f32(v.e[j]);
                    s[0] = fmaf(f, f, s[0]);
                }
            }
            red.sum(s);
            r = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        }
        write_normed<T, V, NV>(x, [&](int c) { return load_pack<T, V>(xr, c, d); }, r, a.out, row, g, d, red, wk);
    }
}

// y = r + s g N(b) (o + w), one vector; `q` = s / sqrt(mean(b^2) + eps).
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> joined(const Pack<T, V> &rv, const Pack<T, V> &bv, const Pack<T, V> &gv, float q,
                                             const float wg[V], int gate_kind)
{
    Pack<T, V> y;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float f = to_f32(bv.e[j]) * q * wg[j];
        if (gate_kind == Q4_GATE_FULL) f *= to_f32(gv.e[j]);
        y.e[j] = from_f32<T>(to_f32(rv.e[j]) + f);
    }
    return y;
}
// (o + w), times the channel's gate where there is one.
template <int V> __device__ __forceinline__ void gated_weights(const NormAfterArgs &a, int c, int d, float out[V])
{
    channel_weights<V>(a.w, a.w_off, c, d, out);
    if (a.gate_kind == Q4_GATE_CHANNEL) {
        float g[V];
        load_params<V>(static_cast<const float *>(a.gate), c, d, g);
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] *= g[j];
    }
}

template <typename T, int V, int NV> __global__ void __launch_bounds__(1024) norm_after_kernel(const NormAfterArgs a)
{
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    const RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32};
    const int d = static_cast<int>(a.d);
    const bool full = a.gate_kind == Q4_GATE_FULL;
    constexpr bool keep = kKeep<V, NV>, ahead = kAhead<T, V, NV>;
    float wk[keep ? NV : 1][V], wn[keep ? NV : 1][V];
    if constexpr (keep) {
#pragma unroll
        for (int i = 0; i < NV; ++i) gated_weights<V>(a, (i * g.G + g.t) * V, d, wk[i]);
    }
    if (a.out.H) keep_weights<V, NV>(wn, a.out.w, a.out.w_off, g, d);
    const T *R = static_cast<const T *>(a.R), *B = static_cast<const T *>(a.B), *Gt = static_cast<const T *>(a.gate);
    Pack<T, V> bn[NV], rn[NV], gn[NV];
    if (ahead && g.row < a.m) {
        load_row<T, V, NV>(bn, B + g.row * a.ldb, g.t, g.G, d);
        load_row<T, V, NV>(rn, R + g.row * a.ldr, g.t, g.G, d);
        if (full) load_row<T, V, NV>(gn, Gt + g.row * a.ldg, g.t, g.G, d);
    }
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *br = B + row * a.ldb, *rr = R + row * a.ldr, *gr = full ? Gt + row * a.ldg : nullptr;
        T *yr = static_cast<T *>(a.Y) + row * a.ldy;
        Pack<T, V> b[NV], r[NV], gt[NV];
        if constexpr (ahead) {
#pragma unroll
            for (int i = 0; i < NV; ++i) b[i] = bn[i], r[i] = rn[i], gt[i] = gn[i];
            if (row + g.step < a.m) {
                load_row<T, V, NV>(bn, br + g.step * a.ldb, g.t, g.G, d);
                load_row<T, V, NV>(rn, rr + g.step * a.ldr, g.t, g.G, d);
                if (full) load_row<T, V, NV>(gn, gr + g.step * a.ldg, g.t, g.G, d);
            }
        } else {
            load_row<T, V, NV>(b, br, g.t, g.G, d);
            load_row<T, V, NV>(r, rr, g.t, g.G, d);
            if (full) load_row<T, V, NV>(gt, gr, g.t, g.G, d);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_f32(b[i].e[j]);
                s[0] = fmaf(f, f, s[0]);
            }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            const Pack<T, V> v = load_pack<T, V>(br, c, d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_f32(v.e[j]);
                s[0] = fmaf(f, f, s[0]);
            }
        }
        red.sum(s);
        float q = a.scale / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        if (a.gate_kind == Q4_GATE_TOKEN) q *= static_cast<const float *>(a.gate)[row];
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            float w[V];
            if constexpr (!keep) gated_weights<V>(a, c, d, w);
            r[i] = joined<T, V>(r[i], b[i], gt[i], q, keep ? wk[keep ? i : 0] : w, a.gate_kind);
            store_pack<T, V>(yr, c, d, r[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = c + j < d ? to_f32(r[i].e[j]) : 0.0f;
                s[0] = fmaf(f, f, s[0]);
            }
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            float w[V];
            gated_weights<V>(a, c, d, w);
            Pack<T, V> gv{};
            if (full) gv = load_pack<T, V>(gr, c, d);
            const Pack<T, V> y = joined<T, V>(load_pack<T, V>(rr, c, d), load_pack<T, V>(br, c, d), gv, q, w, a.gate_kind);
            store_pack<T, V>(yr, c, d, y);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = c + j < d ? to_f32(y.e[j]) : 0.0f;
                s[0] = fmaf(f, f, s[0]);
            }
        }
        if (a.out.H) {
            red.sum(s);
            const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.out_eps);
            write_normed<T, V, NV>(r, [&](int c) { return load_pack<T, V>(yr, c, d); }, rho, a.out, row, g, d, red, wn);
        }
    }
}

// ---------------------------------------------------------------- backward --

// Adds the CTA's groups' column sums (one group: its registers as they are)
// into row blockIdx.x of the partials. The tail past the registers has been
// added there already.
template <int V, int NV>
__device__ __forceinline__ void write_partials(float (&acc)[NV][V], float *partials, const RowGroup &g, int d, float *smem)
{
    float *out = partials + static_cast<int64_t>(blockIdx.x) * d;
    const int groups = static_cast<int>(blockDim.x) / g.G;
    if (groups == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < d) out[c + j] = acc[i][j];
        }
        return;
    }
    const int width = g.G * NV * V;   // >= d
    const int mine = static_cast<int>(threadIdx.x) / g.G;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) smem[mine * width + (i * g.G + g.t) * V + j] = acc[i][j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < groups; ++k) s += smem[k * width + c];
        out[c] = s;
    }
}

template <typename T, int V, int NV> __global__ void __launch_bounds__(512) norm_before_bwd_kernel(const NormBeforeBwdArgs a)
{
    extern __shared__ float dsmem[];
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32};
    const int d = static_cast<int>(a.d);
    const T *X = static_cast<const T *>(a.X), *DH = static_cast<const T *>(a.dH), *DR = static_cast<const T *>(a.dR);
    float acc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
    float *tail = a.partials ? a.partials + static_cast<int64_t>(blockIdx.x) * d : nullptr;
    bool first = true;
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *xr = X + row * a.ldx, *hr = DH + row * a.lddh, *rr = DR ? DR + row * a.lddr : nullptr;
        T *out = static_cast<T *>(a.dX) + row * a.lddx;
        Pack<T, V> x[NV], dh[NV], dr[NV];
        load_row<T, V, NV>(x, xr, g.t, g.G, d);
        load_row<T, V, NV>(dh, hr, g.t, g.G, d);
        if (rr) load_row<T, V, NV>(dr, rr, g.t, g.G, d);
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            float w[V];
            if (c >= d) continue;
            channel_weights<V>(a.w, a.w_off, c, d, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_f32(x[i].e[j]);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(to_f32(dh[i].e[j]) * w[j], f, s[1]);
            }
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            float w[V];
            channel_weights<V>(a.w, a.w_off, c, d, w);
            const Pack<T, V> xv = load_pack<T, V>(xr, c, d), hv = load_pack<T, V>(hr, c, d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_f32(xv.e[j]);
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(to_f32(hv.e[j]) * w[j], f, s[1]);
            }
        }
        red.sum(s);
        const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        const float mean = rho * s[1] / static_cast<float>(d);
        auto one = [&](int c, const Pack<T, V> &xv, const Pack<T, V> &hv, const Pack<T, V> &rv, float *col) {
            float w[V];
            channel_weights<V>(a.w, a.w_off, c, d, w);
            Pack<T, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = to_f32(xv.e[j]) * rho, h = to_f32(hv.e[j]);
                col[j] = fmaf(h, u, col[j]);
                float v = rho * (h * w[j] - u * mean);
                if (rr) v += to_f32(rv.e[j]);
                o.e[j] = from_f32<T>(v);
            }
            store_pack<T, V>(out, c, d, o);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c < d) one(c, x[i], dh[i], dr[i], acc[i]);
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            float col[V];
#pragma unroll
            for (int j = 0; j < V; ++j) col[j] = !first && tail && c + j < d ? tail[c + j] : 0.0f;
            Pack<T, V> rv{};
            if (rr) rv = load_pack<T, V>(rr, c, d);
            one(c, load_pack<T, V>(xr, c, d), load_pack<T, V>(hr, c, d), rv, col);
            if (tail)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < d) tail[c + j] = col[j];
        }
        first = false;
    }
    if (a.partials) write_partials<V, NV>(acc, a.partials, g, d, dsmem);
}

template <typename T, int V, int NV> __global__ void __launch_bounds__(512) norm_after_bwd_kernel(const NormAfterBwdArgs a)
{
    extern __shared__ float dsmem[];
    __shared__ float rbuf[2 * 96];
    pdl_wait();
    pdl_launch_dependents();
    const RowGroup g = row_group(a.G);
    RowReducer red{rbuf, a.G / 32};
    const int d = static_cast<int>(a.d);
    const bool full = a.gate_kind == Q4_GATE_FULL, token = a.gate_kind == Q4_GATE_TOKEN;
    const bool channel = a.gate_kind == Q4_GATE_CHANNEL;
    const T *B = static_cast<const T *>(a.B), *DY = static_cast<const T *>(a.dY), *Gt = static_cast<const T *>(a.gate);
    float acc[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) acc[i][j] = 0.0f;
    float *tail = a.partials ? a.partials + static_cast<int64_t>(blockIdx.x) * d : nullptr;
    bool first = true;
    for (int64_t row = g.row; row < a.m; row += g.step) {
        const T *br = B + row * a.ldb, *dyr = DY + row * a.lddy, *gr = full ? Gt + row * a.ldg : nullptr;
        T *out = static_cast<T *>(a.dB) + row * a.lddb;
        T *dgr = full && a.dgate ? static_cast<T *>(a.dgate) + row * a.lddg : nullptr;
        const float gtok = token ? static_cast<const float *>(a.gate)[row] : 1.0f;
        Pack<T, V> b[NV], dy[NV], gt[NV];
        load_row<T, V, NV>(b, br, g.t, g.G, d);
        load_row<T, V, NV>(dy, dyr, g.t, g.G, d);
        if (full) load_row<T, V, NV>(gt, gr, g.t, g.G, d);
        // sums of b^2, of g w dy b, and (a token's gate) of w dy b
        float s[2] = {0.0f, 0.0f};
        auto sums = [&](int c, const Pack<T, V> &bv, const Pack<T, V> &yv, const Pack<T, V> &gv) {
            float w[V], gc[V];
            channel_weights<V>(a.w, a.w_off, c, d, w);
            if (channel) load_params<V>(static_cast<const float *>(a.gate), c, d, gc);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float f = to_f32(bv.e[j]);
                const float gw = channel ? gc[j] * w[j] : full ? to_f32(gv.e[j]) * w[j] : w[j];
                s[0] = fmaf(f, f, s[0]);
                s[1] = fmaf(to_f32(yv.e[j]) * gw, f, s[1]);
            }
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c < d) sums(c, b[i], dy[i], gt[i]);
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            Pack<T, V> gv{};
            if (full) gv = load_pack<T, V>(gr, c, d);
            sums(c, load_pack<T, V>(br, c, d), load_pack<T, V>(dyr, c, d), gv);
        }
        red.sum(s);
        const float rho = 1.0f / sqrtf(s[0] / static_cast<float>(d) + a.eps);
        if (token && a.dgate && g.t == 0) static_cast<float *>(a.dgate)[row] = a.scale * rho * s[1];
        const float mean = gtok * rho * s[1] / static_cast<float>(d);
        const float q = a.scale * rho;
        auto one = [&](int c, const Pack<T, V> &bv, const Pack<T, V> &yv, const Pack<T, V> &gv, float *col) {
            float w[V], gc[V];
            channel_weights<V>(a.w, a.w_off, c, d, w);
            if (channel) load_params<V>(static_cast<const float *>(a.gate), c, d, gc);
            Pack<T, V> o, og;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float u = to_f32(bv.e[j]) * rho, y = to_f32(yv.e[j]);
                const float gv1 = channel ? gc[j] : full ? to_f32(gv.e[j]) : gtok;
                // the channel's gate, like s, is a factor of the whole column
                col[j] = fmaf(channel ? y : y * gv1, u, col[j]);
                o.e[j] = from_f32<T>(q * (y * (gv1 * w[j]) - u * mean));
                if (full) og.e[j] = from_f32<T>(a.scale * y * u * w[j]);
            }
            store_pack<T, V>(out, c, d, o);
            if (dgr) store_pack<T, V>(dgr, c, d, og);
        };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c < d) one(c, b[i], dy[i], gt[i], acc[i]);
        }
        for (int c = (NV * g.G + g.t) * V; c < d; c += g.G * V) {
            float col[V];
#pragma unroll
            for (int j = 0; j < V; ++j) col[j] = !first && tail && c + j < d ? tail[c + j] : 0.0f;
            Pack<T, V> gv{};
            if (full) gv = load_pack<T, V>(gr, c, d);
            one(c, load_pack<T, V>(br, c, d), load_pack<T, V>(dyr, c, d), gv, col);
            if (tail)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < d) tail[c + j] = col[j];
        }
        first = false;
    }
    if (a.partials) write_partials<V, NV>(acc, a.partials, g, d, dsmem);
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
        for (int p = warp; p < a.rows; p += 32) s += a.partials[p * a.d + c];
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

// `max_threads`: the kernel's launch bound. A warp holds a row where its
// registers do; wider rows take a CTA.
RowPlan plan_rows(int V, bool wide, int64_t m, int64_t d, int max_threads, int64_t max_ctas)
{
    RowPlan p;
    p.V = V;
    const int64_t vecs = ceil_div(d, V);
    const int nvs[2][3] = {{2, 8, 8}, {1, 2, 4}};
    const int *nv = nvs[wide ? 1 : 0];
    const int most = nv[2];
    const bool few = m <= 304;   // fewer rows than CTAs the device holds: threads, not vectors, shorten a row
    p.NV = most;
    p.G = 32;
    if (vecs <= 32 * nv[0]) {
        p.NV = nv[0];
    } else if (!few && vecs <= 32 * most) {
        p.NV = vecs <= 32 * nv[1] ? nv[1] : most;
    } else {
        const int target = few ? max_threads : std::min(512, max_threads);
        for (int i = 0; i < 3; ++i)
            if (ceil_div(vecs, nv[i]) <= target || i == 2) {
                p.NV = nv[i];
                break;
            }
        p.G = static_cast<int>(std::min<int64_t>(max_threads, round_up(ceil_div(vecs, p.NV), 32)));
    }
    p.threads = p.G == 32 ? (few ? 64 : 256) : p.G;
    p.ctas = std::min<int64_t>(ceil_div(m, p.threads / p.G), max_ctas);
    return p;
}

template <template <typename, int, int> class K, typename T, typename Args>
cudaError_t launch_rows_v(const RowPlan &p, bool wide, Args a, size_t smem, cudaStream_t s)
{
    constexpr int W = 16 / sizeof(T);
    const void *fn = nullptr;
    if (wide) fn = p.NV == 1 ? K<T, W, 1>::fn() : p.NV == 2 ? K<T, W, 2>::fn() : K<T, W, 4>::fn();
    else if (sizeof(T) == 2 && p.V == 2) fn = p.NV == 2 ? K<T, 2, 2>::fn() : K<T, 2, 8>::fn();
    else fn = p.NV == 2 ? K<T, 1, 2>::fn() : K<T, 1, 8>::fn();
    a.G = p.G;
    void *args[] = {&a};
    return launch_pdl(fn, dim3(static_cast<unsigned>(p.ctas)), dim3(static_cast<unsigned>(p.threads)), smem, s, args);
}
template <template <typename, int, int> class K, typename Args>
cudaError_t launch_rows(int type, const RowPlan &p, bool wide, const Args &a, size_t smem, cudaStream_t s)
{
    switch (type) {
    case Q4_TYPE_F32: return launch_rows_v<K, float>(p, wide, a, smem, s);
    case Q4_TYPE_F16: return launch_rows_v<K, __half>(p, wide, a, smem, s);
    default: return launch_rows_v<K, __nv_bfloat16>(p, wide, a, smem, s);
    }
}

template <typename T, int V, int NV> struct BeforeKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_before_kernel<T, V, NV>); }
};
template <typename T, int V, int NV> struct AfterKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_kernel<T, V, NV>); }
};
template <typename T, int V, int NV> struct BeforeBwdKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_before_bwd_kernel<T, V, NV>); }
};
template <typename T, int V, int NV> struct AfterBwdKernel {
    static const void *fn() { return reinterpret_cast<const void *>(&norm_after_bwd_kernel<T, V, NV>); }
};

// Shared memory in which the groups of a CTA meet (one group: none).
size_t partial_smem(const RowPlan &p) { return p.threads > p.G ? sizeof(float) * p.threads * p.NV * p.V : 0; }

cudaError_t launch_columns(NormColumnArgs a, cudaStream_t s)
{
    void *args[] = {&a};
    return launch_pdl(reinterpret_cast<const void *>(&column_sum_kernel), dim3(static_cast<unsigned>(ceil_div(a.d, 32))),
                      dim3(1024), 0, s, args);
}

} // namespace

cudaError_t launch_norm_before(const NormBeforeArgs &a, int type, int vec, int sm_count, cudaStream_t s)
{
    const bool wide = vec * type_size(type) == 16;
    const RowPlan p = plan_rows(vec, wide, a.m, a.d, 1024, 8 * static_cast<int64_t>(sm_count));
    return launch_rows<BeforeKernel>(type, p, wide, a, 0, s);
}

cudaError_t launch_norm_after(const NormAfterArgs &a, int type, int vec, int sm_count, cudaStream_t s)
{
    const bool wide = vec * type_size(type) == 16;
    const RowPlan p = plan_rows(vec, wide, a.m, a.d, 1024, 8 * static_cast<int64_t>(sm_count));
    return launch_rows<AfterKernel>(type, p, wide, a, 0, s);
}

cudaError_t launch_norm_before_bwd(const NormBeforeBwdArgs &a, float *dw, int type, int vec, int sm_count, cudaStream_t s)
{
    const bool wide = vec * type_size(type) == 16;
    const RowPlan p = plan_rows(vec, wide, a.m, a.d, 512, std::min<int64_t>(kNormPartials, 2 * static_cast<int64_t>(sm_count)));
    cudaError_t e = launch_rows<BeforeBwdKernel>(type, p, wide, a, partial_smem(p), s);
    if (e != cudaSuccess || !dw) return e;
    NormColumnArgs c{};
    c.partials = a.partials;
    c.rows = static_cast<int>(p.ctas);
    c.d = a.d;
    c.scale = 1.0f;
    c.dw = dw;
    return launch_columns(c, s);
}

cudaError_t launch_norm_after_bwd(const NormAfterBwdArgs &a, float *dw, int type, int vec, int sm_count, cudaStream_t s)
{
    const bool wide = vec * type_size(type) == 16;
    const RowPlan p = plan_rows(vec, wide, a.m, a.d, 512, std::min<int64_t>(kNormPartials, 2 * static_cast<int64_t>(sm_count)));
    cudaError_t e = launch_rows<AfterBwdKernel>(type, p, wide, a, partial_smem(p), s);
    if (e != cudaSuccess || !a.partials) return e;
    NormColumnArgs c{};
    c.partials = a.partials;
    c.rows = static_cast<int>(p.ctas);
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
