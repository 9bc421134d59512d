// q4mm_norm.cuh -- device code shared by the norms' kernels: the general ones
// (q4mm_norm.cu) and those that stream aligned rows through shared memory
// (q4mm_norm_stream.cu).
#pragma once

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

// The channels' weights (with what else is a factor of the channel). A CTA that
// takes many rows keeps them in registers where they are few: read again for
// every row from the first-level cache, fp32 next to 16-bit values, they cost
// more loads than the rows themselves.
template <int V, int NV, bool KEEP> struct Channels {
    static constexpr bool kKept = KEEP && NV * V <= 16;
    float kept[kKept ? NV : 1][V];
    template <typename F> __device__ __forceinline__ void fill(const RowGroup &g, F at)
    {
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < NV; ++i) at((i * g.G + g.t) * V, kept[i]);
        }
    }
    // those of vector i, at element c
    template <typename F> __device__ __forceinline__ void get(int i, int c, F at, float (&out)[V]) const
    {
        if constexpr (kKept) {
#pragma unroll
            for (int j = 0; j < V; ++j) out[j] = kept[i][j];
        } else {
            at(c, out);
        }
    }
};

template <typename T, int V, int NV>
__device__ __forceinline__ void load_row(Pack<T, V> (&x)[NV], const T *row, int t, int G, int d)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * G + t) * V;
        x[i] = c < d ? load_pack<T, V>(row, c, d) : zero_pack<T, V>();
    }
}

// (o + w) of V channels.
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

template <typename T, int V> __device__ __forceinline__ float square_sum(const Pack<T, V> &x, float s)
{
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float f = elem(x, j);
        s = fmaf(f, f, s);
    }
    return s;
}
// The largest |h| of the vector's elements that the row has.
template <int V> __device__ __forceinline__ uint32_t largest(const float h[V], int c, int d, uint32_t mb)
{
#pragma unroll
    for (int j = 0; j < V; ++j) mb = max(mb, c + j < d ? abs_bits(h[j]) : 0u);
    return mb;
}
template <int V> __device__ __forceinline__ void store_codes(int8_t *row, int c, int d, const float h[V], float factor)
{
    int q[V];
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = code_of(h[j], factor);
    store_pack<int8_t, V>(row, c, d, pack_codes<V>(q));
}

// The second half of a row whose sum is known: h = x * r * (o + w), stored as
// values or coded. Vector i is x[i]; vectors past NV are `again(c)`.
template <typename T, int V, int NV, bool KEEP, typename Again>
__device__ __forceinline__ void write_normed(const Pack<T, V> (&x)[NV], Again again, float r, const NormOut &o,
                                             const Channels<V, NV, KEEP> &ch, int64_t row, const RowGroup &g, int d,
                                             RowReducer &red)
{
    const auto at = [&](int c, float (&w)[V]) { channel_weights<V>(o.w, o.w_off, c, d, w); };
    const auto normed = [&](int i, const Pack<T, V> &v, int c, float (&h)[V]) {
        float w[V];
        if (i < 0) at(c, w);
        else ch.get(i, c, at, w);
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = elem(v, j) * r * w[j];
    };
    const int rest = (NV * g.G + g.t) * V;
    float h[V];
    if (!o.codes) {
        T *out = static_cast<T *>(o.H) + row * o.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * g.G + g.t) * V;
            if (c >= d) continue;
            normed(i, x[i], c, h);
            store_pack<T, V>(out, c, d, pack_of<T, V>(h));
        }
        for (int c = rest; c < d; c += g.G * V) {
            normed(-1, again(c), c, h);
            store_pack<T, V>(out, c, d, pack_of<T, V>(h));
        }
        return;
    }
    uint32_t mb = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * g.G + g.t) * V;
        if (c >= d) continue;
        normed(i, x[i], c, h);
        mb = largest<V>(h, c, d, mb);
    }
    for (int c = rest; c < d; c += g.G * V) {
        normed(-1, again(c), c, h);
        mb = largest<V>(h, c, d, mb);
    }
    const CodeScale cs = code_scale(red.max_bits(mb));
    if (g.t == 0) o.h_scale[row] = cs.scale;
    int8_t *out = static_cast<int8_t *>(o.H) + row * o.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * g.G + g.t) * V;
        if (c >= d) continue;
        normed(i, x[i], c, h);
        store_codes<V>(out, c, d, h, cs.factor);
    }
    for (int c = rest; c < d; c += g.G * V) {
        normed(-1, again(c), c, h);
        store_codes<V>(out, c, d, h, cs.factor);
    }
}

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
            if (V % 4 == 0 && (d & 3) == 0) {   // a partial row starts on 16 bytes
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    if (c + j < d)
                        *reinterpret_cast<float4 *>(out + c + j) = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < d) out[c + j] = acc[i][j];
            }
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

} // namespace
} // namespace q4
