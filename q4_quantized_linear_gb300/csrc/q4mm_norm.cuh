// q4mm_norm.cuh -- device code shared by the norms' kernels: the general ones
// (q4mm_norm.cu) and those that stream rows through shared memory
// (q4mm_norm_stream.cuh).
#pragma once

#include "q4mm_norm.h"
#include "q4mm_rows.cuh"

namespace q4 {
namespace {

// Which rows this thread works on, and where in them. Where rows start anywhere
// (ANY) their vectors are the aligned 16-byte words inside them, the same elements
// in every matrix of the call; the few elements before and after those are dealt to
// lanes of the row's last warp, one each. (Edge vectors masked and stored element
// by element were on every row's way: join 4000 x 3999 bf16 49 us, so 34.)
struct RowGroup {
    int t, G;                 // thread of the row, threads of a row
    int64_t row, step;        // first row, rows between two of this group's
    int first = 0, end = 0;   // elements of the vectors
    int loose = -1;           // this thread's element outside them, or -1

    template <int V> __device__ __forceinline__ int at(int i) const { return first + (i * G + t) * V; }   // vector i
    template <bool ANY, typename T> __device__ __forceinline__ void begin(const T *r, int d)
    {
        end = d;
        if (!ANY) return;
        constexpr int V = 16 / sizeof(T);
        first = min(d, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(r) & 15)) & 15) / static_cast<int>(sizeof(T)));
        end = first + (d - first) / V * V;
        const int l = t - (G - 32);
        loose = l < 0 ? -1 : l < first ? l : end + l - first < d ? end + l - first : -1;
    }
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
    float kept[kKept ? NV : 1][V] = {};
    template <typename F> __device__ __forceinline__ void fill(const RowGroup &g, F at)
    {
        if constexpr (kKept) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (g.template at<V>(i) < g.end) at(g.template at<V>(i), kept[i]);
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
__device__ __forceinline__ void load_row(Pack<T, V> (&x)[NV], const T *row, const RowGroup &g, int d)
{
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.at<V>(i);
        x[i] = c < g.end ? load_pack<T, V>(row, c, d) : zero_pack<T, V>();
    }
}

// (o + w) of V channels.
template <int V, bool ANY> __device__ __forceinline__ void channel_weights(const float *w, float off, int c, int d, float out[V])
{
    if (w) {
        load_params<V, ANY>(w, c, d, out);
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] += off;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = 1.0f;
    }
}

// (o + w) of one channel.
__device__ __forceinline__ float channel_weight(const float *w, float off, int c) { return w ? __ldg(w + c) + off : 1.0f; }

// Packed arithmetic on 16-bit values' pairs (join 16384 x 1000 bf16: 41 -> 39 us); fp32
// by elements (2000 x 16384: 123 us, by pairs 129).
template <typename T, int V> constexpr bool kPairs = sizeof(T) == 2 && V > 1;

template <typename T, int V> __device__ __forceinline__ float square_sum(const Pack<T, V> &x, float s)
{
    if constexpr (kPairs<T, V>) {
        F2 q = 0;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) q = f2_fma(pair(x, j), pair(x, j), q);
        return s + f2_sum(q);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) s = fmaf(elem(x, j), elem(x, j), s);
        return s;
    }
}
// a[j] * q * w[j] [+ r[j]].
template <typename T, int V> __device__ __forceinline__ void scaled(const Pack<T, V> &a, float q, const float (&w)[V], float (&out)[V])
{
    if constexpr (kPairs<T, V>) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j)
            f2_split(f2_mul(f2_mul(pair(a, j), f2(q, q)), f2(w[2 * j], w[2 * j + 1])), out[2 * j], out[2 * j + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = elem(a, j) * q * w[j];
    }
}
template <typename T, int V>
__device__ __forceinline__ void scaled_sum(const Pack<T, V> &a, float q, const float (&w)[V], const Pack<T, V> &r, float (&out)[V])
{
#pragma unroll
    for (int j = 0; j < V / 2; ++j)
        f2_split(f2_fma(f2_mul(pair(a, j), f2(q, q)), f2(w[2 * j], w[2 * j + 1]), pair(r, j)), out[2 * j], out[2 * j + 1]);
}
// The largest |h| of the vector's elements that the row has.
template <int V> __device__ __forceinline__ uint32_t largest(const float h[V], int c, int d, uint32_t mb)
{
#pragma unroll
    for (int j = 0; j < V; ++j) mb = max(mb, c + j < d ? abs_bits(h[j]) : 0u);
    return mb;
}
template <int V, bool ANY> __device__ __forceinline__ void store_codes(int8_t *row, int c, int d, const float h[V], float factor)
{
    int q[V];
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] = code_of(h[j], factor);
    store_pack<int8_t, V, ANY>(row, c, d, pack_codes<V>(q));
}

// The second half of a row whose sum is known: h = x * r * (o + w), stored as
// values or coded. Vector i is x[i]; vectors past NV are `again(c)`; `alone` is the
// thread's element outside the vectors.
template <typename T, int V, int NV, bool KEEP, bool ANY, typename Again>
__device__ __forceinline__ void write_normed(const Pack<T, V> (&x)[NV], Again again, float alone, float r, const NormOut &o,
                                             const Channels<V, NV, KEEP> &ch, int64_t row, const RowGroup &g, int d,
                                             RowReducer &red)
{
    const auto at = [&](int c, float (&w)[V]) { channel_weights<V, ANY>(o.w, o.w_off, c, d, w); };
    const auto normed = [&](int i, const Pack<T, V> &v, int c, float (&h)[V]) {
        float w[V];
        if (i < 0) at(c, w);
        else ch.get(i, c, at, w);
        scaled<T, V>(v, r, w, h);
    };
    const int rest = g.at<V>(NV);
    const float ha = g.loose >= 0 ? alone * r * channel_weight(o.w, o.w_off, g.loose) : 0.0f;
    float h[V];
    if (!o.codes) {
        T *out = static_cast<T *>(o.H) + row * o.ldh;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (c >= g.end) continue;
            normed(i, x[i], c, h);
            store_pack<T, V>(out, c, d, pack_of<T, V>(h));
        }
        for (int c = rest; c < g.end; c += g.G * V) {
            normed(-1, again(c), c, h);
            store_pack<T, V>(out, c, d, pack_of<T, V>(h));
        }
        if (g.loose >= 0) store_elem<T>(out, g.loose, ha);
        return;
    }
    uint32_t mb = abs_bits(ha);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.at<V>(i);
        if (c >= g.end) continue;
        normed(i, x[i], c, h);
        mb = largest<V>(h, c, d, mb);
    }
    for (int c = rest; c < g.end; c += g.G * V) {
        normed(-1, again(c), c, h);
        mb = largest<V>(h, c, d, mb);
    }
    const CodeScale cs = code_scale(red.max_bits(mb));
    if (g.t == 0) o.h_scale[row] = cs.scale;
    int8_t *out = static_cast<int8_t *>(o.H) + row * o.ldh;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = g.at<V>(i);
        if (c >= g.end) continue;
        normed(i, x[i], c, h);
        store_codes<V, ANY>(out, c, d, h, cs.factor);
    }
    for (int c = rest; c < g.end; c += g.G * V) {
        normed(-1, again(c), c, h);
        store_codes<V, ANY>(out, c, d, h, cs.factor);
    }
    if (g.loose >= 0) out[g.loose] = static_cast<int8_t>(code_of(ha, cs.factor));
}

// Adds the CTA's groups' column sums (one group: its registers as they are)
// into row blockIdx.x of the partials. The tail past the registers has been
// added there already.
template <int V, int NV, bool ANY>
__device__ __forceinline__ void write_partials(float (&acc)[NV][V], float alone, float *partials, const RowGroup &g, int d,
                                               float *smem)
{
    float *out = partials + static_cast<int64_t>(blockIdx.x) * d;
    const int groups = static_cast<int>(blockDim.x) / g.G;
    if (groups == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = g.at<V>(i);
            if (!ANY && V % 4 == 0 && (d & 3) == 0) {   // a partial row starts on 16 bytes
#pragma unroll
                for (int j = 0; j < V; j += 4)
                    if (c + j < d)
                        *reinterpret_cast<float4 *>(out + c + j) = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (c + j < g.end) out[c + j] = acc[i][j];
            }
        }
        if (g.loose >= 0) out[g.loose] = alone;
        return;
    }
    const int width = d;
    const int mine = static_cast<int>(threadIdx.x) / g.G;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = g.at<V>(i) + j;
            if (c < g.end) smem[mine * width + c] = acc[i][j];
        }
    if (g.loose >= 0) smem[mine * width + g.loose] = alone;
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float s = 0.0f;
        for (int k = 0; k < groups; ++k) s += smem[k * width + c];
        out[c] = s;
    }
}

} // namespace
} // namespace q4
