// q4mm_rows.cuh -- what the kernels over rows of activations share: typed
// vector loads and stores, sums over the threads of a row, the int8 coding of
// a row, and the choice of vector width and threads a row.
//
// A row of d values is held by G threads: a warp (several rows a CTA) or the
// whole CTA (one row). Vector i of thread t covers the elements
// (i * G + t) * V .. + V - 1, so every load and store of a warp is contiguous.
// The first NV vectors of a thread stay in registers; a row longer than
// G * NV * V is finished by a loop that reads the remaining vectors again
// where they are needed.
#pragma once

#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q4mm_device.cuh"

namespace q4 {

// ------------------------------------------------------- typed elements --

// Rounded once, to nearest even.
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V elements of type T, moved by one access of V * sizeof(T) bytes and held as
// words: an array of 16-bit elements would take a register each.
template <typename T, int V, int B = static_cast<int>(sizeof(T)) * V> struct Pack {
    using Word = uint32_t;
    static constexpr int kWords = B / 4;
    Word w[kWords];
};
template <typename T, int V> struct Pack<T, V, 2> {
    using Word = uint16_t;
    static constexpr int kWords = 1;
    Word w[1];
};
template <typename T, int V> struct Pack<T, V, 1> {
    using Word = uint8_t;
    static constexpr int kWords = 1;
    Word w[1];
};

// Element i (a constant where it matters) in fp32.
template <typename T, int V> __device__ __forceinline__ float elem(const Pack<T, V> &p, int i)
{
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(p.w[i]);
    } else {
        const uint32_t u = V == 1 ? p.w[0] : p.w[i / 2] >> (16 * (i & 1));
        if constexpr (__is_same(T, __nv_bfloat16)) return __uint_as_float(V > 1 && (i & 1) ? p.w[i / 2] & 0xFFFF0000u : u << 16);
        else return __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
    }
}
template <typename T> __device__ __forceinline__ uint32_t bits16(float f)
{
    if constexpr (__is_same(T, __nv_bfloat16)) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    else return __half_as_ushort(__float2half_rn(f));
}
template <typename T, int V> __device__ __forceinline__ Pack<T, V> pack_of(const float (&f)[V])
{
    Pack<T, V> p;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) p.w[i] = __float_as_uint(f[i]);
    } else if constexpr (V == 1) {
        p.w[0] = static_cast<uint16_t>(bits16<T>(f[0]));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            if constexpr (__is_same(T, __nv_bfloat16)) p.w[i / 2] = pack_bf16x2_rn(f[i], f[i + 1]);
            else p.w[i / 2] = bits16<T>(f[i]) | bits16<T>(f[i + 1]) << 16;
        }
    }
    return p;
}
// Two fp32 values in a register pair, and the packed arithmetic on them (each
// half rounded once, as by itself): one issue slot for two operations.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float lo, float hi)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(F2 v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_sum(F2 v)
{
    float lo, hi;
    f2_split(v, lo, hi);
    return lo + hi;
}
// Elements 2 i and 2 i + 1.
template <typename T, int V> __device__ __forceinline__ F2 pair(const Pack<T, V> &p, int i) { return f2(elem(p, 2 * i), elem(p, 2 * i + 1)); }
template <typename T, int V> __device__ __forceinline__ Pack<T, V> pack_pairs(const F2 (&f)[V / 2])
{
    float e[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f2_split(f[i], e[2 * i], e[2 * i + 1]);
    return pack_of<T, V>(e);
}

// V int8 codes as the bytes of their words.
template <int V> __device__ __forceinline__ Pack<int8_t, V> pack_codes(const int (&c)[V])
{
    Pack<int8_t, V> p;
    if constexpr (V == 1) {
        p.w[0] = static_cast<uint8_t>(c[0]);
    } else if constexpr (V == 2) {
        p.w[0] = static_cast<uint16_t>((c[0] & 0xFF) | (c[1] & 0xFF) << 8);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            p.w[i / 4] = static_cast<uint32_t>(c[i] & 0xFF) | static_cast<uint32_t>(c[i + 1] & 0xFF) << 8 |
                         static_cast<uint32_t>(c[i + 2] & 0xFF) << 16 | static_cast<uint32_t>(c[i + 3]) << 24;
    }
    return p;
}

template <int B> struct AccessOf;
template <> struct AccessOf<16> { using type = uint4; };
template <> struct AccessOf<8> { using type = uint2; };
template <> struct AccessOf<4> { using type = uint32_t; };
template <> struct AccessOf<2> { using type = uint16_t; };
template <> struct AccessOf<1> { using type = uint8_t; };

template <typename T, int V> __device__ __forceinline__ Pack<T, V> zero_pack()
{
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < Pack<T, V>::kWords; ++i) p.w[i] = 0;
    return p;
}
// Elements c .. c + V - 1 of a row of d, zeros past its end. row + c is aligned to
// the pack.
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_pack(const T *row, int64_t c, int64_t d)
{
    using A = typename AccessOf<static_cast<int>(sizeof(T)) * V>::type;
    Pack<T, V> p;
    if (c + V <= d) {
        const A v = *reinterpret_cast<const A *>(row + c);
        memcpy(p.w, &v, sizeof(A));
    } else {
        p = zero_pack<T, V>();
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < d) {
                if constexpr (sizeof(T) == 4) p.w[i] = reinterpret_cast<const uint32_t *>(row)[c + i];
                else if constexpr (V == 1) p.w[0] = reinterpret_cast<const uint16_t *>(row)[c];
                else p.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(row)[c + i]) << (16 * (i & 1));
            }
    }
    return p;
}
template <typename T, int V, bool ANY = false>
__device__ __forceinline__ void store_pack(T *row, int64_t c, int64_t d, const Pack<T, V> &p)
{
    using A = typename AccessOf<static_cast<int>(sizeof(T)) * V>::type;
    // ANY: codes beside values whose vectors are aligned; theirs may not be
    if (c + V <= d && (!ANY || (reinterpret_cast<uintptr_t>(row + c) & (sizeof(A) - 1)) == 0)) {
        A v;
        memcpy(&v, p.w, sizeof(A));
        *reinterpret_cast<A *>(row + c) = v;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < d) {
                if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t *>(row)[c + i] = p.w[i];
                else if constexpr (sizeof(T) == 2)
                    reinterpret_cast<uint16_t *>(row)[c + i] =
                        static_cast<uint16_t>(V == 1 ? p.w[0] : p.w[i / 2] >> (16 * (i & 1)));
                else
                    reinterpret_cast<uint8_t *>(row)[c + i] =
                        static_cast<uint8_t>(V <= 2 ? p.w[0] >> (8 * i) : p.w[i / 4] >> (8 * (i & 3)));
            }
    }
}

// Sixteen bytes at any 2-byte boundary: bytes by .. by + 15 of two neighbouring
// aligned words.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, int by)
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const int r = 8 * (by & 3);
    switch (by >> 2) {   // the same for a whole row
    case 0: return make_uint4(__funnelshift_r(w[0], w[1], r), __funnelshift_r(w[1], w[2], r), __funnelshift_r(w[2], w[3], r),
                              __funnelshift_r(w[3], w[4], r));
    case 1: return make_uint4(__funnelshift_r(w[1], w[2], r), __funnelshift_r(w[2], w[3], r), __funnelshift_r(w[3], w[4], r),
                              __funnelshift_r(w[4], w[5], r));
    case 2: return make_uint4(__funnelshift_r(w[2], w[3], r), __funnelshift_r(w[3], w[4], r), __funnelshift_r(w[4], w[5], r),
                              __funnelshift_r(w[5], w[6], r));
    default: return make_uint4(__funnelshift_r(w[3], w[4], r), __funnelshift_r(w[4], w[5], r), __funnelshift_r(w[5], w[6], r),
                               __funnelshift_r(w[6], w[7], r));
    }
}
// Eight 16-bit elements from element c of a row that starts anywhere, all of
// them the row's. Each aligned word that is read holds one of them, so it lies in
// the row's allocation.
template <typename T> __device__ __forceinline__ Pack<T, 8> load_anywhere(const T *row, int64_t c)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + c);
    const int by = static_cast<int>(at & 15);
    const uint4 *in = reinterpret_cast<const uint4 *>(at - by);
    uint4 v = in[0];
    if (by) v = shifted(v, in[1], by);
    Pack<T, 8> p;
    p.w[0] = v.x, p.w[1] = v.y, p.w[2] = v.z, p.w[3] = v.w;
    return p;
}

// Element c of a row, and its store; the stored value.
template <typename T> __device__ __forceinline__ float load_elem(const T *row, int c) { return elem(load_pack<T, 1>(row, c, c + 1), 0); }
template <typename T> __device__ __forceinline__ float store_elem(T *row, int c, float v)
{
    const float f[1] = {v};
    const Pack<T, 1> p = pack_of<T, 1>(f);
    store_pack<T, 1>(row, c, c + 1, p);
    return elem(p, 0);
}

// V fp32 parameters (weights or gates of the channels) at c, zeros past the end.
// Their base is aligned to min(16, 4 V) bytes; ANY: it and c are not, all V are in
// the row, and the aligned words that hold one of them are shifted.
template <int V, bool ANY = false> __device__ __forceinline__ void load_params(const float *p, int64_t c, int64_t d, float out[V])
{
    if constexpr (ANY) {
        constexpr int W = V / 4 + 1;
        const int by = static_cast<int>(reinterpret_cast<uintptr_t>(p + c) >> 2 & 3);   // the same for a whole row
        const float4 *in = reinterpret_cast<const float4 *>(p + c - by);
        float f[4 * W];
#pragma unroll
        for (int k = 0; k < W; ++k) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < W - 1 || by) v = __ldg(in + k);
            f[4 * k] = v.x, f[4 * k + 1] = v.y, f[4 * k + 2] = v.z, f[4 * k + 3] = v.w;
        }
        const auto take = [&](int s) {
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = f[s + i];
        };
        switch (by) {
        case 0: take(0); break;
        case 1: take(1); break;
        case 2: take(2); break;
        default: take(3); break;
        }
    } else if (c + V <= d) {
        if constexpr (V % 4 == 0) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(p + c + i));
                out[i] = f.x, out[i + 1] = f.y, out[i + 2] = f.z, out[i + 3] = f.w;
            }
        } else if constexpr (V == 2) {
            const float2 f = __ldg(reinterpret_cast<const float2 *>(p + c));
            out[0] = f.x, out[1] = f.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = __ldg(p + c + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = c + i < d ? __ldg(p + c + i) : 0.0f;
    }
}

// ---------------------------------------------------------- row reductions --

// Sums and maxima over the G threads of a row: a shuffle tree in each warp,
// then, where a row takes the whole CTA, the warps' values through shared
// memory, which every thread adds in the same order, so all hold the same bits
// (four warps a vector load: a second shuffle tree would take three times as
// long, and a row waits for its sums). Two buffers in turn: a
// thread reaches the second use of a buffer only past the barrier of the use
// between, which follows every read of the first.
constexpr int kReduceFloats = 2 * 4 * 32;   // shared floats of a reducer
struct RowReducer {
    float *buf;   // [2][4][32], 16-byte aligned
    int warps;    // warps of a row; 1: no shared memory, no barrier
    bool part;    // the CTA has other warps too: the row's meet at a barrier of their own
    int turn = 0;

    // once, by every thread of the CTA or of the row, before a barrier of theirs
    __device__ __forceinline__ void clear(int threads) const
    {
        for (int i = threadIdx.x; i < kReduceFloats; i += threads) buf[i] = 0.0f;
    }
    __device__ __forceinline__ void meet() const
    {
        if (part) asm volatile("bar.sync 1, %0;" ::"r"(warps * 32) : "memory");
        else __syncthreads();
    }

    template <int N> __device__ __forceinline__ void sum(float (&v)[N])
    {
        static_assert(N <= 4, "four sums at most");
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
        if (warps == 1) return;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        float *b = buf + turn * 128;
        turn ^= 1;
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
        meet();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float t = 0.0f;
            for (int w = 0; w < warps; w += 4) {   // zeros past the last warp
                const float4 p = *reinterpret_cast<const float4 *>(b + i * 32 + w);
                t += p.x, t += p.y, t += p.z, t += p.w;
            }
            v[i] = t;
        }
    }

    // the largest of unsigned words (the bits of absolute values)
    __device__ __forceinline__ uint32_t max_bits(uint32_t v)
    {
        // (words past the last warp stay zeros here too)
        v = __reduce_max_sync(0xFFFFFFFFu, v);
        if (warps == 1) return v;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        uint32_t *b = reinterpret_cast<uint32_t *>(buf + turn * 128);
        turn ^= 1;
        if (lane == 0) b[warp] = v;
        meet();
        return __reduce_max_sync(0xFFFFFFFFu, b[lane]);
    }
};

// 1 / sqrt(sum / d + eps); the hardware's reciprocal root is within two units in
// the last place, an IEEE root and quotient would be a few hundred clocks on
// every row's way.
__device__ __forceinline__ float rms_factor(float sum, float inv_d, float eps) { return rsqrtf(fmaf(sum, inv_d, eps)); }

// ------------------------------------------------------------- int8 codes --

// Scale s = amax / 127 and factor 127 / amax of a row whose largest |x| has
// the bits `amax_bits`, each one IEEE quotient. Below 2^-110 the factor could
// overflow and s be subnormal: such a row codes to zeros with s = 0. A row
// holding a NaN or an infinity codes to zeros with s = NaN, so that its
// outputs are NaN.
struct CodeScale {
    float scale, factor;
};
__device__ __forceinline__ CodeScale code_scale(uint32_t amax_bits)
{
    CodeScale c;
    if (amax_bits >= 0x7F800000u) {
        c.scale = __uint_as_float(0x7FC00000u);
        c.factor = 0.0f;
    } else if (amax_bits < 0x08800000u) {   // 2^-110
        c.scale = 0.0f;
        c.factor = 0.0f;
    } else {
        const float amax = __uint_as_float(amax_bits);
        c.scale = __fdiv_rn(amax, 127.0f);
        c.factor = __fdiv_rn(127.0f, amax);
    }
    return c;
}
// round-half-even(x * factor), |code| <= 127; 0 where the row's factor is 0.
__device__ __forceinline__ int code_of(float x, float factor)
{
    return factor == 0.0f ? 0 : __float2int_rn(__fmul_rn(x, factor));
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

} // namespace q4
