// Activations in memory: fp32, bf16 or f16, read to fp32 and written back with
// one rounding, four or eight neighbouring values at a time where 16-byte
// words fit, and the rotary angles that rope.cu and kvcache.cu share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "common.cuh"

namespace rfp2 {

RFP2_DEV float to_f32(float v) { return v; }
RFP2_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
RFP2_DEV float to_f32(__half v) { return __half2float(v); }
template <typename T>
RFP2_DEV T from_f32(float v);
template <>
RFP2_DEV float from_f32<float>(float v) { return v; }
template <>
RFP2_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
RFP2_DEV __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N neighbouring values; as 16-byte words where N * sizeof(T) allows it (the
// caller has checked the alignment), else one by one.
template <typename T, int N>
RFP2_DEV void load_values(const T *p, float (&v)[N]) {
    if constexpr (N * sizeof(T) % 16 == 0) {
        constexpr int W = N * sizeof(T) / 16, E = 16 / sizeof(T);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const uint4 u = reinterpret_cast<const uint4 *>(p)[w];
            T t[E];
            memcpy(t, &u, 16);
#pragma unroll
            for (int e = 0; e < E; ++e) v[w * E + e] = to_f32(t[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = to_f32(p[e]);
    }
}

template <typename T, int N>
RFP2_DEV void store_values(T *p, const float (&v)[N]) {
    if constexpr (N * sizeof(T) % 16 == 0) {
        constexpr int W = N * sizeof(T) / 16, E = 16 / sizeof(T);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            T t[E];
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = from_f32<T>(v[w * E + e]);
            uint4 u;
            memcpy(&u, t, 16);
            reinterpret_cast<uint4 *>(p)[w] = u;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = from_f32<T>(v[e]);
    }
}

// Rotary angles.  theta = position * f in turns is position * (f / 2 pi) mod
// 1.  With f / 2 pi mod 1 as a 64-bit binary fraction, the product with an
// integer position wraps at whole turns by itself: no range reduction, and no
// loss of angle however long the context is.  The fraction is the exact
// product of f's 24 bits with 128 bits of 1 / 2 pi, in integers: fp64 is slow
// here.
RFP2_DEV uint64_t turn_fraction(float f) {
    constexpr uint64_t hi = 0x28BE60DB9391054Aull, lo = 0x7F09D5F47D4D3770ull;  // 2^128 / 2 pi
    const uint32_t bits = __float_as_uint(f), e = bits >> 23 & 255u;
    const uint64_t m = e ? (bits & 0x7FFFFFu) | 0x800000u : (bits & 0x7FFFFFu) << 1;
    // m * (hi, lo) in words w2 w1 w0, to be divided by 2^(150 - e)
    const uint64_t w0 = m * lo, c0 = __umul64hi(m, lo), p1 = m * hi, w1 = p1 + c0;
    const uint64_t w2 = __umul64hi(m, hi) + (w1 < p1);
    const int s = 150 - (int)e;
    uint64_t r;
    if (s >= 64)
        r = s >= 128 ? 0ull : w2 >> (s - 64);
    else if (s > 0)
        r = w1 >> s | w2 << (64 - s);
    else
        r = s == 0 ? w1 : s > -64 ? w1 << -s | w0 >> (64 + s) : 0ull;
    return bits >> 31 ? 0ull - r : r;
}

// (cos, sin) of position turns of `fraction`: the top 32 bits as a signed
// share of a turn (2^-32 turn = 1.5e-9 rad), of which sincospi, exact in its
// argument, takes what a float holds; the rest, up to 9.4e-8 rad, turns the result.
RFP2_DEV float2 rotary_cos_sin(int position, uint64_t fraction) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
    const int share = static_cast<int>(turn >> 32);
    const float held = static_cast<float>(share);
    const float rest = static_cast<float>(share - static_cast<int>(held)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    float s, c;
    sincospif(held * 4.656612873077393e-10f, &s, &c);
    return make_float2(fmaf(-s, rest, c), fmaf(c, rest, s));
}

// The place of pair p in a table of `pairs` cosines or sines that is read four
// to a 16-byte word.  V = 8: a thread reads eight; its first words come before
// all second words, so that neighbouring threads read neighbouring words.
template <int V>
RFP2_DEV int table_place(int p, int pairs) {
    return V == 8 ? ((p >> 2 & 1) * (pairs >> 3) + (p >> 3)) * 4 + (p & 3) : p;
}

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery 1994): with 2^(s-1) < d <= 2^s and
// mul = floor(2^32 (2^s - d) / d) + 1, n / d = (mulhi(n, mul) + n) >> s.
struct FastDiv {
    uint32_t d, mul, shift;
    FastDiv() = default;
    explicit FastDiv(uint32_t divisor) : d(divisor), shift(0) {
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    RFP2_DEV uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// The cosines and sines of tokens [0, n) of a CTA into shared memory: table
// [n][cos, sin][pairs], times factor and sine_factor; pair p at table_place<V>.
// A thread stays with its pairs, so their fractions are found once.
template <int V, int THREADS>
RFP2_DEV void rotary_table(float *table, const int32_t *positions, const float *inv_freq, int n,
                           int pairs, const FastDiv &by_pairs, float factor, float sine_factor) {
    const int row = pairs < THREADS ? (int)by_pairs(threadIdx.x) : 0;
    const int rows = pairs < THREADS ? (int)by_pairs(THREADS) : 1;
    if (row >= rows) return;
    for (int p = threadIdx.x - row * pairs; p < pairs; p += THREADS) {
        const uint64_t fraction = turn_fraction(inv_freq[p]);
        float *at = table + table_place<V>(p, pairs);
        for (int t = row; t < n; t += rows) {
            const float2 cs = rotary_cos_sin(positions[t], fraction);
            at[2 * t * pairs] = cs.x * factor;
            at[(2 * t + 1) * pairs] = cs.y * sine_factor;
        }
    }
}

// Host: bytes of one value, 0 for an unknown type.
inline int dtype_bytes(int dtype) {
    return dtype == RFP2_F32 ? 4 : dtype == RFP2_BF16 || dtype == RFP2_F16 ? 2 : 0;
}

}  // namespace rfp2
