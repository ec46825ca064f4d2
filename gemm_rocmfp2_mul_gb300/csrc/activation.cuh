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
// loss of angle however long the context is (one fp64 multiply per frequency;
// error below 2^-54 turns per position for f <= 1).
RFP2_DEV uint64_t turn_fraction(float f) {
    double t = static_cast<double>(f) * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    // t rounds to 1 for a tiny negative f; the fraction wraps to 0 there
    return t < 1.0 ? __double2ull_rz(t * 18446744073709551616.0) : 0ull;
}

// (cos, sin) of position turns of `fraction`: the top 32 bits as a signed
// share of a turn (2^-32 turn = 1.5e-9 rad), then sincospi, exact in its
// argument.
RFP2_DEV float2 rotary_cos_sin(int position, uint64_t fraction) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(position)) * fraction;
    const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c, s);
}

// Host: bytes of one value, 0 for an unknown type.
inline int dtype_bytes(int dtype) {
    return dtype == RFP2_F32 ? 4 : dtype == RFP2_BF16 || dtype == RFP2_F16 ? 2 : 0;
}

}  // namespace rfp2
