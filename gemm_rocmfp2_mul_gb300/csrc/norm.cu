// Root-mean-square norm after the residual's addition:
//   s = x + residual (rounded to the activations' type), r = 1 / sqrt(mean s^2 + eps), y = s r weight,
// as values and / or in Q8 blocks.  Bound by memory: a value is read once (twice with a residual) and
// written once to three times, against about ten operations.
//
// A row belongs to a CTA, or to a warp where it is short; it stays in registers between its sum and its
// outputs.  Q8 codes are those of the formula, not of its fp32 roundings: code = round-half-away(127 u / U)
// with u = |s weight| and U a block's largest, in which r drops out.  In fp32 the quotient is off by
// 5.4e-7 of itself at most (nine roundings); where a half-integer is that near, u and U as integers (48 bits) decide.
//
// Measured (one GB300, GPU time a call): 16384 x 5120 bf16 with a residual 97.5 us, 6.9 TB/s read and written
// (the copy rate); 4999 x 1376 f16 to values and codes 15.9 us, bound by instructions; 4 x 4096 fp32 to
// codes 3.4 us.  A persistent grid took 205 us of the first: its loop kept the addresses of a row's
// values in registers that the values then lacked.  Rows of odd length or alignment above 4096 values hold 32 fp32
// values a thread of up to 1024 and spill (4999 x 5121 bf16 112 us, 0.9 TB/s), as fp32 rows with codes above 8192 do
// (2000 x 16384 68 us).
#include <algorithm>
#include <type_traits>

#include "activation.cuh"

namespace rfp2 {
namespace {

struct NormArgs {
    const void *x, *residual, *weight;
    void *total, *y;
    int8_t *q;
    float *d;
    int64_t T, xs, rs, ts, ys;
    int K, weight_type, y_type;
    float eps;
};

// V values of `type` (a uniform branch) at element `at`; four of 16 bits as one word of 8 bytes.
template <typename T, int V>
RFP2_DEV void load_run(const T *p, float (&v)[V]) {
    if constexpr (V * sizeof(T) == 8) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        T t[V];
        memcpy(t, &u, 8);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = to_f32(t[e]);
    } else {
        load_values(p, v);
    }
}
template <typename T, int V>
RFP2_DEV void store_run(T *p, const float (&v)[V]) {
    if constexpr (V * sizeof(T) == 8) {
        T t[V];
#pragma unroll
        for (int e = 0; e < V; ++e) t[e] = from_f32<T>(v[e]);
        uint2 u;
        memcpy(&u, t, 8);
        *reinterpret_cast<uint2 *>(p) = u;
    } else {
        store_values(p, v);
    }
}
template <int V>
RFP2_DEV void load_typed(const void *p, int type, int64_t at, float (&v)[V]) {
    if (type == RFP2_F32)
        load_run(static_cast<const float *>(p) + at, v);
    else if (type == RFP2_BF16)
        load_run(static_cast<const __nv_bfloat16 *>(p) + at, v);
    else
        load_run(static_cast<const __half *>(p) + at, v);
}
template <int V>
RFP2_DEV void store_typed(void *p, int type, int64_t at, const float (&v)[V]) {
    if (type == RFP2_F32)
        store_run(static_cast<float *>(p) + at, v);
    else if (type == RFP2_BF16)
        store_run(static_cast<__nv_bfloat16 *>(p) + at, v);
    else
        store_run(static_cast<__half *>(p) + at, v);
}

// Sum (or maximum) over the warps that share a row; `part` has 32 places, and successive calls take
// turns between two of them.
template <bool MAX>
RFP2_DEV float over_row(float v, int warps, float *part) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    return v;
}

// |s w| exactly, as an integer in the same order: 48 bits of significand, normalised, below the exponent.
RFP2_DEV uint64_t product_key(float s, float w) {
    const auto part = [](float v, uint32_t &m) {
        const uint32_t b = __float_as_uint(v), e = b >> 23 & 255u;
        m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
        return (int)max(e, 1u);
    };
    uint32_t ms, mw;
    const int e = part(s, ms) + part(w, mw);
    uint64_t m = (uint64_t)ms * mw;
    if (m == 0) return 0;
    const int up = __clzll((long long)m) - 16;
    return (uint64_t)(e + 64 - up) << 48 | (m << up & 0xFFFFFFFFFFFFull);
}

// Is 254 u >= c U, for keys u <= U of products and 1 <= c <= 255?
RFP2_DEV bool reaches(uint64_t u, int c, uint64_t U) {
    const int down = (int)(U >> 48) - (int)(u >> 48);
    if (u == 0 || down > 8) return false;  // 254 u < 2^56 <= 2^47 2^9
    const auto significand = [](uint64_t k) { return k & 0xFFFFFFFFFFFFull; };
    return 254u * significand(u) >= ((uint64_t)c * significand(U)) << down;
}

// The codes of the values s w of a block that 32 / V neighbouring lanes share, where they are `near` a border.
// In integers: fp64, in which a product is exact too, has two lanes an SM here, and a decode step's few rows
// waited 2 us for it.
template <int V>
__device__ __noinline__ void exact_codes(const float *s, const float *w, int8_t *code, bool near) {
    uint64_t U = 0;
#pragma unroll 1
    for (int e = 0; e < V; ++e) U = max(U, product_key(s[e], w[e]));
#pragma unroll
    for (int off = 1; off < 32 / V; off <<= 1) U = max(U, __shfl_xor_sync(0xffffffffu, U, off));
    if (!near || U == 0) return;
    const auto size = [](uint64_t k) { return (float)(k & 0xFFFFFFFFFFFFull); };
#pragma unroll 1
    for (int e = 0; e < V; ++e) {
        const uint64_t u = product_key(s[e], w[e]);
        const int down = min((int)(U >> 48) - (int)(u >> 48), 32);
        int k = u ? (int)(127.0f * (size(u) / size(U)) * __uint_as_float((127u - down) << 23) + 0.5f) : 0;
        if (k < 127 && reaches(u, 2 * k + 1, U))
            ++k;
        else if (k > 0 && !reaches(u, 2 * k - 1, U))
            --k;
        code[e] = (int8_t)((__float_as_uint(s[e]) ^ __float_as_uint(w[e])) >> 31 ? -k : k);
    }
}

// The codes of V values of a block that 32 / V neighbouring lanes share, as bytes; s and w as they are, y = s r w
// in fp32.  Returns the block's scale.  A quotient t + 1.5 2^23 has the nearest whole number, two's complement,
// in its low byte; where t is a half-integer but for its error, which one is decided exactly.
template <int V>
RFP2_DEV float block_codes(const float (&s)[V], const float (&w)[V], const float (&y)[V], uint32_t (&code)[V]) {
    constexpr int kLanes = 32 / V;
    constexpr float kWhole = 12582912.0f;
    uint32_t top = 0;  // of |y|'s bits: NaN above infinity above all else
#pragma unroll
    for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int off = 1; off < kLanes; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const float most = __uint_as_float(top), d = most * (1.0f / 127.0f);
    const bool finite = top < 0x7F800000u, any = finite && d != 0.0f;
    const float by = __fdividef(127.0f, most);  // (0 for the largest, infinity for the smallest: those are decided exactly)
    bool near = any && (most < 0x1p-90f || most > 0x1p120f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float t = y[e] * by, m = t + kWhole;
        code[e] = __float_as_uint(m);
        near |= fabsf(t - (m - kWhole)) >= fmaf(fabsf(t), -6e-7f, 0.5f);
    }
    near &= any;
    if (__any_sync(0xffffffffu, near)) {
        // (copies, so that the values themselves stay in registers)
        float cs[V], cw[V];
        int8_t k[V];
#pragma unroll
        for (int e = 0; e < V; ++e) cs[e] = s[e], cw[e] = w[e], k[e] = (int8_t)code[e];
        exact_codes<V>(cs, cw, k, near);
#pragma unroll
        for (int e = 0; e < V; ++e) code[e] = (uint8_t)k[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) code[e] = any ? code[e] : 0;
    return finite ? d : CUDART_NAN_F;
}

// Low bytes of four words.
RFP2_DEV uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// A row's values: N runs of V a thread, run i of thread t at V (i threads + t).
// At most so many threads, for the registers that their values take.
template <int V, int N>
constexpr int most_threads() {
    return (V > 1 && N == 4) || N * V > 32 || (V == 1 && N == 8) ? 512 : 1024;
}
template <typename T, int V, int N, bool Q8>
__global__ void __launch_bounds__(most_threads<V, N>(), 1) norm_kernel(const NormArgs a, int warps) {
    __shared__ float part[2][32];
    pdl_wait();
    pdl_launch_dependents();
    // warps == 1: each warp of the CTA has a row of its own
    const int lanes = warps == 1 ? 32 : blockDim.x;
    const int tid = warps == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int rows = warps == 1 ? blockDim.x >> 5 : 1;
    const int64_t row = (int64_t)blockIdx.x * rows + (warps == 1 ? threadIdx.x >> 5 : 0);
    if (row >= a.T) return;
    const T *x = static_cast<const T *>(a.x) + row * a.xs;
    const T *rest = a.residual ? static_cast<const T *>(a.residual) + row * a.rs : nullptr;
    // all loads of a row that is not too long travel together
    constexpr bool kHeld = N <= (V > 1 ? 4 : 8);
    Held<T, V> hx[N], hr[kHeld ? N : 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = V * (i * lanes + tid);
        if (at < a.K) hx[i].load(x + at);
        if constexpr (kHeld)
            if (rest && at < a.K) hr[i].load(rest + at);
    }
    float s[N][V];
    constexpr bool kEarly = N * V <= 8;  // few values: their weights are fetched before the sum, not after it
    float early[kEarly ? N : 1][V];
    if constexpr (kEarly) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = V * (i * lanes + tid);
            if (at < a.K) load_typed(a.weight, a.weight_type, at, early[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = V * (i * lanes + tid);
        const bool in = at < a.K;
        if constexpr (!kHeld)
            if (rest && in) hr[0].load(rest + at);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            s[i][e] = in ? to_f32(hx[i].v[e]) : 0.0f;
            if (rest && in) s[i][e] = to_f32(from_f32<T>(s[i][e] + to_f32(hr[kHeld ? i : 0].v[e])));
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) sum = fmaf(s[i][e], s[i][e], sum);
    sum = over_row<false>(sum, warps, part[0]);
    const float square = sum / (float)a.K + a.eps;
    float r = 1.0f / sqrtf(square);
    if (!(square < CUDART_INF_F) || sum < 0x1p-90f) {
        // squares (or their mean and eps) out of range: of values below 1 in size, by a power of two
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) most = fmaxf(most, fabsf(s[i][e]));
        most = over_row<true>(most, warps, part[1]);
        if (most > 0.0f && most < CUDART_INF_F && sum == sum) {
            int ex;
            frexpf(most, &ex);
            const float down = ldexpf(1.0f, -ex / 2), down2 = ldexpf(1.0f, -ex - -ex / 2);
            float part_sum = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float v = s[i][e] * down * down2;
                    part_sum = fmaf(v, v, part_sum);
                }
            if (warps > 1) __syncthreads();
            part_sum = over_row<false>(part_sum, warps, part[0]);
            // r = 2^-ex / sqrt(mean + eps 2^-2ex)
            const float mean = part_sum / (float)a.K + a.eps * down * down * down2 * down2;
            r = mean < CUDART_INF_F ? down * (down2 / sqrtf(mean)) : r;
        }
    }
    if (a.total && a.residual) {
        T *to = static_cast<T *>(a.total) + row * a.ts;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = V * (i * lanes + tid);
            if (at < a.K) store_values(to + at, s[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = V * (i * lanes + tid);
        if (!Q8 && at >= a.K) continue;
        float w[V], y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) w[e] = 0.0f;
        if (at < a.K) {
            if constexpr (kEarly)
                memcpy(w, early[i], sizeof(w));
            else
                load_typed(a.weight, a.weight_type, at, w);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = s[i][e] * r * w[e];
        if (a.y && at < a.K) store_typed(a.y, a.y_type, row * a.ys + at, y);
        if constexpr (Q8) {
            uint32_t code[V];
            const float d = block_codes<V>(s[i], w, y, code);
            if (at < a.K) {
                int8_t *q = a.q + row * a.K + at;
                if constexpr (V == 8)
                    *reinterpret_cast<uint2 *>(q) = make_uint2(low_bytes(code[0], code[1], code[2], code[3]),
                                                               low_bytes(code[4], code[5], code[6], code[7]));
                else if constexpr (V == 4)
                    *reinterpret_cast<uint32_t *>(q) = low_bytes(code[0], code[1], code[2], code[3]);
                else
                    *q = (int8_t)code[0];
                if ((at & 31) == 0) a.d[row * (a.K >> 5) + (at >> 5)] = d;
            }
        }
    }
}

template <typename T>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
    constexpr int W = 16 / sizeof(T);
    const auto fits = [&](const void *p, int64_t stride, int size) {
        return !p || (aligned(p, 16) && stride * size % 16 == 0);
    };
    const int ysize = a.y ? dtype_bytes(a.y_type) : 4;
    const bool wide = a.K % W == 0 && fits(a.x, a.xs, sizeof(T)) && fits(a.residual, a.rs, sizeof(T)) &&
                      fits(a.total, a.ts, sizeof(T)) && aligned(a.weight, 16) && fits(a.y, a.ys, ysize);
    const int V = wide ? W : 1;
    const int runs = (a.K + V - 1) / V;
    // Few rows: a run a thread, for the shortest wait.  Many: four, so that a row's loads travel together
    // and few warps wait for its sum; two where there are codes to make, whose registers cost more in rows at once.
    const int sms = sm_count(current_device());
    const auto warps_for = [&](int n) { return (runs + 32 * n - 1) / (32 * n); };
    int n = !wide ? 8 : a.T <= 2 * sms ? 1 : a.q ? 2 : 4;
    if (wide && n == 1 && warps_for(1) > 32) n = 2;
    if (wide && ((n == 2 && warps_for(2) > 32) || (n == 4 && warps_for(4) > 16))) n = 8;
    if (!wide && warps_for(8) > 16) n = 32;
    const int warps = warps_for(n);
    const int threads = warps == 1 ? 128 : warps * 32, rows = warps == 1 ? 4 : 1;
    const int64_t ctas = (a.T + rows - 1) / rows;
    const dim3 grid((unsigned)ctas);
    void (*k)(NormArgs, int);
    const auto pick = [&](auto q8) {
        constexpr bool Q8 = decltype(q8)::value;
        if (wide)
            k = n == 1 ? norm_kernel<T, W, 1, Q8> : n == 2 ? norm_kernel<T, W, 2, Q8> : norm_kernel<T, W, 8, Q8>;
        else
            k = n == 8 ? norm_kernel<T, 1, 8, Q8> : norm_kernel<T, 1, 32, Q8>;
        if constexpr (!Q8)
            if (n == 4) k = norm_kernel<T, W, 4, false>;
    };
    if (a.q)
        pick(std::true_type());
    else
        pick(std::false_type());
    return launch(k, grid, dim3(threads), 0, stream, true, a, warps);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" rfp2_status rfp2_rms_norm(const void *x, int dtype, int64_t T, int64_t K, int64_t x_stride,
                                     const void *residual, int64_t residual_stride, void *total,
                                     int64_t total_stride, const void *weight, int weight_dtype, float eps,
                                     void *y, int y_dtype, int64_t y_stride, int8_t *q, float *d,
                                     rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype), wsize = dtype_bytes(weight_dtype), ysize = y ? dtype_bytes(y_dtype) : 1;
    if (T < 0 || K < 0 || !size || !wsize || !ysize || !(eps > 0.0f && isfinite(eps))) return RFP2_EINVAL;
    if (K > 32768 || T > (1ll << 31) - 1 || (q && K % 32 != 0)) return RFP2_ESHAPE;
    if (T == 0 || K == 0) return RFP2_OK;
    if (!x || !weight || (!y && !q) || !q != !d || (total && !residual)) return RFP2_EINVAL;
    const auto strided = [&](const void *p, int64_t stride, int64_t least) { return !p || T == 1 || stride >= least; };
    if (!strided(x, x_stride, 0) || !strided(residual, residual_stride, 0) || !strided(total, total_stride, K) ||
        !strided(y, y_stride, K))
        return RFP2_ESHAPE;
    if (!aligned(x, size) || !aligned(residual, size) || !aligned(total, size) || !aligned(weight, wsize) ||
        !aligned(y, ysize) || !aligned(q, 16) || !aligned(d, 4))
        return RFP2_EALIGN;
    // A value is read before its place in total and y is written, and by the same thread.
    const Rows in[] = {{x, T, K * size, x_stride * size},
                       {residual, T, K * size, residual_stride * size},
                       {weight, 1, K * wsize, 0}};
    const Rows out[] = {{total, T, K * size, total_stride * size},
                        {y, T, K * ysize, y_stride * ysize},
                        {q, 1, T * K, 0},
                        {d, 1, T * (K / 32) * 4, 0}};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (out[i].meet(in[j]) && !(i < 2 && j < 2 && out[i].same(in[j]))) return RFP2_EINVAL;
        for (int j = 0; j < i; ++j)
            if (out[i].meet(out[j])) return RFP2_EINVAL;
    }
    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.total = total;
    a.y = y;
    a.q = q;
    a.d = d;
    a.T = T;
    a.xs = x_stride;
    a.rs = residual_stride;
    a.ts = total_stride;
    a.ys = y_stride;
    a.K = (int)K;
    a.weight_type = weight_dtype;
    a.y_type = y_dtype;
    a.eps = eps;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_norm<float>(a, st)
                     : dtype == RFP2_BF16 ? launch_norm<__nv_bfloat16>(a, st)
                                          : launch_norm<__half>(a, st));
}
