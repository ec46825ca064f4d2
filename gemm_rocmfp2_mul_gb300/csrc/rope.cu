// Rotary positions: the first R of each head's D values turn in pairs (a, b)
// by theta = position * inv_freq[i], pairs (i, i + R/2) or (2i, 2i + 1):
//   a' = factor (a cos - b sin),  b' = factor (b cos + a sin).
// Its gradient is the same kernel with the angles negated.
//
// Bound by memory: 2 * size bytes a value against four multiplies and a share
// of a cos/sin pair.  A CTA takes a few tokens and a run of their heads: its
// threads first compute each (token, pair)'s cos and sin once into shared
// memory, then walk the heads' rows.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 2048;  // (token, pair) entries of a CTA's cos/sin table

struct RopeArgs {
    const void *x;
    void *out;
    const int32_t *positions;
    const float *inv_freq;
    int64_t T, xt, xh, ot, oh;
    int H, D, pairs;
    int tokens, heads;  // of a CTA
    float factor;
    int inverse, copy;  // copy: the values past R move to `out`
};

// V pairs a step: 2V values, as two runs of V.  V = 1 takes any alignment.
template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    extern __shared__ float2 table[];  // [tokens][pairs]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int h0 = blockIdx.y * a.heads;
    const int nt = (int)min((int64_t)a.tokens, a.T - t0), nh = min(a.heads, a.H - h0);
    for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        float2 cs = rotary_cos_sin(a.positions[t0 + t], turn_fraction(a.inv_freq[p]));
        cs.x *= a.factor;
        cs.y *= a.inverse ? -a.factor : a.factor;
        table[i] = cs;
    }
    __syncthreads();
    const int turned = a.pairs / V;  // steps that turn; V divides pairs
    const int steps = turned + (a.copy ? (a.D / 2 - a.pairs) / V : 0);
    const int n = nt * nh * steps;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int row = i / steps, s = i - row * steps;
        const int t = row / nh, h = row - t * nh;
        const T *x = static_cast<const T *>(a.x) + (t0 + t) * a.xt + (h0 + h) * a.xh;
        T *o = static_cast<T *>(a.out) + (t0 + t) * a.ot + (h0 + h) * a.oh;
        float u[V], w[V];
        if (s < turned) {
            const float2 *cs = table + t * a.pairs + s * V;
            if (INTERLEAVED) {
                load_values<T, V>(x + 2 * V * s, u);
                load_values<T, V>(x + 2 * V * s + V, w);
                float y[2 * V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    y[e] = u[e];
                    y[V + e] = w[e];
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = y[2 * e], q = y[2 * e + 1];
                    y[2 * e] = p * cs[e].x - q * cs[e].y;
                    y[2 * e + 1] = q * cs[e].x + p * cs[e].y;
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    u[e] = y[e];
                    w[e] = y[V + e];
                }
                store_values<T, V>(o + 2 * V * s, u);
                store_values<T, V>(o + 2 * V * s + V, w);
            } else {
                load_values<T, V>(x + V * s, u);
                load_values<T, V>(x + a.pairs + V * s, w);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float p = u[e], q = w[e];
                    u[e] = p * cs[e].x - q * cs[e].y;
                    w[e] = q * cs[e].x + p * cs[e].y;
                }
                store_values<T, V>(o + V * s, u);
                store_values<T, V>(o + a.pairs + V * s, w);
            }
        } else {
            const int at = 2 * a.pairs + 2 * V * (s - turned);
            load_values<T, V>(x + at, u);
            load_values<T, V>(x + at + V, w);
            store_values<T, V>(o + at, u);
            store_values<T, V>(o + at + V, w);
        }
    }
}

template <typename T>
cudaError_t launch_rope(RopeArgs &a, bool interleaved, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const auto even = [](int64_t v) { return v % V == 0; };
    const bool wide = aligned(a.x, 16) && aligned(a.out, 16) && even(a.xt) && even(a.xh) &&
                      even(a.ot) && even(a.oh) && even(a.pairs) && even(a.D / 2 - a.pairs);
    const dim3 grid((unsigned)((a.T + a.tokens - 1) / a.tokens), (a.H + a.heads - 1) / a.heads);
    const size_t smem = (size_t)a.tokens * a.pairs * sizeof(float2);
    void (*k)(RopeArgs) = wide ? (interleaved ? rope_kernel<T, V, true> : rope_kernel<T, V, false>)
                               : (interleaved ? rope_kernel<T, 1, true> : rope_kernel<T, 1, false>);
    return launch(k, grid, dim3(kThreads), smem, stream, true, a);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" rfp2_status rfp2_rope_frequencies(int64_t R, double base, int scaling, double stretch,
                                             double trained, double fast, double slow,
                                             float *inv_freq, float *factor) {
    const auto positive = [](double v) { return v > 0.0 && isfinite(v); };
    if (R < 2 || R % 2 != 0 || R > 65536 || (scaling == RFP2_ROPE_BASE && R < 4)) return RFP2_ESHAPE;
    if (!inv_freq || scaling < RFP2_ROPE_PLAIN || scaling > RFP2_ROPE_RAMP || !positive(base) ||
        !positive(stretch))
        return RFP2_EINVAL;
    if (scaling == RFP2_ROPE_RAMP &&
        (!positive(trained) || !isfinite(fast) || !isfinite(slow) || !(fast > slow)))
        return RFP2_EINVAL;
    if (scaling == RFP2_ROPE_BASE) base *= pow(stretch, (double)R / (double)(R - 2));
    for (int64_t i = 0; i < R / 2; ++i) {
        double f = pow(base, -2.0 * (double)i / (double)R);
        if (scaling == RFP2_ROPE_LINEAR) f /= stretch;
        if (scaling == RFP2_ROPE_RAMP) {
            const double turns = trained * f / 6.283185307179586477;
            const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            f = f * keep + f / stretch * (1.0 - keep);
        }
        inv_freq[i] = (float)f;
    }
    if (factor)
        *factor = scaling == RFP2_ROPE_RAMP && stretch > 1.0 ? (float)(0.1 * log(stretch) + 1.0) : 1.0f;
    return RFP2_OK;
}

extern "C" rfp2_status rfp2_rope(const void *x, int dtype, int64_t T, int64_t H, int64_t D,
                                 int64_t x_token_stride, int64_t x_head_stride,
                                 const int32_t *positions, const float *inv_freq, int64_t R,
                                 float factor, int flags, void *out, int64_t out_token_stride,
                                 int64_t out_head_stride, rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype);
    if (T < 0 || H < 0 || D < 0 || !size || (flags & ~(RFP2_ROPE_INTERLEAVED | RFP2_ROPE_INVERSE)))
        return RFP2_EINVAL;
    if (R < 0 || R % 2 != 0 || D % 2 != 0 || R > D || R > 2 * kMaxPairs) return RFP2_ESHAPE;
    if (T == 0 || H == 0 || D == 0) return RFP2_OK;
    if (D > 65536 || H > 65536 || T > (1ll << 31) - 1) return RFP2_ESHAPE;
    if (!x || !out || !positions || (R > 0 && !inv_freq)) return RFP2_EINVAL;
    if (!aligned(x, size) || !aligned(out, size) || !aligned(positions, 4) || !aligned(inv_freq, 4))
        return RFP2_EALIGN;
    RopeArgs a;
    a.x = x;
    a.out = out;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.T = T;
    a.xt = x_token_stride;
    a.xh = x_head_stride;
    a.ot = out_token_stride;
    a.oh = out_head_stride;
    a.H = (int)H;
    a.D = (int)D;
    a.pairs = (int)(R / 2);
    a.factor = factor;
    a.inverse = (flags & RFP2_ROPE_INVERSE) != 0;
    a.copy = R < D && x != out;
    a.tokens = 1;
    a.heads = 8;
    const bool interleaved = (flags & RFP2_ROPE_INTERLEAVED) != 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_rope<float>(a, interleaved, s)
                     : dtype == RFP2_BF16 ? launch_rope<__nv_bfloat16>(a, interleaved, s)
                                          : launch_rope<__half>(a, interleaved, s));
}
