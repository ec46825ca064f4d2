// Rotary positions: the first R of each head's D values turn in pairs (a, b)
// by theta = position * inv_freq[i], pairs (i, i + R/2) or (2i, 2i + 1):
//   a' = factor (a cos - b sin),  b' = factor (b cos + a sin).
// Its gradient is the same kernel with the angles negated.
//
// Bound by memory: 2 * size bytes a value against four multiplies and a share
// of a cos/sin pair.  A CTA takes a few tokens and a run of their heads.  Each
// thread first sends off its rows' loads, then the CTA computes the cos and
// sin of its (token, pair)s once into shared memory while they travel.
//
// Measured (one GB300, back to back): 16383 x 20 heads of 192, f16, 64 rotated:
// 41.4 us, 6.1 TB/s read and written (copy rate 6.8); 2048 x 40 x 128 bf16: 9.3
// us; 4 x 32 x 128 fp32: 1.9 us.  Two steps ahead at five CTAs an SM, a whole number
// of times, beat two at four (43.2 and 9.8 us), one at eight (41.5 and 9.3) and four at
// three (45.9 and 11.3); 32-bit angles from fp64 products took twice as long.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 2;        // steps of a thread whose loads travel together
constexpr int kSteps = 8;        // of a thread, about, at most
constexpr int kMaxPairs = 2048;  // (token, pair) entries of a CTA's table

struct RopeArgs {
    const void *x;
    void *out;
    const int32_t *positions;
    const float *inv_freq;
    int64_t T, xt, xh, ot, oh;
    int H, D, pairs;
    int tokens, heads;  // of a CTA
    float factor;
    int inverse;
    int turned, steps;  // steps of a row: those that turn, and those that copy what lies past R
    FastDiv by_pairs, by_steps, by_heads;
};

// 2V values of a row: V pairs, as two runs of V values.  Runs are 16 bytes, or
// (V = 1) single values of any alignment.
template <typename T, int V>
struct alignas(V * sizeof(T)) Runs {
    T u[V], w[V];
    RFP2_DEV void load(const T *p, const T *q) { copy(u, p), copy(w, q); }
    RFP2_DEV void store(T *p, T *q) const { copy(p, u), copy(q, w); }
    static RFP2_DEV void copy(T *to, const T *from) {
        if constexpr (V * sizeof(T) == 16) {
            *reinterpret_cast<uint4 *>(to) = *reinterpret_cast<const uint4 *>(from);
        } else {
            *to = *from;
        }
    }
};

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const RopeArgs a) {
    extern __shared__ __align__(16) float table[];  // [tokens][cos, sin][pairs]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int h0 = blockIdx.y * a.heads;
    const int nt = (int)min((int64_t)a.tokens, a.T - t0), nh = min(a.heads, a.H - h0);
    const int n = nt * a.heads * a.steps;

    // step i: token t, head h, values at `at` and `at2` of its row; h may lie past the last head
    const auto place = [&](int i, int &t, int &h, int &s, int &at, int &at2) {
        const int row = a.by_steps(i);
        s = i - row * a.steps;
        t = a.by_heads(row);
        h = row - t * a.heads;
        if (s < a.turned && !INTERLEAVED) {
            at = V * s;
            at2 = at + a.pairs;
        } else {
            at = 2 * V * s;
            at2 = at + V;
        }
        return i < n && h < nh;
    };
    const auto load = [&](int i, Runs<T, V> &x) {
        int t, h, s, at, at2;
        if (!place(i, t, h, s, at, at2)) return;
        const T *p = static_cast<const T *>(a.x) + (t0 + t) * a.xt + (h0 + h) * a.xh;
        x.load(p + at, p + at2);
    };
    const auto turn = [&](int i, Runs<T, V> &x) {
        int t, h, s, at, at2;
        if (!place(i, t, h, s, at, at2)) return;
        if (s < a.turned) {
            const float *cs = table + 2 * t * a.pairs;
            float c[V], sn[V];
            if constexpr (V == 1) {
                c[0] = cs[s];
                sn[0] = cs[a.pairs + s];
            } else {
#pragma unroll
                for (int w = 0; w < V / 4; ++w) {
                    const float *q = cs + (w * (a.pairs >> 3) + s) * 4;
                    const float4 u = *reinterpret_cast<const float4 *>(q);
                    const float4 v = *reinterpret_cast<const float4 *>(q + a.pairs);
                    c[4 * w] = u.x, c[4 * w + 1] = u.y, c[4 * w + 2] = u.z, c[4 * w + 3] = u.w;
                    sn[4 * w] = v.x, sn[4 * w + 1] = v.y, sn[4 * w + 2] = v.z, sn[4 * w + 3] = v.w;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // pair e: values 2e and 2e + 1 of the run of 2V, or e of each run
                T &p = INTERLEAVED ? (2 * e < V ? x.u[2 * e % V] : x.w[2 * e % V]) : x.u[e];
                T &q = INTERLEAVED ? (2 * e + 1 < V ? x.u[(2 * e + 1) % V] : x.w[(2 * e + 1) % V]) : x.w[e];
                const float u = to_f32(p), w = to_f32(q);
                p = from_f32<T>(u * c[e] - w * sn[e]);
                q = from_f32<T>(w * c[e] + u * sn[e]);
            }
        }
        T *o = static_cast<T *>(a.out) + (t0 + t) * a.ot + (h0 + h) * a.oh;
        x.store(o + at, o + at2);
    };

    Runs<T, V> x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(threadIdx.x + k * kThreads, x[k]);
    rotary_table<V, kThreads>(table, a.positions + t0, a.inv_freq, nt, a.pairs, a.by_pairs, a.factor,
                              a.inverse ? -a.factor : a.factor);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) turn(i + k * kThreads, x[k]);
        if (i + kAhead * kThreads < n)
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load(i + (kAhead + k) * kThreads, x[k]);
    }
}

template <typename T>
cudaError_t launch_rope(RopeArgs &a, bool interleaved, bool copy, cudaStream_t stream) {
    constexpr int W = 16 / sizeof(T);
    const auto even = [](int64_t v) { return v % W == 0; };
    const bool wide = aligned(a.x, 16) && aligned(a.out, 16) && even(a.xt) && even(a.xh) &&
                      even(a.ot) && even(a.oh) && even(a.pairs) && even(a.D / 2 - a.pairs);
    const int V = wide ? W : 1;
    a.turned = a.pairs / V;
    a.steps = a.turned + (copy ? (a.D / 2 - a.pairs) / V : 0);
    // Up to kSteps steps a thread: tokens share a CTA where a token's heads are fewer, and heads are
    // divided where they are more, or where there are few tokens.  The tokens are dealt so that the CTAs
    // fill the SMs, five on each, a whole number of times.
    constexpr int kMost = kSteps * kThreads;
    const int64_t at_once = 5 * (int64_t)sm_count(current_device());
    a.heads = std::max(1, std::min(a.H, kMost / std::max(1, a.steps)));
    while (a.heads > 1 && a.heads * a.steps > kThreads && a.T * ((a.H + a.heads - 1) / a.heads) < at_once)
        a.heads = (a.heads + 1) / 2;
    a.tokens = 1;
    if (a.heads == a.H) {
        const int64_t most = std::max<int64_t>(
            1, std::min(kMost / (a.heads * std::max(1, a.steps)), kMaxPairs / std::max(1, a.pairs)));
        const int64_t waves = (a.T + at_once * most - 1) / (at_once * most);
        a.tokens = (int)((a.T + at_once * waves - 1) / (at_once * waves));
    }
    a.by_pairs = FastDiv(std::max(1, a.pairs));
    a.by_steps = FastDiv(std::max(1, a.steps));
    a.by_heads = FastDiv(a.heads);
    if (a.steps == 0) return cudaSuccess;  // nothing turns, in place
    const dim3 grid((unsigned)((a.T + a.tokens - 1) / a.tokens), (a.H + a.heads - 1) / a.heads);
    const size_t smem = (size_t)a.tokens * a.pairs * 8;
    void (*k)(RopeArgs) = wide ? (interleaved ? rope_kernel<T, W, true> : rope_kernel<T, W, false>)
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
    if (D > 65536 || H > 65535 || T > (1ll << 31) - 1) return RFP2_ESHAPE;
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
    const bool copy = x != out, interleaved = (flags & RFP2_ROPE_INTERLEAVED) != 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_rope<float>(a, interleaved, copy, s)
                     : dtype == RFP2_BF16 ? launch_rope<__nv_bfloat16>(a, interleaved, copy, s)
                                          : launch_rope<__half>(a, interleaved, copy, s));
}
