// The router: the top_k experts of each token and their weights, from its logits.
//   score = softmax(x) or 1 / (1 + exp(-x));  value = score + bias;  groups of experts by the sum of their
//   group_top largest values;  the top_k largest values of the kept groups;  weights = scores.
//
// A warp has a token, lane l its experts l, l + 32, ...; a pick is the largest value over the warp (one
// redux of order-preserving integers) and the lowest index that has it (another).
//
// What is chosen is what the formula in 64 bits chooses.  Without a bias values are compared by their
// logits, exactly.  With one, picks whose fp32 values are further apart than twice what such a value may be off by
// (`slack` below) are in their true order; a run of nearer ones is taken to its end, past top_k, and put in
// order by values in fp64, one of them a lane.  What that cannot settle (a run of more than a warp's
// lanes; groups too near to tell apart) is done by fp64 values of all experts.
//
// Bound by instructions, not by the logits' bytes: about 1500 a token with a bias, groups and eight picks.
// Measured (one GB300, GPU time a call): 16384 x 256, sigmoid, bias, 4 of 8 groups, 8 experts: 33 us, four tokens of
// it 3.7 us; 4 x 256 softmax 2.5 us; 4999 x 60 3.0 us.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kWarps = 4;  // tokens of a CTA
constexpr unsigned kAll = 0xffffffffu;

struct RouteArgs {
    const void *logits;
    const float *bias;
    int32_t *ids;
    float *weights;
    int64_t T, stride;
    int E, top_k, groups, keep, group_top, group_size, renormalise;
    float scale;
    FastDiv by_size;  // experts of a group
};

// fp32 as integers in the same order, -0 as 0; -infinity is 0x007FFFFF, and 0 is below all of them.
RFP2_DEV uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
RFP2_DEV float unordered(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); }

RFP2_DEV float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return (x >= 0.0f ? 1.0f : e) / (1.0f + e);
}
// What experts are compared by at first: off by 5e-7 at most (__expf of -|x| by (2 + 1.2 |x|) 2^-23 of itself, which
// is largest at 0; the quotient 2 ulp), in a third of the instructions.
RFP2_DEV float near_sigmoid(float x) {
    const float e = __expf(-fabsf(x));
    return __fdividef(x >= 0.0f ? 1.0f : e, 1.0f + e);
}
// exp(x - y): what the difference loses to rounding (up to 2^-18 where it is 64) is put back to first order.
RFP2_DEV float exp_of_difference(float x, float y) {
    const float d = x - y, back = d - x, lost = (x - (d - back)) - (y + back);
    const float e = expf(d);
    return e > 0.0f ? fmaf(e, lost, e) : 0.0f;  // (0: the difference may be infinite)
}
RFP2_DEV double sigmoid(double x) { return 1.0 / (1.0 + exp(-x)); }

RFP2_DEV float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}
RFP2_DEV double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}

// Twice how far a value in fp32 may be off.  A softmax score is off by 1.2e-6 at most, absolutely (of itself a small
// one by far more): its exponential's (2 + 1.2 d) 2^-23 e^-d at distance d from the top is largest at d = 0, the
// rounding of d adds at most 2^-25, the sum is off by ten levels of 2^-24 and by what its terms are, which share
// what a score of 1 leaves, and reciprocal and product round once each.  A sigmoid is off by 5e-7 (near_sigmoid).
// Their sum with the bias is rounded.
template <bool SOFTMAX>
RFP2_DEV float slack(float v) { return (SOFTMAX ? 2.4e-6f : 1e-6f) + 1.3e-7f * fabsf(v); }

// Does pair (v, i) come before (w, j)?
template <typename F>
RFP2_DEV bool before(F v, int i, F w, int j) {
    return v > w || (v == w && i < j);
}

// fp64 as integers in the same order (fp64 comparisons are as slow as fp64 sums here); 0: not to be chosen.
RFP2_DEV uint64_t ordered(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);  // -0 is 0
    return v == -CUDART_INF ? 0ull : b >> 63 ? ~b : b | 1ull << 63;
}
RFP2_DEV double unordered(uint64_t k) {
    return k ? __longlong_as_double((long long)(k >> 63 ? k & ~(1ull << 63) : ~k)) : -CUDART_INF;
}

// What experts are chosen by, in fp64, for rows with near ties that fp32 cannot settle: values[e] is the ordered
// score, with the bias if there is one.
template <typename T, bool SOFTMAX>
__device__ __noinline__ void exact_values(const RouteArgs &a, const T *x, uint64_t *values, int lane) {
    double top = 0.0, total = 1.0;
    if (SOFTMAX) {
        float m = -CUDART_INF_F;
        for (int e = lane; e < a.E; e += 32) m = fmaxf(m, to_f32(x[e]));
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, off));
        top = m;
        total = 0.0;
        for (int e = lane; e < a.E; e += 32)
            if (to_f32(x[e]) > -CUDART_INF_F) total += exp((double)to_f32(x[e]) - top);
        total = warp_sum(total);
    }
    __syncwarp();
#pragma unroll 2
    for (int e = lane; e < a.E; e += 32) {
        const double l = to_f32(x[e]);
        double v = SOFTMAX ? exp(l - top) / total : sigmoid(l);
        if (a.bias) v += (double)a.bias[e];
        values[e] = l > -CUDART_INF ? ordered(v) : 0ull;
    }
    __syncwarp();
}

// The groups that are kept, a bit each, by values in fp64.  (`values`: a place for E numbers, here and below.)
template <typename T, bool SOFTMAX>
__device__ __noinline__ unsigned keep_exactly(const RouteArgs &a, const T *x, uint64_t *values, int lane) {
    exact_values<T, SOFTMAX>(a, x, values, lane);
    uint64_t mine = 0;  // lane g: what group g counts
    for (int g = 0; g < a.groups; ++g) {
        uint64_t b1 = 0, b2 = 0;
        for (int e = g * a.group_size + lane; e < (g + 1) * a.group_size; e += 32) {
            const uint64_t v = values[e];
            b2 = max(b2, min(b1, v));
            b1 = max(b1, v);
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const uint64_t o1 = __shfl_xor_sync(kAll, b1, off), o2 = __shfl_xor_sync(kAll, b2, off);
            b2 = max(min(b1, o1), max(b2, o2));
            b1 = max(b1, o1);
        }
        if (a.group_top > 1 && b2) b1 = ordered(unordered(b1) + unordered(b2));
        if (lane == g) mine = b1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const uint64_t o = __shfl_sync(kAll, mine, g);
        rank += before(o, g, mine, lane);
    }
    return __ballot_sync(kAll, lane < a.groups && rank < a.keep && mine);
}

// Lane j's pick j of the kept groups' experts (-1: none), by values in fp64 (of a call with a bias: without one
// picks are certain).
template <typename T, bool SOFTMAX>
__device__ __noinline__ int choose_exactly(const RouteArgs &a, const T *x, uint64_t *values, unsigned kept, int lane) {
    exact_values<T, SOFTMAX>(a, x, values, lane);
    uint64_t last = ~0ull;
    int last_e = -1, pick = -1;
    for (int p = 0; p < a.top_k; ++p) {
        uint64_t best = 0;
        int at = a.E;
        for (int e = lane; e < a.E; e += 32) {
            if (a.groups > 1 && !(kept >> a.by_size(e) & 1)) continue;
            const uint64_t v = values[e];
            if (v > best && before(last, last_e, v, e)) {
                best = v;
                at = e;
            }
        }
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) {
            const uint64_t v = __shfl_xor_sync(kAll, best, off);
            const int e = __shfl_xor_sync(kAll, at, off);
            if (before(v, e, best, at)) {
                best = v;
                at = e;
            }
        }
        if (best == 0) break;
        if (lane == p) pick = at;
        last = best;
        last_e = at;
    }
    return pick;
}

// V experts a lane.  (The arguments stay in constant memory although the functions above take their address: from
// a copy on the stack the picks of a few tokens took half as long again.)
template <typename T, int V, bool SOFTMAX>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ uint64_t values[];  // [kWarps][E], of rows that need them
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const T *row = static_cast<const T *>(a.logits) + t * a.stride;
    float x[V];
    bool bad = false;
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = j * 32 + lane < a.E ? to_f32(row[j * 32 + lane]) : -CUDART_INF_F;
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bias[j] = a.bias && j * 32 + lane < a.E ? a.bias[j * 32 + lane] : 0.0f;
        bad |= x[j] != x[j] || bias[j] != bias[j] || (SOFTMAX && x[j] == CUDART_INF_F);
    }
    if (__any_sync(kAll, bad)) {
        if (lane < a.top_k) {
            a.ids[t * a.top_k + lane] = -1;
            a.weights[t * a.top_k + lane] = CUDART_NAN_F;
        }
        return;
    }
    float top = 0.0f, total = 1.0f;
    if (SOFTMAX) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, ordered(x[j]));
        top = unordered(__reduce_max_sync(kAll, m));
        if (top == -CUDART_INF_F) top = 0.0f;  // all are masked
        float e[V];
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = expf(x[j] - top);
#pragma unroll
        for (int w = V / 2; w >= 1; w /= 2)
#pragma unroll
            for (int j = 0; j < w; ++j) e[j] += e[j + w];
        total = warp_sum(e[0]);
    }
    const bool by_sum = a.groups > 1 && a.group_top > 1;
    const float part_of = 1.0f / total;
    // keys: what experts are chosen by; `part`: what groups are
    uint32_t key[V], part[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float score = 0.0f;
        if (a.bias || by_sum) score = SOFTMAX ? __expf(x[j] - top) * part_of : near_sigmoid(x[j]);
        const float value = a.bias ? score + bias[j] : x[j];
        key[j] = x[j] > -CUDART_INF_F && value > -CUDART_INF_F ? ordered(value) : 0u;
        part[j] = key[j] == 0 ? 0u : by_sum && !a.bias ? ordered(score) : key[j];
    }
    unsigned kept = kAll;
    if (a.groups > 1) {
        float mine = -CUDART_INF_F;  // lane g: what group g counts
        float room = 0.0f;           // how far any of them may be off
        // What a group of largest values m1 and m2 (0: none) counts, and how far that may be off.  A sum of two
        // finite values may leave fp32's range: kept within it, a group that has experts is never taken for one
        // without (-infinity), and sums past one end are equal here, for fp64 to tell apart.
        const auto counts = [&](uint32_t m1, uint32_t m2, float &off) {
            float v = m1 ? unordered(m1) : -CUDART_INF_F;
            off = m1 ? slack<SOFTMAX>(v) : 0.0f;
            if (by_sum && m2) {
                off += slack<SOFTMAX>(unordered(m2));
                v = fminf(fmaxf(v + unordered(m2), -CUDART_MAX_NORMAL_F), CUDART_MAX_NORMAL_F);
            }
            return v;
        };
        // group g's largest values, from each lane's two largest
        const auto count = [&](int g, uint32_t b1, uint32_t b2) {
            const uint32_t m1 = __reduce_max_sync(kAll, b1);
            uint32_t m2 = 0;
            if (by_sum) {
                const int owner = __ffs(__ballot_sync(kAll, b1 == m1)) - 1;
                m2 = __reduce_max_sync(kAll, lane == owner ? b2 : b1);
            }
            float off;
            const float v = counts(m1, m2, off);
            room = fmaxf(room, off);
            if (lane == g) mine = v;
        };
        bool counted = false;
        if constexpr (V >= 8) {
            // The lanes' values fall into eight slots of whole groups or whole parts of them: all slots are
            // reduced at once, half of them handed to the other half of the lanes at each step (16384 rows of
            // 256 experts in 8 groups: 47.5 us with two redux a group, 44 like this).
            if (a.E == V * 32 && a.groups <= 8 && (a.groups & (a.groups - 1)) == 0) {
                counted = true;
                uint32_t b1[8], b2[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    b1[g] = b2[g] = 0;
#pragma unroll
                    for (int j = g * (V / 8); j < (g + 1) * (V / 8); ++j) {
                        b2[g] = max(b2[g], min(b1[g], part[j]));
                        b1[g] = max(b1[g], part[j]);
                    }
                }
                const auto merge = [&](uint32_t &u1, uint32_t &u2, uint32_t o1, uint32_t o2) {
                    u2 = max(min(u1, o1), max(u2, o2));
                    u1 = max(u1, o1);
                };
#pragma unroll
                for (int half = 4; half >= 1; half /= 2) {
                    const bool upper = lane & (4 * half);
#pragma unroll
                    for (int g = 0; g < half; ++g) {
                        const uint32_t o1 = __shfl_xor_sync(kAll, upper ? b1[g] : b1[g + half], 4 * half);
                        const uint32_t o2 = __shfl_xor_sync(kAll, upper ? b2[g] : b2[g + half], 4 * half);
                        b1[g] = upper ? b1[g + half] : b1[g];
                        b2[g] = upper ? b2[g + half] : b2[g];
                        merge(b1[g], b2[g], o1, o2);
                    }
                }
                // lanes 4 s ... have slot s
                merge(b1[0], b2[0], __shfl_xor_sync(kAll, b1[0], 2), __shfl_xor_sync(kAll, b2[0], 2));
                merge(b1[0], b2[0], __shfl_xor_sync(kAll, b1[0], 1), __shfl_xor_sync(kAll, b2[0], 1));
                int shift = 2;
                for (int n = 8; n > a.groups; n /= 2, ++shift)
                    merge(b1[0], b2[0], __shfl_xor_sync(kAll, b1[0], 1 << shift), __shfl_xor_sync(kAll, b2[0], 1 << shift));
                float off;
                float v = counts(b1[0], b2[0], off);
                room = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(off)));
                v = __shfl_sync(kAll, v, (lane << shift) & 31);
                if (lane < a.groups) mine = v;
            }
        }
        if (!counted) {
            for (int g = 0; g < a.groups; ++g) {
                const int from = g * a.group_size, to = from + a.group_size;
                uint32_t b1 = 0, b2 = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int e = j * 32 + lane;
                    const uint32_t k = e >= from && e < to ? part[j] : 0u;
                    b2 = max(b2, min(b1, k));
                    b1 = max(b1, k);
                }
                count(g, b1, b2);
            }
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const float o = __shfl_sync(kAll, mine, g);
            rank += before(o, g, mine, lane);
        }
        kept = __ballot_sync(kAll, lane < a.groups && rank < a.keep && mine > -CUDART_INF_F);
        if (a.keep < a.groups && (a.bias || by_sum)) {
            // Are the last group that is kept and the first that is not far enough apart?
            const unsigned in = __ballot_sync(kAll, lane < a.groups && rank == a.keep - 1);
            const unsigned out = __ballot_sync(kAll, lane < a.groups && rank == a.keep);
            const float u = __shfl_sync(kAll, mine, __ffs(in) - 1), w = __shfl_sync(kAll, mine, __ffs(out) - 1);
            if (w > -CUDART_INF_F && !(u - w > 2.0f * room))
                kept = keep_exactly<T, SOFTMAX>(a, row, values + (threadIdx.x >> 5) * a.E, lane);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int e = j * 32 + lane;
            if (e < a.E && !(kept >> a.by_size(e) & 1)) key[j] = 0;
        }
    }
    int pick = -1;
    bool unsure = false;
    {
        int n = 0;           // picks so far
        bool near = false;   // are two neighbours too near to tell apart?
        float last = 0.0f;
        while (true) {
            uint32_t best = 0, at = ~0u;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (key[j] > best) {
                    best = key[j];
                    at = j * 32 + lane;
                }
            const uint32_t m = __reduce_max_sync(kAll, best);
            if (m == 0) break;
            if (a.bias) {
                const float v = unordered(m);
                const bool apart = last - v > slack<SOFTMAX>(last);
                if (n >= a.top_k && apart) break;
                near |= n > 0 && !apart;
                last = v;
            }
            if (n == 32) {
                unsure = true;  // the run goes on past the lanes
                break;
            }
            const uint32_t e = __reduce_min_sync(kAll, best == m ? at : ~0u);
            if (lane == n) pick = e;
            ++n;
            if (n >= a.top_k && !a.bias) break;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if ((uint32_t)(j * 32 + lane) == e) key[j] = 0;
        }
        if (near && !unsure) {
            double denominator = 1.0;
            if (SOFTMAX) {
                denominator = 0.0;
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (x[j] > -CUDART_INF_F) denominator += exp((double)x[j] - (double)top);
                denominator = warp_sum(denominator);
            }
            uint64_t v = 0;
            if (lane < n) {
                const double l = to_f32(row[pick]);
                v = ordered((SOFTMAX ? exp(l - (double)top) / denominator : sigmoid(l)) + (double)a.bias[pick]);
            }
            int rank = 0;
            for (int o = 0; o < n; ++o) {
                const uint64_t w = __shfl_sync(kAll, v, o);
                const int e = __shfl_sync(kAll, pick, o);
                rank += before(w, e, v, pick);
            }
            int mine = -1;
            for (int o = 0; o < n; ++o) {
                const int r = __shfl_sync(kAll, rank, o), e = __shfl_sync(kAll, pick, o);
                if (r == lane) mine = e;
            }
            pick = mine;
        }
    }
    if (unsure) pick = choose_exactly<T, SOFTMAX>(a, row, values + (threadIdx.x >> 5) * a.E, kept, lane);
    if (lane >= a.top_k) pick = -1;
    // Scores of the picks.  Their shares of one another are formed from the logits, so that they hold
    // where the scores themselves underflow.
    const float l = pick >= 0 ? to_f32(row[pick]) : -CUDART_INF_F;
    float w = 0.0f;
    if (a.renormalise) {
        float most = l;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
        if (!SOFTMAX) most = fminf(most, 0.0f);
        if (pick >= 0) w = SOFTMAX ? exp_of_difference(l, most) : exp_of_difference(fminf(l, 0.0f), most) / (1.0f + expf(-fabsf(l)));
        const float sum = warp_sum(w);
        w = sum > 0.0f ? w / sum : 0.0f;
    } else if (pick >= 0) {
        w = SOFTMAX ? exp_of_difference(l, top) / total : sigmoid(l);
    }
    if (lane < a.top_k) {
        a.ids[t * a.top_k + lane] = pick;
        a.weights[t * a.top_k + lane] = w * a.scale;
    }
}

template <typename T, bool SOFTMAX>
cudaError_t launch_route(const RouteArgs &a, cudaStream_t stream) {
    void (*const kinds[])(RouteArgs) = {route_kernel<T, 1, SOFTMAX>, route_kernel<T, 2, SOFTMAX>,
                                        route_kernel<T, 4, SOFTMAX>, route_kernel<T, 8, SOFTMAX>,
                                        route_kernel<T, 16, SOFTMAX>, route_kernel<T, 32, SOFTMAX>};
    int k = 0;
    while (32 << k < a.E) ++k;
    const int64_t ctas = (a.T + kWarps - 1) / kWarps;
    return launch(kinds[k], dim3((unsigned)ctas), dim3(kWarps * 32), (size_t)kWarps * a.E * 8, stream, true, a);
}

template <typename T>
cudaError_t launch_scoring(const RouteArgs &a, int scoring, cudaStream_t s) {
    return scoring == RFP2_SOFTMAX ? launch_route<T, true>(a, s) : launch_route<T, false>(a, s);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" rfp2_status rfp2_moe_route(const void *logits, int dtype, int64_t T, int64_t E, int64_t logits_stride,
                                      int scoring, const float *bias, int64_t groups, int64_t keep,
                                      int64_t group_top, int64_t top_k, int renormalise, float scale,
                                      int32_t *ids, float *weights, rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype);
    if (T < 0 || !size || (scoring != RFP2_SOFTMAX && scoring != RFP2_SIGMOID) || !isfinite(scale))
        return RFP2_EINVAL;
    if (E < 1 || E > 1024 || top_k < 1 || top_k > 32 || top_k > E || groups < 1 || groups > 32 || E % groups != 0 ||
        keep < 1 || keep > groups || group_top < 1 || group_top > 2 || T > (1ll << 31) - 1)
        return RFP2_ESHAPE;
    if (T == 0) return RFP2_OK;
    if (!logits || !ids || !weights) return RFP2_EINVAL;
    if (T > 1 && logits_stride < 0) return RFP2_ESHAPE;
    if (!aligned(logits, size) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return RFP2_EALIGN;
    const Rows in[] = {{logits, T, E * size, logits_stride * size}, {bias, 1, E * 4, E * 4}};
    const Rows to(ids, 1, T * top_k * 4, 0), other(weights, 1, T * top_k * 4, 0);
    if (to.meet(other) || to.meet(in[0]) || to.meet(in[1]) || other.meet(in[0]) || other.meet(in[1])) return RFP2_EINVAL;
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.stride = logits_stride;
    a.E = (int)E;
    a.top_k = (int)top_k;
    a.groups = (int)groups;
    a.keep = (int)keep;
    a.group_top = (int)group_top;
    a.group_size = (int)(E / groups);
    a.by_size = FastDiv((uint32_t)(E / groups));
    a.renormalise = renormalise;
    a.scale = scale;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_scoring<float>(a, scoring, s)
                     : dtype == RFP2_BF16 ? launch_scoring<__nv_bfloat16>(a, scoring, s)
                                          : launch_scoring<__half>(a, scoring, s));
}
