// The sum of a token's experts: out[t] = sum_j weights[t, j] y[t, j] + residual[t], summed in fp32 in the
// order of the slots.  Bound by memory: each of a token's top_k rows is read once.
//
// A thread has a run of 16 bytes or more of a token's row (or four single values, a CTA's width apart, where
// rows have no such alignment) and sends off the loads of up to eight slots before it adds any; they
// stay as they were loaded until then, which is half the registers of fp32 values.
//
// Measured (one GB300, GPU time a call): 16384 x 8 x 2048 bf16 with a residual 128 us, 5.2 TB/s (173 us with a CTA a
// token, which waits for its slots before it can ask for rows; 317 with fp32 values in registers); 4999 x 3 x
// 1001 f16 18.5 us; 4 x 8 x 2048 1.8 us.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
constexpr int kResident = 4;  // CTAs of an SM

struct CombineArgs {
    const void *y, *residual;
    void *out;
    const float *weights;
    const int32_t *ids;
    int64_t T, yt, yj, rs, os;
    int top_k, M, runs;   // runs of V values of a row
    int lanes, tokens;    // threads of a token, tokens of a CTA
    int eights;           // weights and ids of eight slots are aligned words
    FastDiv by_lanes;
};

// Weights of up to N slots, and which of them are read.
template <int N>
struct Slots {
    float w[N];
    int id[N];
    RFP2_DEV void load(const CombineArgs &a, int64_t t, int j0) {
        const float *weights = a.weights + t * a.top_k + j0;
        const int32_t *ids = a.ids ? a.ids + t * a.top_k + j0 : nullptr;
        if (N == 8 && a.eights) {
            const float4 w0 = reinterpret_cast<const float4 *>(weights)[0], w1 = reinterpret_cast<const float4 *>(weights)[1];
            const float ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            int4 i0 = make_int4(0, 0, 0, 0), i1 = i0;
            if (ids) i0 = reinterpret_cast<const int4 *>(ids)[0], i1 = reinterpret_cast<const int4 *>(ids)[1];
            const int is[8] = {i0.x, i0.y, i0.z, i0.w, i1.x, i1.y, i1.z, i1.w};
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = ws[j & 7], id[j] = is[j & 7];
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool in = j0 + j < a.top_k;
                w[j] = in ? weights[j] : 0.0f;
                id[j] = !in ? -1 : ids ? ids[j] : 0;
            }
        }
    }
};

// C runs a thread, a.lanes apart, of one token after another: the next one's slots are fetched while this one's
// rows are on their way.
template <typename Ty, typename To, int V, int C>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    constexpr int kAhead = 8 / C;  // slots whose loads travel together
    pdl_wait();
    pdl_launch_dependents();
    const int tt = (int)a.by_lanes(threadIdx.x);
    int64_t t = (int64_t)blockIdx.x * a.tokens + tt;
    if (tt >= a.tokens || t >= a.T) return;
    const int r0 = blockIdx.y * a.lanes * C + (threadIdx.x - tt * a.lanes);
    const int64_t step = (int64_t)gridDim.x * a.tokens;
    Slots<kAhead> slots;
    slots.load(a, t, 0);
    for (; t < a.T; t += step) {
        const Ty *y = static_cast<const Ty *>(a.y) + t * a.yt;
        Held<To, V> rest[C];
        float sum[C][V];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (a.residual && r0 + c * a.lanes < a.runs)
                rest[c].load(static_cast<const To *>(a.residual) + t * a.rs + (int64_t)(r0 + c * a.lanes) * V);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[c][e] = 0.0f;
        }
        for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
            Held<Ty, V> v[kAhead][C];
            const Slots<kAhead> now = slots;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (now.id[j] >= 0 && r0 + c * a.lanes < a.runs)
                        v[j][c].load(y + (j0 + j) * a.yj + (int64_t)(r0 + c * a.lanes) * V);
            if (j0 + kAhead < a.top_k)
                slots.load(a, t, j0 + kAhead);
            else if (t + step < a.T)
                slots.load(a, t + step, 0);
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        sum[c][e] = fmaf(now.w[j], now.id[j] >= 0 ? to_f32(v[j][c].v[e]) : 0.0f, sum[c][e]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (r0 + c * a.lanes >= a.runs) continue;
            if (a.residual)
#pragma unroll
                for (int e = 0; e < V; ++e) sum[c][e] += to_f32(rest[c].v[e]);
            store_values(static_cast<To *>(a.out) + t * a.os + (int64_t)(r0 + c * a.lanes) * V, sum[c]);
        }
    }
}

template <typename Ty, typename To>
cudaError_t launch_combine(CombineArgs &a, cudaStream_t stream) {
    // 16 bytes of y or of out, whichever has fewer values to them is two words of the other
    constexpr int W = 16 / (sizeof(Ty) < sizeof(To) ? sizeof(Ty) : sizeof(To));
    const auto fits = [](const void *p, int64_t stride, size_t size) {
        return !p || (aligned(p, 16) && stride * (int64_t)size % 16 == 0);
    };
    const bool wide = a.M % W == 0 && fits(a.y, a.yt, sizeof(Ty)) && fits(a.y, a.yj, sizeof(Ty)) &&
                      fits(a.residual, a.rs, sizeof(To)) && fits(a.out, a.os, sizeof(To));
    constexpr int C = 4;  // single values a thread
    a.runs = wide ? a.M / W : a.M;
    const int each = wide ? 1 : C;
    a.lanes = std::min(kThreads, (a.runs + each - 1) / each);
    a.tokens = kThreads / a.lanes;
    a.by_lanes = FastDiv((uint32_t)a.lanes);
    const int64_t ctas = (a.T + a.tokens - 1) / a.tokens, parts = (a.runs + (int64_t)a.lanes * each - 1) / ((int64_t)a.lanes * each);
    // as many CTAs as the SMs hold, so that most tokens have their slots fetched beforehand
    const int64_t held = std::max<int64_t>(1, (int64_t)kResident * sm_count(current_device()) / parts);
    const dim3 grid((unsigned)std::min(ctas, held), (unsigned)parts);
    return launch(wide ? combine_kernel<Ty, To, W, 1> : combine_kernel<Ty, To, 1, C>, grid, dim3(kThreads), 0, stream, true, a);
}

template <typename Ty>
cudaError_t launch_to(CombineArgs &a, int out_dtype, cudaStream_t s) {
    return out_dtype == RFP2_F32    ? launch_combine<Ty, float>(a, s)
           : out_dtype == RFP2_BF16 ? launch_combine<Ty, __nv_bfloat16>(a, s)
                                    : launch_combine<Ty, __half>(a, s);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" rfp2_status rfp2_moe_combine(const void *y, int dtype, int64_t T, int64_t top_k, int64_t M,
                                        int64_t y_token_stride, int64_t y_slot_stride, const float *weights,
                                        const int32_t *ids, const void *residual, int64_t residual_stride,
                                        void *out, int out_dtype, int64_t out_stride, rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype), osize = dtype_bytes(out_dtype);
    if (T < 0 || M < 0 || !size || !osize) return RFP2_EINVAL;
    if (top_k < 1 || top_k > 1024 || T > (1ll << 31) - 1 || M > 1 << 24 || y_token_stride < 0 ||
        y_slot_stride < 0)
        return RFP2_ESHAPE;
    if (T == 0 || M == 0) return RFP2_OK;
    if (!y || !weights || !out) return RFP2_EINVAL;
    if (T > 1 && (out_stride < M || (residual && residual_stride < 0))) return RFP2_ESHAPE;
    if (!aligned(y, size) || !aligned(weights, 4) || !aligned(ids, 4) || !aligned(residual, osize) ||
        !aligned(out, osize))
        return RFP2_EALIGN;
    const Rows to(out, T, M * osize, out_stride * osize), rest(residual, T, M * osize, residual_stride * osize);
    const Rows w(weights, 1, T * top_k * 4, 0), slots(ids, 1, T * top_k * 4, 0);
    bool meet = (to.meet(rest) && !to.same(rest)) || to.meet(w) || to.meet(slots);
    for (int64_t j = 0; j < top_k; ++j)
        meet |= to.meet(Rows(static_cast<const uint8_t *>(y) + j * y_slot_stride * size, T, M * size, y_token_stride * size));
    if (meet) return RFP2_EINVAL;
    CombineArgs a;
    a.y = y;
    a.residual = residual;
    a.out = out;
    a.weights = weights;
    a.ids = ids;
    a.T = T;
    a.yt = y_token_stride;
    a.yj = y_slot_stride;
    a.rs = residual_stride;
    a.os = out_stride;
    a.top_k = (int)top_k;
    a.M = (int)M;
    a.eights = top_k % 8 == 0 && aligned(weights, 16) && aligned(ids, 16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_to<float>(a, out_dtype, s)
                     : dtype == RFP2_BF16 ? launch_to<__nv_bfloat16>(a, out_dtype, s)
                                          : launch_to<__half>(a, out_dtype, s));
}
