// The sum of a token's experts: out[t] = sum_j weights[t, j] y[t, j] + residual[t], summed in fp32 in the
// order of the slots.  Bound by memory: each of a token's top_k rows is read once.  A thread takes a run of
// 16 bytes of the output's row and sends off the loads of up to eight slots before it adds.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // slots whose loads travel together

struct CombineArgs {
    const void *y, *residual;
    void *out;
    const float *weights;
    const int32_t *ids;
    int64_t T, yt, yj, rs, os;
    int top_k, M, runs;  // runs of V values of a row
};

template <typename Ty, typename To, int V>
__global__ void __launch_bounds__(kThreads) combine_kernel(const CombineArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t n = a.T * a.runs;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / a.runs;
        const int at = (int)(i - t * a.runs) * V;
        const Ty *y = static_cast<const Ty *>(a.y) + t * a.yt + at;
        float sum[V];
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        for (int j0 = 0; j0 < a.top_k; j0 += kAhead) {
            float v[kAhead][V], w[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const bool in = j0 + j < a.top_k;
                w[j] = in ? a.weights[t * a.top_k + j0 + j] : 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) v[j][e] = 0.0f;
                if (in && (!a.ids || a.ids[t * a.top_k + j0 + j] >= 0)) load_values(y + (j0 + j) * a.yj, v[j]);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
#pragma unroll
                for (int e = 0; e < V; ++e) sum[e] = fmaf(w[j], v[j][e], sum[e]);
        }
        if (a.residual) {
            float r[V];
            load_values(static_cast<const To *>(a.residual) + t * a.rs + at, r);
#pragma unroll
            for (int e = 0; e < V; ++e) sum[e] += r[e];
        }
        store_values(static_cast<To *>(a.out) + t * a.os + at, sum);
    }
}

template <typename Ty, typename To>
cudaError_t launch_combine(CombineArgs &a, cudaStream_t stream) {
    // V: 16 bytes of y's type, whatever the output's
    constexpr int W = 16 / sizeof(Ty) * sizeof(To) % 16 == 0 ? 16 / sizeof(Ty) : 16 / sizeof(To);
    const auto fits = [](const void *p, int64_t stride, size_t size) {
        return !p || (aligned(p, 16) && stride * (int64_t)size % 16 == 0);
    };
    const bool wide = a.M % W == 0 && fits(a.y, a.yt, sizeof(Ty)) && fits(a.y, a.yj, sizeof(Ty)) &&
                      fits(a.residual, a.rs, sizeof(To)) && fits(a.out, a.os, sizeof(To));
    a.runs = wide ? a.M / W : a.M;
    const int64_t ctas = (a.T * a.runs + kThreads - 1) / kThreads;
    const dim3 grid((unsigned)std::min<int64_t>(ctas, 1 << 30));
    return launch(wide ? combine_kernel<Ty, To, W> : combine_kernel<Ty, To, 1>, grid, dim3(kThreads), 0, stream, true, a);
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
    if (top_k < 1 || top_k > 1024 || T > (1ll << 31) - 1 || M > (1ll << 31) - 1 || y_token_stride < 0 ||
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
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_to<float>(a, out_dtype, s)
                     : dtype == RFP2_BF16 ? launch_to<__nv_bfloat16>(a, out_dtype, s)
                                          : launch_to<__half>(a, out_dtype, s));
}
