// Attention of the newest tokens of each sequence over the paged Q8 cache:
//   s_j = scale * sum_b dK[j, b] (sum over block b of q kq[j]),   softcap tanh(s / softcap)
//   out = sum_j p_j dV[j, b] vq[j] / sum_j p_j,  p_j = exp(s_j - max s),  lse = max s + ln sum_j p_j
// in one pass over the keys with the running maximum and sum of the softmax.
//
// One CTA per (sequence, query, head): warps take keys in turn, a lane holds
// one value of every block; the warps' states join in shared memory.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kWarps = 8;

struct AttnArgs {
    const void *q;
    int64_t qb, qt, qh;
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int32_t *table, *lens;
    int64_t pages, table_stride, page_size, capacity;
    int nq, Hq, heads;
    float scale, softcap;
    int64_t window;
    void *out;
    float *lse;
    int32_t *status;
};

template <typename T, int NB>
__global__ void __launch_bounds__(kWarps * 32) attn_simple_kernel(const AttnArgs a) {
    constexpr int D = 32 * NB;
    __shared__ float m_s[kWarps], l_s[kWarps], o_s[kWarps][D];
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.nq;
    const int64_t b = blockIdx.x / a.Hq / a.nq;
    const int hk = h / (a.Hq / a.heads);
    const int64_t len = a.lens[b];
    const bool bad_len = len < 0 || len > a.capacity;
    if (bad_len && threadIdx.x == 0) record_status(a.status, RFP2_EBADID);
    const int64_t end = bad_len ? 0 : len - a.nq + 1 + i;
    const int64_t begin = a.window > 0 ? max((int64_t)0, end - a.window) : 0;
    float q[NB], o[NB];
    const T *qp = static_cast<const T *>(a.q) + b * a.qb + i * a.qt + h * a.qh;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        q[n] = to_f32(qp[32 * n + lane]);
        o[n] = 0.0f;
    }
    float m = -CUDART_INF_F, l = bad_len ? CUDART_NAN_F : 0.0f;
    for (int64_t j = begin + warp; j < end; j += kWarps) {
        const int64_t page = a.table[b * a.table_stride + j / a.page_size];
        float s;
        int64_t row = -1;
        if (page < 0 || page >= a.pages) {
            if (lane == 0) record_status(a.status, RFP2_EBADID);
            s = CUDART_NAN_F;
        } else {
            row = (page * a.heads + hk) * a.page_size + j % a.page_size;
            float part = 0.0f;
#pragma unroll
            for (int n = 0; n < NB; ++n)
                part += a.k_scales[row * NB + n] * (float)a.k_codes[row * D + 32 * n + lane] * q[n];
#pragma unroll
            for (int off = 16; off; off >>= 1) part += __shfl_xor_sync(0xffffffffu, part, off);
            s = part * a.scale;
            if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap);
        }
        const float top = fmaxf(m, s);
        const float keep = top == -CUDART_INF_F ? 1.0f : expf(m - top);
        const float p = s == -CUDART_INF_F ? 0.0f : expf(s - top);
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const float v =
                row < 0 ? 0.0f : a.v_scales[row * NB + n] * (float)a.v_codes[row * D + 32 * n + lane];
            o[n] = o[n] * keep + p * v;
        }
    }
    if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) o_s[warp][32 * n + lane] = o[n];
    __syncthreads();
    float top = -CUDART_INF_F, total = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w]);
    for (int w = 0; w < kWarps; ++w)
        total += l_s[w] * (m_s[w] == -CUDART_INF_F ? 1.0f : expf(m_s[w] - top));
    const int64_t at = (b * a.nq + i) * a.Hq + h;
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float sum = 0.0f;
        for (int w = 0; w < kWarps; ++w)
            sum += o_s[w][d] * (m_s[w] == -CUDART_INF_F ? 1.0f : expf(m_s[w] - top));
        static_cast<T *>(a.out)[at * D + d] = from_f32<T>(total == 0.0f ? 0.0f : sum / total);
    }
    if (a.lse && threadIdx.x == 0) a.lse[at] = total == 0.0f ? -CUDART_INF_F : top + logf(total);
}

template <typename T>
cudaError_t launch_attn(const AttnArgs &a, int D, int64_t ctas, cudaStream_t s) {
    void (*k)(AttnArgs) = nullptr;
    switch (D / 32) {
        case 1: k = attn_simple_kernel<T, 1>; break;
        case 2: k = attn_simple_kernel<T, 2>; break;
        case 3: k = attn_simple_kernel<T, 3>; break;
        case 4: k = attn_simple_kernel<T, 4>; break;
        case 5: k = attn_simple_kernel<T, 5>; break;
        case 6: k = attn_simple_kernel<T, 6>; break;
        case 7: k = attn_simple_kernel<T, 7>; break;
        default: k = attn_simple_kernel<T, 8>; break;
    }
    return launch(k, dim3((unsigned)ctas), dim3(kWarps * 32), 0, s, true, a);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" size_t rfp2_attn_decode_workspace_bytes(int64_t B, int64_t nq, int64_t Hq,
                                                   int64_t heads, int64_t D) {
    if (B < 1 || nq < 1 || Hq < 1 || heads < 1 || Hq % heads != 0 || D < 32) return 0;
    return 256;
}

extern "C" rfp2_status rfp2_attn_decode(const void *q, int dtype, int64_t B, int64_t nq,
                                        int64_t Hq, int64_t D, int64_t q_batch_stride,
                                        int64_t q_token_stride, int64_t q_head_stride,
                                        const int8_t *k_codes, const float *k_scales,
                                        const int8_t *v_codes, const float *v_scales,
                                        int64_t pages, int64_t heads, int64_t page_size,
                                        const int32_t *table, int64_t table_width,
                                        int64_t table_stride, const int32_t *lens, float scale,
                                        int64_t window, float softcap, void *out, float *lse,
                                        void *workspace, size_t workspace_bytes,
                                        int32_t *dev_status, rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype);
    if (!size || window < 0 || !(softcap >= 0.0f)) return RFP2_EINVAL;
    if (B < 1 || nq < 1 || Hq < 1 || heads < 1 || Hq % heads != 0 || Hq > 65536 ||
        nq > 65536 / Hq || B > (1 << 20) || D < 32 || D > 256 || D % 32 != 0 || pages < 1 ||
        page_size < 1 || page_size >= (1ll << 32) / heads ||
        pages >= (1ll << 32) / (heads * page_size) || table_width < 1 ||
        table_stride < table_width || table_width > (1ll << 30) / page_size)
        return RFP2_ESHAPE;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !table || !lens || !out)
        return RFP2_EINVAL;
    if (!workspace || workspace_bytes < rfp2_attn_decode_workspace_bytes(B, nq, Hq, heads, D))
        return RFP2_EWORKSPACE;
    if (!aligned(q, size) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(k_codes, 16) || !aligned(k_scales, 16) ||
        !aligned(v_codes, 16) || !aligned(v_scales, 16) || !aligned(workspace, 256))
        return RFP2_EALIGN;
    AttnArgs a;
    a.q = q;
    a.qb = q_batch_stride;
    a.qt = q_token_stride;
    a.qh = q_head_stride;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.table = table;
    a.lens = lens;
    a.pages = pages;
    a.table_stride = table_stride;
    a.page_size = page_size;
    a.capacity = table_width * page_size;
    a.nq = (int)nq;
    a.Hq = (int)Hq;
    a.heads = (int)heads;
    a.scale = scale;
    a.softcap = softcap;
    a.window = window;
    a.out = out;
    a.lse = lse;
    a.status = dev_status;
    const int64_t ctas = B * nq * Hq;
    if (ctas > (1ll << 31) - 1) return RFP2_ESHAPE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_attn<float>(a, (int)D, ctas, s)
                     : dtype == RFP2_BF16 ? launch_attn<__nv_bfloat16>(a, (int)D, ctas, s)
                                          : launch_attn<__half>(a, (int)D, ctas, s));
}
