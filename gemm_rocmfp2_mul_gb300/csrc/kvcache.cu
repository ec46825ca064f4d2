// The paged key-value cache in Q8_1-style blocks: tokens quantised as they are
// written (the keys rotated first, where asked) and read back by slot.
//   scale = max|a| / 127 over 32 neighbouring values, code = round-half-away(a / scale)
//
// Bound by memory: a written value is 2 or 4 bytes in and 9/8 bytes out, a read
// one the reverse.  A CTA takes a few tokens: the place of each in the cache
// and, for a rotation, each (token, pair)'s cos and sin are computed once into
// shared memory; then every thread takes eight neighbouring values of a head's
// row (four threads a block of 32).
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;

struct WriteArgs {
    const void *k, *v;
    int64_t T, kt, kh, vt, vh;
    const int64_t *slots;
    const int32_t *positions;
    const float *inv_freq;
    int8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t pages, page_size;
    int heads, D, pairs, tokens, interleaved;
    float factor;
    int32_t *status;
};

// Row of the cache arrays (of D codes, D / 32 scales) at which a slot's head 0
// lies; the next head is page_size rows on.  -1: left out, -2: no such slot.
RFP2_DEV int64_t slot_row(int64_t slot, int64_t pages, int64_t page_size, int heads) {
    if (slot == -1) return -1;
    if (slot < 0 || slot >= pages * page_size) return -2;
    const int64_t page = slot / page_size;
    return page * heads * page_size + (slot - page * page_size);
}

// WIDE: rows whose eight values are 16-byte words; else any alignment.
template <typename T, bool WIDE>
RFP2_DEV void load8(const T *p, float (&v)[8]) {
    if constexpr (WIDE) {
        load_values<T, 8>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32(p[e]);
    }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const WriteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    int64_t *row0 = reinterpret_cast<int64_t *>(smem);               // [tokens]
    float2 *table = reinterpret_cast<float2 *>(smem + 8 * a.tokens);  // [tokens][pairs]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)min((int64_t)a.tokens, a.T - t0);
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        row0[i] = slot_row(a.slots[t0 + i], a.pages, a.page_size, a.heads);
        if (row0[i] == -2) record_status(a.status, RFP2_EBADID);
    }
    for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        float2 cs = rotary_cos_sin(a.positions[t0 + t], turn_fraction(a.inv_freq[p]));
        table[i] = make_float2(cs.x * a.factor, cs.y * a.factor);
    }
    __syncthreads();
    const int chunks = a.D / 8, per_token = a.heads * chunks;
    const int n = 2 * nt * per_token;  // a multiple of 8, so blocks' four lanes go together
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int token2 = i / per_token, rest = i - token2 * per_token;
        const int t = token2 >> 1, is_v = token2 & 1;
        const int h = rest / chunks, c = rest - h * chunks;
        const int64_t base = row0[t];
        float x[8];
        if (base >= 0) {
            const T *row = is_v ? static_cast<const T *>(a.v) + (t0 + t) * a.vt + h * a.vh
                                : static_cast<const T *>(a.k) + (t0 + t) * a.kt + h * a.kh;
            load8<T, WIDE>(row + 8 * c, x);
            if (!is_v && 8 * c < 2 * a.pairs) {
                const float2 *cs = table + t * a.pairs;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int p = 4 * c + e;
                        if (p < a.pairs) {
                            const float u = x[2 * e], w = x[2 * e + 1];
                            x[2 * e] = u * cs[p].x - w * cs[p].y;
                            x[2 * e + 1] = w * cs[p].x + u * cs[p].y;
                        }
                    }
                } else if (a.pairs % 8 == 0) {
                    // the chunk lies in one half; its partners in the other
                    const bool low = 8 * c < a.pairs;
                    float y[8];
                    load8<T, WIDE>(row + 8 * c + (low ? a.pairs : -a.pairs), y);
                    const int p = 8 * c - (low ? 0 : a.pairs);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = low ? x[e] * cs[p + e].x - y[e] * cs[p + e].y
                                   : x[e] * cs[p + e].x + y[e] * cs[p + e].y;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = 8 * c + e;
                        if (j < a.pairs)
                            x[e] = x[e] * cs[j].x - to_f32(row[j + a.pairs]) * cs[j].y;
                        else if (j < 2 * a.pairs)
                            x[e] = x[e] * cs[j - a.pairs].x + to_f32(row[j - a.pairs]) * cs[j - a.pairs].y;
                    }
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0.0f;
        }
        // the maximum of |a| as bits: a NaN is above everything and stays
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        const uint32_t lanes = 0xFu << (threadIdx.x & 28);
        top = max(top, __shfl_xor_sync(lanes, top, 1));
        top = max(top, __shfl_xor_sync(lanes, top, 2));
        if (base < 0) continue;
        const float d = __fdiv_rn(__uint_as_float(top), 127.0f);
        const bool finite = top < 0x7F800000u && d != 0.0f;
        uint32_t word[2] = {0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            int q = 0;
            if (finite) q = (int)fminf(fmaxf(roundf(__fdiv_rn(x[e], d)), -127.0f), 127.0f);
            word[e >> 2] |= (uint32_t)(q & 255) << (8 * (e & 3));
        }
        const int64_t row = base + (int64_t)h * a.page_size;
        *reinterpret_cast<uint2 *>((is_v ? a.v_codes : a.k_codes) + row * a.D + 8 * c) =
            make_uint2(word[0], word[1]);
        if ((c & 3) == 0) (is_v ? a.v_scales : a.k_scales)[row * (a.D / 32) + (c >> 2)] = d;
    }
}

struct ReadArgs {
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int64_t *slots;
    int64_t T, pages, page_size;
    void *k, *v;
    int heads, D, tokens;
    int32_t *status;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
    extern __shared__ int64_t row0[];  // [tokens]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)min((int64_t)a.tokens, a.T - t0);
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        row0[i] = slot_row(a.slots[t0 + i], a.pages, a.page_size, a.heads);
        if (row0[i] == -2) record_status(a.status, RFP2_EBADID);
    }
    __syncthreads();
    const int chunks = a.D / 8, per_token = a.heads * chunks;
    const int n = 2 * nt * per_token;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int token2 = i / per_token, rest = i - token2 * per_token;
        const int t = token2 >> 1, is_v = token2 & 1;
        T *out = static_cast<T *>(is_v ? a.v : a.k);
        if (!out) continue;
        const int h = rest / chunks, c = rest - h * chunks;
        float x[8];
        const int64_t base = row0[t];
        if (base >= 0) {
            const int64_t row = base + (int64_t)h * a.page_size;
            const uint2 w = *reinterpret_cast<const uint2 *>((is_v ? a.v_codes : a.k_codes) +
                                                             row * a.D + 8 * c);
            const float d = (is_v ? a.v_scales : a.k_scales)[row * (a.D / 32) + (c >> 2)];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t word = e < 4 ? w.x : w.y;
                x[e] = (float)(int)(int8_t)(word >> (8 * (e & 3))) * d;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = base == -1 ? 0.0f : CUDART_NAN_F;
        }
        store_values<T, 8>(out + (t0 + t) * per_token * 8 + rest * 8, x);
    }
}

rfp2_status check_cache(const void *k_codes, const void *k_scales, const void *v_codes,
                        const void *v_scales, int64_t pages, int64_t heads, int64_t page_size,
                        int64_t D) {
    if (pages < 1 || heads < 1 || page_size < 1 || D < 32 || D > 256 || D % 32 != 0 ||
        heads > 65536 || pages > (1ll << 40) / heads / page_size)
        return RFP2_ESHAPE;
    if (!k_codes || !k_scales || !v_codes || !v_scales) return RFP2_EINVAL;
    if (!aligned(k_codes, 16) || !aligned(k_scales, 16) || !aligned(v_codes, 16) ||
        !aligned(v_scales, 16))
        return RFP2_EALIGN;
    return RFP2_OK;
}

template <typename T>
cudaError_t launch_write(const WriteArgs &a, bool wide, dim3 grid, size_t smem, cudaStream_t s) {
    return launch(wide ? kv_write_kernel<T, true> : kv_write_kernel<T, false>, grid,
                  dim3(kThreads), smem, s, true, a);
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" rfp2_status rfp2_kv_write(const void *k, const void *v, int dtype, int64_t T,
                                     int64_t k_token_stride, int64_t k_head_stride,
                                     int64_t v_token_stride, int64_t v_head_stride,
                                     const int64_t *slots, const int32_t *positions,
                                     const float *inv_freq, int64_t R, float factor, int flags,
                                     int8_t *k_codes, float *k_scales, int8_t *v_codes,
                                     float *v_scales, int64_t pages, int64_t heads,
                                     int64_t page_size, int64_t D, int32_t *dev_status,
                                     rfp2_stream_t stream) {
    const int size = dtype_bytes(dtype);
    if (T < 0 || !size || (flags & ~RFP2_ROPE_INTERLEAVED) || !positions != !inv_freq)
        return RFP2_EINVAL;
    if (T > (1ll << 31) - 1 || (positions && (R < 0 || R % 2 != 0 || R > D))) return RFP2_ESHAPE;
    const rfp2_status st =
        check_cache(k_codes, k_scales, v_codes, v_scales, pages, heads, page_size, D);
    if (st != RFP2_OK) return st;
    if (T == 0) return RFP2_OK;
    if (!k || !v || !slots) return RFP2_EINVAL;
    if (!aligned(k, size) || !aligned(v, size) || !aligned(slots, 8) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4))
        return RFP2_EALIGN;
    WriteArgs a;
    a.k = k;
    a.v = v;
    a.T = T;
    a.kt = k_token_stride;
    a.kh = k_head_stride;
    a.vt = v_token_stride;
    a.vh = v_head_stride;
    a.slots = slots;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.pages = pages;
    a.page_size = page_size;
    a.heads = (int)heads;
    a.D = (int)D;
    a.pairs = positions ? (int)(R / 2) : 0;
    a.tokens = 1;
    a.interleaved = (flags & RFP2_ROPE_INTERLEAVED) != 0;
    a.factor = factor;
    a.status = dev_status;
    const int64_t V = 16 / size;
    const bool wide = aligned(k, 16) && aligned(v, 16) && a.kt % V == 0 && a.kh % V == 0 &&
                      a.vt % V == 0 && a.vh % V == 0;
    const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
    const size_t smem = (size_t)a.tokens * (8 + 8 * (size_t)a.pairs);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return from_cuda(dtype == RFP2_F32    ? launch_write<float>(a, wide, grid, smem, s)
                     : dtype == RFP2_BF16 ? launch_write<__nv_bfloat16>(a, wide, grid, smem, s)
                                          : launch_write<__half>(a, wide, grid, smem, s));
}

extern "C" rfp2_status rfp2_kv_read(const int8_t *k_codes, const float *k_scales,
                                    const int8_t *v_codes, const float *v_scales, int64_t pages,
                                    int64_t heads, int64_t page_size, int64_t D,
                                    const int64_t *slots, int64_t T, int dtype, void *k, void *v,
                                    int32_t *dev_status, rfp2_stream_t stream) {
    if (T < 0 || !dtype_bytes(dtype)) return RFP2_EINVAL;
    if (T > (1ll << 31) - 1) return RFP2_ESHAPE;
    const rfp2_status st =
        check_cache(k_codes, k_scales, v_codes, v_scales, pages, heads, page_size, D);
    if (st != RFP2_OK) return st;
    if (T == 0 || (!k && !v)) return RFP2_OK;
    if (!slots) return RFP2_EINVAL;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return RFP2_EALIGN;
    ReadArgs a;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.slots = slots;
    a.T = T;
    a.pages = pages;
    a.page_size = page_size;
    a.k = k;
    a.v = v;
    a.heads = (int)heads;
    a.D = (int)D;
    a.tokens = 1;
    a.status = dev_status;
    const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = 8 * (size_t)a.tokens;
    return from_cuda(
        dtype == RFP2_F32    ? launch(kv_read_kernel<float>, grid, dim3(kThreads), smem, s, true, a)
        : dtype == RFP2_BF16 ? launch(kv_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, s, true, a)
                             : launch(kv_read_kernel<__half>, grid, dim3(kThreads), smem, s, true, a));
}
