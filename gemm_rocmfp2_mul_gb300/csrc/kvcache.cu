// The paged key-value cache in Q8_1-style blocks: tokens quantised as they are
// written (the keys rotated first, where asked) and read back by slot.
//   scale = max|a| / 127 over 32 neighbouring values, code = round-half-away(a / scale)
//
// Bound by memory: a written value is 2 or 4 bytes in and 9/8 bytes out, a read
// one the reverse.  A CTA takes a few tokens.  Each thread first sends off the
// loads of its steps (eight neighbouring values of a head's row, four threads a
// block of 32); the place of each token in the cache and, for a rotation, each
// (token, pair)'s cos and sin are computed once into shared memory meanwhile.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // steps of a thread whose loads travel together

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
    FastDiv by_pairs, by_token, by_chunks;  // a token's pairs, steps (of keys or values), a row's steps
    float factor;
    int32_t *status;
};

// Row of the cache arrays (of D codes, D / 32 scales) at which a slot's head 0
// lies; the next head is page_size rows on.  -1: left out, -2: no such slot.
RFP2_DEV int64_t slot_row(int64_t slot, int64_t pages, int64_t page_size, int heads) {
    if (slot == -1) return -1;
    if (slot < 0 || slot >= pages * page_size) return -2;
    const int64_t page = (slot | page_size) >> 32 ? slot / page_size
                                                  : (int64_t)((uint32_t)slot / (uint32_t)page_size);
    return page * heads * page_size + (slot - page * page_size);
}

// Eight values as they lie in memory.  WIDE: rows of 16-byte words; else any
// alignment.
template <typename T, bool WIDE>
struct alignas(8 * sizeof(T)) Eight {
    T v[8];
    RFP2_DEV void load(const T *p) {
        if constexpr (WIDE) {
#pragma unroll
            for (int w = 0; w < (int)sizeof(T) / 2; ++w)
                reinterpret_cast<uint4 *>(v)[w] = reinterpret_cast<const uint4 *>(p)[w];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[e];
        }
    }
};

// Codes of eight values by their block's scale d, as two words.  z = a / d to
// within 2^-14 by an approximate reciprocal; where z is not within 2^-12 of a
// half-integer it rounds as the IEEE quotient does, else, and for scales so
// small that the reciprocal or z may leave fp32's range, the division decides.
RFP2_DEV uint2 codes_of(const float (&x)[8], float d) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer
    float by;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(d));
    uint32_t q[8];
    float off = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float z = x[e] * by, r = z + kMagic;
        off = fmaxf(off, fabsf(z - (r - kMagic)));
        q[e] = __float_as_uint(r);
    }
    if (off > 0.5f - 0x1p-12f || d < 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            q[e] = (uint32_t)(int)fminf(fmaxf(roundf(__fdiv_rn(x[e], d)), -127.0f), 127.0f);
    }
    uint2 w;
    w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    return w;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, 3) kv_write_kernel(const WriteArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    int64_t *row0 = reinterpret_cast<int64_t *>(smem);                // [tokens]
    float2 *table = reinterpret_cast<float2 *>(smem + 8 * a.tokens);  // [tokens][pairs]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)min((int64_t)a.tokens, a.T - t0);
    const int chunks = a.D / 8, per_token = a.heads * chunks;
    const int n = 2 * nt * per_token;  // a multiple of 8, so blocks' four lanes go together

    // step i: keys or values of token t, values 8c .. 8c + 7 of head h
    const auto place = [&](int i, int &t, int &is_v, int &h, int &c) {
        const int token2 = a.by_token(i), rest = i - token2 * per_token;
        t = token2 >> 1;
        is_v = token2 & 1;
        h = a.by_chunks(rest);
        c = rest - h * chunks;
    };
    const auto row_of = [&](int t, int is_v, int h) {
        return is_v ? static_cast<const T *>(a.v) + (t0 + t) * a.vt + h * a.vh
                    : static_cast<const T *>(a.k) + (t0 + t) * a.kt + h * a.kh;
    };
    const auto load = [&](int i, Eight<T, WIDE> &x) {
        if (i >= n) return;
        int t, is_v, h, c;
        place(i, t, is_v, h, c);
        x.load(row_of(t, is_v, h) + 8 * c);
    };
    const auto write = [&](int i, const Eight<T, WIDE> &raw) {
        if (i >= n) return;
        int t, is_v, h, c;
        place(i, t, is_v, h, c);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f32(raw.v[e]);
        if (!is_v && 8 * c < 2 * a.pairs) {
            const float2 *cs = table + t * a.pairs;
            const T *row = row_of(t, 0, h);
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
                // the eight lie in one half; their partners, in the other, have just been read nearby
                const bool low = 8 * c < a.pairs;
                Eight<T, WIDE> y;
                y.load(row + 8 * c + (low ? a.pairs : -a.pairs));
                const float2 *p = cs + 8 * c - (low ? 0 : a.pairs);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float w = to_f32(y.v[e]);
                    x[e] = x[e] * p[e].x + (low ? -w : w) * p[e].y;
                }
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
        // the maximum of |a| as bits: a NaN is above everything and stays
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        const uint32_t lanes = 0xFu << (threadIdx.x & 28);
        top = max(top, __shfl_xor_sync(lanes, top, 1));
        top = max(top, __shfl_xor_sync(lanes, top, 2));
        const int64_t base = row0[t];
        if (base < 0) return;
        const float d = __fdiv_rn(__uint_as_float(top), 127.0f);
        // a block that is zero, or not finite, has codes 0
        const uint2 w = top < 0x7F800000u && d != 0.0f ? codes_of(x, d) : make_uint2(0u, 0u);
        const int64_t row = base + (int64_t)h * a.page_size;
        *reinterpret_cast<uint2 *>((is_v ? a.v_codes : a.k_codes) + row * a.D + 8 * c) = w;
        if ((c & 3) == 0) (is_v ? a.v_scales : a.k_scales)[row * (a.D / 32) + (c >> 2)] = d;
    };

    Eight<T, WIDE> x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(threadIdx.x + k * kThreads, x[k]);
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        row0[i] = slot_row(a.slots[t0 + i], a.pages, a.page_size, a.heads);
        if (row0[i] == -2) record_status(a.status, RFP2_EBADID);
    }
    for (int i = threadIdx.x; i < nt * a.pairs; i += kThreads) {
        const int t = a.by_pairs(i), p = i - t * a.pairs;
        const float2 cs = rotary_cos_sin(a.positions[t0 + t], turn_fraction(a.inv_freq[p]));
        table[i] = make_float2(cs.x * a.factor, cs.y * a.factor);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kAhead * kThreads) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) write(i + k * kThreads, x[k]);
        if (i + kAhead * kThreads < n)
#pragma unroll
            for (int k = 0; k < kAhead; ++k) load(i + (kAhead + k) * kThreads, x[k]);
    }
}

struct ReadArgs {
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int64_t *slots;
    int64_t T, pages, page_size;
    void *k, *v;
    int heads, D, tokens;
    FastDiv by_token, by_chunks;
    int32_t *status;
};

// A step is a 16-byte word of outputs.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) kv_read_kernel(const ReadArgs a) {
    constexpr int E = 16 / sizeof(T);
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
    const int chunks = a.D / E, per_token = a.heads * chunks;
    const int n = 2 * nt * per_token;
    for (int i0 = threadIdx.x; i0 < n; i0 += kAhead * kThreads) {
        uint32_t w[kAhead][E / 4];
        float d[kAhead];
        T *out[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kThreads;
            out[k] = nullptr;
            if (i >= n) continue;
            const int token2 = a.by_token(i), rest = i - token2 * per_token, t = token2 >> 1;
            T *to = static_cast<T *>(token2 & 1 ? a.v : a.k);
            if (!to) continue;
            out[k] = to + ((t0 + t) * per_token + rest) * E;
            const int h = a.by_chunks(rest), c = rest - h * chunks;
            const int64_t base = row0[t];
#pragma unroll
            for (int e = 0; e < E / 4; ++e) w[k][e] = 0u;
            d[k] = base == -1 ? 0.0f : CUDART_NAN_F;
            if (base >= 0) {
                const int64_t row = base + (int64_t)h * a.page_size;
                const int8_t *from = (token2 & 1 ? a.v_codes : a.k_codes) + row * a.D + E * c;
                if constexpr (E == 8) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(from);
                    w[k][0] = u.x;
                    w[k][1] = u.y;
                } else {
                    w[k][0] = *reinterpret_cast<const uint32_t *>(from);
                }
                d[k] = (token2 & 1 ? a.v_scales : a.k_scales)[row * (a.D / 32) + c / (32 / E)];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (!out[k]) continue;
            float x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // the code's byte above 2^23 + 128, exact, less as much
                const uint32_t u = __byte_perm(w[k][e >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (e & 3));
                x[e] = (__uint_as_float(u) - 8388736.0f) * d[k];
            }
            store_values<T, E>(out[k], x);
        }
    }
}

// Tokens of a CTA: enough for kAhead steps a thread, but a few CTAs for every
// SM before that, and no more table than `most`.
int tokens_a_cta(int64_t T, int64_t steps_a_token, int64_t most) {
    const int64_t by_work = std::max<int64_t>(1, kAhead * kThreads / steps_a_token);
    const int64_t by_sms = std::max<int64_t>(1, T / (6 * (int64_t)sm_count(current_device())));
    return (int)std::max<int64_t>(1, std::min({by_work, by_sms, most}));
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
    const int64_t chunks = D / 8;
    a.tokens = tokens_a_cta(T, 2 * heads * chunks, 4096 / std::max(1, a.pairs));
    a.by_pairs = FastDiv(std::max(1, a.pairs));
    a.by_token = FastDiv((uint32_t)(heads * chunks));
    a.by_chunks = FastDiv((uint32_t)chunks);
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
    const int64_t chunks = D / (16 / dtype_bytes(dtype));
    a.tokens = tokens_a_cta(T, 2 * heads * chunks, 1024);
    a.by_token = FastDiv((uint32_t)(heads * chunks));
    a.by_chunks = FastDiv((uint32_t)chunks);
    a.status = dev_status;
    const dim3 grid((unsigned)((T + a.tokens - 1) / a.tokens));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = 8 * (size_t)a.tokens;
    return from_cuda(
        dtype == RFP2_F32    ? launch(kv_read_kernel<float>, grid, dim3(kThreads), smem, s, true, a)
        : dtype == RFP2_BF16 ? launch(kv_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, s, true, a)
                             : launch(kv_read_kernel<__half>, grid, dim3(kThreads), smem, s, true, a));
}
