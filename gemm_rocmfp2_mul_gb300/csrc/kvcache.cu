// The paged key-value cache in Q8_1-style blocks: tokens quantised as they are
// written (the keys rotated first, where asked) and read back by slot.
//   scale = max|a| / 127 over 32 neighbouring values, code = round-half-away(a / scale)
//
// Bound by memory: a written value is 2 or 4 bytes in and 9/8 bytes out, a read
// one the reverse.  A CTA takes a few tokens.  Each thread first sends off the
// loads of its steps (eight neighbouring values of a head's row, four threads a
// block of 32); the place of each token in the cache and, for a rotation, each
// (token, pair)'s cos and sin are computed once into shared memory meanwhile.
//
// Measured (one GB300, back to back), 16384 tokens x 8 heads of 128 values, bf16:
// write 24.6 us, rotated 30.2 (105 MB; the instructions, 172 a warp of 8-value
// steps, set the pace), read 15.2 us, written and read in turn 48.8.  Eight fp32
// tokens: 2.2 and 2.2.  Codes by division took 47 us.  Writes at three CTAs of 80
// registers an SM against four of 64: 30.7 and 30.3 us, but 6.0 and 7.3 for 4999
// tokens of 5 x 96 f16, whose interleaved rotation spills at 64 (rows of 16 bits at
// any alignment spill 48 bytes at 80 too); reads at five against six: 19.0 and 19.2,
// 3.75 and 4.1.
#include <algorithm>

#include "activation.cuh"

namespace rfp2 {
namespace {

constexpr int kThreads = 256;
// Entries of a CTA's table, one of a token and one of each (token, pair): 32 KB.  A write's CTAs take as many tokens
// as fill the SMs once, where they fit there: a thread stays with its place and its loads follow one another.
// Against 36 tokens at most, 17500 tokens x 8 heads of 128, bf16: 30.9 -> 29.8 us, 40000: 65.2 -> 61.3, of 5 x 96 f16:
// 31.8 -> 28.6.
constexpr int kMaxTable = 4096;
// A read's, at most: its CTAs are short, and those that come late fill what others leave.  20, 32 and 64 tokens,
// 40000 x 8 x 128: 42.3 us, 42.3 and 46.4; 16384: 17.7, 17.0 and 17.0.
constexpr int kReadTokens = 32;

// A token's steps (a head's eight or, reading fp32, four values of key and of
// value) are dealt to neighbouring threads; a CTA holds `rows` tokens at a
// time, or a stretch of a token that has more steps than the CTA threads.  So a
// thread keeps its head and its place in the row, and goes from token to token.
struct Deal {
    int steps, rows, tokens;  // steps of a token; tokens at a time; tokens of a CTA
    FastDiv by_steps, by_chunks;
    RFP2_DEV bool mine(int chunks, int &row, int &h, int &c, int &step) const {
        row = rows > 1 ? by_steps(threadIdx.x) : 0;
        step = threadIdx.x - row * steps + blockIdx.y * kThreads;
        h = by_chunks(step);
        c = step - h * chunks;
        return row < rows && step < steps;
    }
};

// The tokens are dealt so that the CTAs fill the SMs, `resident` on each, a whole
// number of times: at most `most` tokens a CTA, and few tokens spread one by one.
Deal deal(int64_t T, int64_t heads, int64_t chunks, int resident, int64_t most) {
    Deal w;
    w.steps = (int)(heads * chunks);
    w.rows = std::max(1, kThreads / w.steps);
    const int64_t stretches = (w.steps + kThreads - 1) / kThreads;
    const int64_t at_once = std::max<int64_t>(1, resident * (int64_t)sm_count(current_device()) / stretches);
    const int64_t waves = (T + at_once * most - 1) / (at_once * most);
    int64_t tokens = (T + at_once * waves - 1) / (at_once * waves);
    if (tokens > w.rows) tokens = (tokens + w.rows - 1) / w.rows * w.rows;
    w.tokens = (int)std::max<int64_t>(1, tokens);
    w.rows = std::min(w.rows, w.tokens);
    w.by_steps = FastDiv((uint32_t)w.steps);
    w.by_chunks = FastDiv((uint32_t)chunks);
    return w;
}
dim3 grid_of(const Deal &w, int64_t T) {
    return dim3((unsigned)((T + w.tokens - 1) / w.tokens), (unsigned)((w.steps + kThreads - 1) / kThreads));
}

struct WriteArgs {
    const void *k, *v;
    int64_t T, kt, kh, vt, vh;
    const int64_t *slots;
    const int32_t *positions;
    const float *inv_freq;
    int8_t *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t pages, page_size;
    int heads, D, pairs, interleaved;
    Deal deal;
    FastDiv by_pairs;
    float factor;
    int32_t *status;
};

// Place in the codes (a 32nd of that in the scales) of a slot's head 0; the next
// head is page_size * D on.  -1: left out, -2: no such slot.
RFP2_DEV int64_t slot_place(int64_t slot, int64_t pages, int64_t page_size, int heads, int D) {
    if (slot == -1) return -1;
    if (slot < 0 || slot >= pages * page_size) return -2;
    const int64_t page = (slot | page_size) >> 32 ? slot / page_size
                                                  : (int64_t)((uint32_t)slot / (uint32_t)page_size);
    return (page * heads * page_size + (slot - page * page_size)) * D;
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

RFP2_DEV float max_abs(float a, float b, float c) {  // of |a|, |b|, |c|; a NaN stays
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// round-half-away(fl(x / d)) by the division, as a byte; 0 where the block is
// zero or not finite.  For scales so small that a reciprocal or a product of
// them leaves fp32's range.
__device__ __noinline__ uint32_t code_of_odd(float x, float d) {
    if (!(d > 0.0f && d <= 3.402823466e38f)) return 0u;
    return (uint32_t)(int)fminf(fmaxf(roundf(__fdiv_rn(x, d)), -127.0f), 127.0f) & 255u;
}

// round-half-away(fl(x / d)) for eight values and 2^-90 <= d < inf, as bytes of
// two words, without a division.
//
// 1/d to 2^-22 and a little more either way brackets x / d and its rounded
// quotient: where both products round to the same integer (adding 1.5 * 2^23
// rounds, and leaves the integer in the low bits), that is the result.  Else a
// half-integer H = n + 1/2 lies between, as often happens for 16-bit types, and
// fl(|x| / d) >= H exactly when |x| / d >= H - u/2, u being fp32's spacing just
// below H (at equality |x| would need 25 bits).  R = |x| - H d is a small
// multiple of d's last place, so the fused product gives it exactly, and
// (u/2) d is d times a power of two: 2^(k-24) for H in (2^k, 2^(k+1)), 2^-26 for
// H = 1/2, in both cases the power of two below H's predecessor times 2^-24.
RFP2_DEV uint2 codes_of(const float (&x)[8], float d) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23
    float by;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(d));
    const float more = by * (1.0f + 0x1p-20f), less = by * (1.0f - 0x1p-20f);
    uint32_t q[8], differ = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = __float_as_uint(fmaf(x[e], less, kMagic));
        differ |= q[e] ^ __float_as_uint(fmaf(x[e], more, kMagic));
    }
    if (differ) {
        const float scaled = d * 0x1p-24f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float far = fmaf(x[e], more, kMagic);
            if (q[e] == __float_as_uint(far)) continue;
            const float H = fabsf(__uint_as_float(q[e]) - kMagic) + 0.5f;
            const float below = __uint_as_float((__float_as_uint(H) - 1u) & 0x7F800000u);
            const bool up = fmaf(-H, d, fabsf(x[e])) > -below * scaled;
            q[e] = up ? __float_as_uint(far) : q[e];
        }
    }
    uint2 w;
    w.x = __byte_perm(__byte_perm(q[0], q[1], 0x0040), __byte_perm(q[2], q[3], 0x0040), 0x5410);
    w.y = __byte_perm(__byte_perm(q[4], q[5], 0x0040), __byte_perm(q[6], q[7], 0x0040), 0x5410);
    return w;
}

// Eight values of a block, in four neighbouring lanes, to the cache's codes;
// the block's scale at the place that goes with them.
RFP2_DEV void write_block(const float (&x)[8], int8_t *codes, float *scale, bool first) {
    float top = max_abs(max_abs(x[0], x[1], x[2]), max_abs(x[3], x[4], x[5]), max_abs(x[6], x[7], x[7]));
    const uint32_t lanes = 0xFu << (threadIdx.x & 28);
    top = max_abs(top, __shfl_xor_sync(lanes, top, 1), top);
    top = max_abs(top, __shfl_xor_sync(lanes, top, 2), top);
    // top / 127 rounded to nearest: the rounded product with 1/127, corrected by its exact remainder
    // (Markstein 1990; checked for every significand).  Away from the ends of fp32's range.
    constexpr float kOver127 = 1.0f / 127.0f;
    const float near_d = top * kOver127;
    float d = fmaf(fmaf(-near_d, 127.0f, top), kOver127, near_d);
    uint2 w = make_uint2(0u, 0u);
    if (d >= 0x1p-90f && d <= 3.402823466e38f) {
        w = codes_of(x, d);
    } else {
        d = __fdiv_rn(top, 127.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w.x |= code_of_odd(x[e], d) << (8 * e);
            w.y |= code_of_odd(x[4 + e], d) << (8 * e);
        }
    }
    *reinterpret_cast<uint2 *>(codes) = w;
    if (first) *scale = d;
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, 3) kv_write_kernel(const WriteArgs a) {
    constexpr int AHEAD = 4 / sizeof(T);
    extern __shared__ __align__(16) uint8_t smem[];
    float *table = reinterpret_cast<float *>(smem);                                       // [tokens][cos, sin][pairs]
    int64_t *place = reinterpret_cast<int64_t *>(smem + 8 * a.deal.tokens * a.pairs);      // [tokens]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.deal.tokens;
    const int nt = (int)min((int64_t)a.deal.tokens, a.T - t0);
    int row, h, c, step;
    const bool mine = a.deal.mine(a.D / 8, row, h, c, step);
    const T *k = static_cast<const T *>(a.k) + t0 * a.kt + h * a.kh + 8 * c;
    const T *v = static_cast<const T *>(a.v) + t0 * a.vt + h * a.vh + 8 * c;
    Eight<T, WIDE> x[AHEAD], y[AHEAD];
    const auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (mine && t + i * a.deal.rows < nt) {
                x[i].load(k + (t + i * a.deal.rows) * a.kt);
                y[i].load(v + (t + i * a.deal.rows) * a.vt);
            }
    };
    load(row);
    // four cosines a word; where eight neighbouring pairs go to a thread, in the order that it reads
    const bool words = a.interleaved ? a.pairs % 4 == 0 : a.pairs % 8 == 0;
    const bool halves = words && !a.interleaved;
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        place[i] = slot_place(a.slots[t0 + i], a.pages, a.page_size, a.heads, a.D);
        if (place[i] == -2) record_status(a.status, RFP2_EBADID);
    }
    if (a.pairs) {
        if (halves)
            rotary_table<8, kThreads>(table, a.positions + t0, a.inv_freq, nt, a.pairs, a.by_pairs, a.factor, a.factor);
        else
            rotary_table<1, kThreads>(table, a.positions + t0, a.inv_freq, nt, a.pairs, a.by_pairs, a.factor, a.factor);
    }
    __syncthreads();
    if (!mine) return;

    // the eight keys of this thread's place in token t's row, turned
    const auto turn = [&](int t, float (&u)[8]) {
        const float *cs = table + 2 * t * a.pairs;
        if (halves) {
            // the eight lie in one half; their partners, in the other, have just been read nearby
            const bool low = 8 * c < a.pairs;
            const int p = c - (low ? 0 : a.pairs >> 3);
            Eight<T, WIDE> z;
            z.load(k + t * a.kt + (low ? a.pairs : -a.pairs));
            const uint32_t sign = low ? 0x80000000u : 0u;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float *q = cs + (w * (a.pairs >> 3) + p) * 4;
                const float4 co = *reinterpret_cast<const float4 *>(q);
                const float4 si = *reinterpret_cast<const float4 *>(q + a.pairs);
                const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[4 * w + e] = u[4 * w + e] * cc[e] +
                                   __uint_as_float(__float_as_uint(ss[e]) ^ sign) * to_f32(z.v[4 * w + e]);
            }
        } else if (words) {
            const float4 co = *reinterpret_cast<const float4 *>(cs + 4 * c);
            const float4 si = *reinterpret_cast<const float4 *>(cs + a.pairs + 4 * c);
            const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = u[2 * e], q = u[2 * e + 1];
                u[2 * e] = p * cc[e] - q * ss[e];
                u[2 * e + 1] = q * cc[e] + p * ss[e];
            }
        } else {
            // pairs that lie anyhow: each value with its partner, from memory
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int j = 8 * c + e;
                if (j >= 2 * a.pairs) continue;
                const bool first = a.interleaved ? j % 2 == 0 : j < a.pairs;
                const int p = a.interleaved ? j / 2 : first ? j : j - a.pairs;
                const int away = a.interleaved ? (first ? 1 : -1) : (first ? a.pairs : -a.pairs);
                const float other = to_f32(k[t * a.kt + e + away]);
                u[e] = u[e] * cs[p] + (first ? -cs[a.pairs + p] : cs[a.pairs + p]) * other;
            }
        }
    };
    const int64_t own = (int64_t)h * a.page_size * a.D + 8 * c;
    for (int t = row; t < nt; t += AHEAD * a.deal.rows) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = t + i * a.deal.rows;
            if (at >= nt || place[at] < 0) continue;
            const int64_t to = place[at] + own;
            float u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = to_f32(x[i].v[e]);
            if (8 * c < 2 * a.pairs) turn(at, u);
            write_block(u, a.k_codes + to, a.k_scales + (to >> 5), (c & 3) == 0);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = to_f32(y[i].v[e]);
            write_block(u, a.v_codes + to, a.v_scales + (to >> 5), (c & 3) == 0);
        }
        load(t + AHEAD * a.deal.rows);
    }
}

struct ReadArgs {
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int64_t *slots;
    int64_t T, pages, page_size;
    void *k, *v;
    int heads, D;
    Deal deal;
    int32_t *status;
};

// E codes to a 16-byte word of outputs.
template <typename T, int E>
RFP2_DEV void read_word(const uint32_t (&w)[E / 4], float d, T *out) {
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        // the code's byte above 2^23 + 128, exact, less as much
        const uint32_t u = __byte_perm(w[e >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (e & 3));
        x[e] = (__uint_as_float(u) - 8388736.0f) * d;
    }
    store_values<T, E>(out, x);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 5) kv_read_kernel(const ReadArgs a) {
    constexpr int E = 16 / sizeof(T), AHEAD = 1;
    extern __shared__ int64_t place[];  // [tokens]
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t0 = (int64_t)blockIdx.x * a.deal.tokens;
    const int nt = (int)min((int64_t)a.deal.tokens, a.T - t0);
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        place[i] = slot_place(a.slots[t0 + i], a.pages, a.page_size, a.heads, a.D);
        if (place[i] == -2) record_status(a.status, RFP2_EBADID);
    }
    int row, h, c, step;
    const bool mine = a.deal.mine(a.D / E, row, h, c, step);
    __syncthreads();
    if (!mine) return;
    T *k = static_cast<T *>(a.k), *v = static_cast<T *>(a.v);
    const int64_t own = (int64_t)h * a.page_size * a.D + E * c;
    struct Batch {
        uint32_t k[AHEAD][E / 4], v[AHEAD][E / 4];
        float kd[AHEAD], vd[AHEAD];
    };
    const auto load = [&](int t, Batch &b) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = t + i * a.deal.rows;
            const int64_t base = at < nt ? place[at] : -1;
#pragma unroll
            for (int e = 0; e < E / 4; ++e) b.k[i][e] = b.v[i][e] = 0u;
            b.kd[i] = b.vd[i] = base == -1 ? 0.0f : CUDART_NAN_F;
            if (base >= 0) {
                const int64_t from = base + own;
                const uint32_t *ks = reinterpret_cast<const uint32_t *>(a.k_codes + from);
                const uint32_t *vs = reinterpret_cast<const uint32_t *>(a.v_codes + from);
                if constexpr (E == 8) {
                    const uint2 p = *reinterpret_cast<const uint2 *>(ks), q = *reinterpret_cast<const uint2 *>(vs);
                    b.k[i][0] = p.x, b.k[i][1] = p.y;
                    b.v[i][0] = q.x, b.v[i][1] = q.y;
                } else {
                    b.k[i][0] = *ks;
                    b.v[i][0] = *vs;
                }
                b.kd[i] = a.k_scales[from >> 5];
                b.vd[i] = a.v_scales[from >> 5];
            }
        }
    };
    const auto store = [&](int t, const Batch &b) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int at = t + i * a.deal.rows;
            if (at >= nt) continue;
            const int64_t to = ((t0 + at) * a.deal.steps + step) * E;
            if (k) read_word<T, E>(b.k[i], b.kd[i], k + to);
            if (v) read_word<T, E>(b.v[i], b.vd[i], v + to);
        }
    };
    Batch here, next;
    const int stride = AHEAD * a.deal.rows;
    load(row, here);
    for (int t = row; t < nt; t += 2 * stride) {
        load(t + stride, next);
        store(t, here);
        load(t + 2 * stride, here);
        store(t + stride, next);
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
    if (T < 0 || !size || (flags & ~RFP2_ROPE_INTERLEAVED)) return RFP2_EINVAL;
    if (T > (1ll << 31) - 1 || (positions && (R < 0 || R % 2 != 0 || R > D))) return RFP2_ESHAPE;
    const rfp2_status st =
        check_cache(k_codes, k_scales, v_codes, v_scales, pages, heads, page_size, D);
    if (st != RFP2_OK) return st;
    if (T == 0) return RFP2_OK;
    if (!k || !v || !slots || !positions != !inv_freq) return RFP2_EINVAL;
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
    a.by_pairs = FastDiv(std::max(1, a.pairs));
    a.deal = deal(T, heads, D / 8, 3, kMaxTable / (1 + a.pairs));
    a.interleaved = (flags & RFP2_ROPE_INTERLEAVED) != 0;
    a.factor = factor;
    a.status = dev_status;
    const int64_t V = 16 / size;
    const bool wide = aligned(k, 16) && aligned(v, 16) && a.kt % V == 0 && a.kh % V == 0 &&
                      a.vt % V == 0 && a.vh % V == 0;
    const dim3 grid = grid_of(a.deal, T);
    const size_t smem = (size_t)a.deal.tokens * (8 + 8 * (size_t)a.pairs);
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
    a.status = dev_status;
    a.deal = deal(T, heads, D * dtype_bytes(dtype) / 16, 5, kReadTokens);
    const dim3 grid = grid_of(a.deal, T);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = 8 * (size_t)a.deal.tokens;
    return from_cuda(
        dtype == RFP2_F32    ? launch(kv_read_kernel<float>, grid, dim3(kThreads), smem, s, true, a)
        : dtype == RFP2_BF16 ? launch(kv_read_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, s, true, a)
                             : launch(kv_read_kernel<__half>, grid, dim3(kThreads), smem, s, true, a));
}
