// Decode attention over the paged Q8 cache: the kernel and its arguments.  The
// translation units attn_*.cu instantiate it by head size.
//
//   s_j = scale * sum_b dK[j, b] (sum over block b of q kq[j]),   softcap tanh(s / softcap)
//   out = sum_j p_j dV[j, b] vq[j] / sum_j p_j,  p_j = exp(s_j - max s),  lse = max s + ln sum_j p_j
//
// Bound by memory: each key of a head is 2 (D + D/8) bytes, read once for all
// its query heads and tokens ("columns").  Work is cut in tiles of 16 keys; the
// tiles of all (sequence, key head, column tile) units lie on one line that the
// CTAs share out evenly whatever the lengths are, and tile x of a CTA goes to
// warp x % 8.  Each warp streams its tiles through its own ring in shared
// memory (cp.async) and keeps its own softmax state; the warps join at the end
// of a unit's stretch, and a unit that several CTAs share is joined by the last
// of them to finish, always in the order of the keys.
//
// Products run on f16 matrix instructions (16 keys x 8 columns x 16 values):
// codes are exact in f16, q goes in scaled by a power of two (one f16 piece is
// exact for 16-bit q; two pieces leave 2^-22 of fp32 q).  The scores' block sums
// are scaled by dK in fp32.  p dV goes in as one f16 piece for 16-bit outputs
// and two for fp32.  Its range: the softmax's reference r is kept near
// max(s + log2 dV) instead of max s, so p dV stays below 2^15 whatever the
// scales of the values are, and what is lost lies 2^-33 below the largest.
#pragma once

#include <atomic>

#include "activation.cuh"

namespace rfp2 {

constexpr int kAttnWarps = 8;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr int kAttnTile = 16;         // keys
constexpr int kAttnMaxBatch = 1024;   // sequences of one launch
constexpr int kAttnCounterBytes = 4096;

struct AttnArgs {
    const void *q;
    int64_t qb, qt, qh;
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int32_t *table, *lens;
    int64_t pages, table_stride, capacity;
    int B, nq, Hq, heads, group, columns, column_tiles;
    int page_size, page_shift;  // shift: log2 of page_size, or -1
    int dtype, q_words;         // q_words: q can be read as 16-byte words
    float scale, softcap;
    int64_t window;
    void *out;
    float *lse;
    int *counters;
    float *partials;
    int32_t *status;
};

// One piece of the row layout: strides (bytes) of a tile's rows in shared
// memory, padded so that the fragment reads meet no bank twice.  K is read 8
// bytes a lane, four keys a half-warp: 32-byte steps between keys need an odd
// number of them a row.  V is read 4 bytes a lane, keys two apart: an odd number
// of 16-byte steps.
template <int NB>
struct AttnLayout {
    static constexpr int D = 32 * NB;
    static constexpr int k_stride = NB % 2 ? D : D + 32;
    static constexpr int v_stride = D + 16;
    static constexpr int k_bytes = kAttnTile * k_stride, v_bytes = kAttnTile * v_stride;
    static constexpr int scale_bytes = kAttnTile * NB * 4;
    static constexpr int stage_bytes = k_bytes + v_bytes + 2 * scale_bytes;
};

// Shared memory: rings, then the join buffer, the warps' references and sums,
// and the sequences' tile prefix.
template <int NB, int NT>
struct AttnShared {
    static constexpr int chunk = NB >= 2 ? 64 : 32;  // values joined at a time
    static constexpr int row = chunk + 4;            // floats, padded against bank conflicts
    static constexpr int join_bytes = kAttnWarps * 8 * NT * row * 4;
    static constexpr int state_bytes = 2 * kAttnWarps * 8 * NT * 4;
    static constexpr int other = join_bytes + state_bytes + 64;
    static constexpr int stages_for(int budget) {
        const int s = (budget - other - (kAttnMaxBatch + 1) * 12) /
                      (kAttnWarps * AttnLayout<NB>::stage_bytes);
        return s > 8 ? 8 : s;
    }
};

template <int NB, int NT>
constexpr int attn_ctas_per_sm() { return NB * NT <= 2 ? 2 : 1; }
template <int NB, int NT>
constexpr int attn_stages() {
    return AttnShared<NB, NT>::stages_for((attn_ctas_per_sm<NB, NT>() == 2 ? 113 : 227) * 1024);
}
template <int NB, int NT>
int attn_smem(int B) {
    return kAttnWarps * attn_stages<NB, NT>() * AttnLayout<NB>::stage_bytes +
           AttnShared<NB, NT>::other + (B + 1) * 8 + B * 4;
}

RFP2_DEV void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
template <int N>
RFP2_DEV void cp_async_small(uint32_t dst, const void *src, uint32_t bytes) {
    if constexpr (N == 16)
        cp_async16(dst, src, bytes);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N),
                     "r"(bytes)
                     : "memory");
}
RFP2_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
RFP2_DEV void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// D[16 x 8] += A[16 x 16] B[16 x 8], f16 in, fp32 sums.
RFP2_DEV void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
RFP2_DEV uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Two f16 of 1024 + u (u a byte) less 1152: the codes u - 128, exact.
RFP2_DEV uint32_t less_1152(uint32_t h) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x64806480u));
    return d;
}
RFP2_DEV uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
RFP2_DEV float2 unpack_f16(uint32_t h) {
    __half2 v;
    memcpy(&v, &h, 4);
    return __half22float2(v);
}
RFP2_DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
RFP2_DEV float log2_fast(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A place on the line of tiles: unit (b, hk, ct) and tile t of its `tiles`.
struct AttnPlace {
    int b, hk, ct, t, tiles;
};

template <int NB, int NT, int PIECES>
__global__ void __launch_bounds__(kAttnThreads, attn_ctas_per_sm<NB, NT>())
    attn_kernel(const AttnArgs a) {
    using L = AttnLayout<NB>;
    using S = AttnShared<NB, NT>;
    constexpr int D = L::D, STAGES = attn_stages<NB, NT>(), COLS = 8 * NT;
    constexpr float kShift = 8.0f, kMost = 15.0f;  // p dV aims at 2^8 and stays below 2^15
    constexpr float kNone = -3.4e38f;              // the reference before any key
    // p is up to 2^15 / dV: 2^125 where the values are tiny (dV is taken as 2^-110 at least here)
    constexpr float kSumScale = 2.3283064365386963e-10f, kSumShift = 32.0f;  // 2^-32
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *rings = smem;
    float *join = reinterpret_cast<float *>(rings + kAttnWarps * STAGES * L::stage_bytes);
    float *state_r = join + S::join_bytes / 4, *state_l = state_r + kAttnWarps * COLS;
    int64_t *small = reinterpret_cast<int64_t *>(state_l + kAttnWarps * COLS);  // 8 words of 8 bytes
    int64_t *prefix = small + 8;                                                // [B + 1]
    int32_t *slen = reinterpret_cast<int32_t *>(prefix + a.B + 1);              // [B]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // ---- the line of tiles: how many each sequence has, and their prefix ----
    const auto tile_low = [&](int len) {
        if (a.window == 0) return 0;
        const int64_t low = (int64_t)len - a.nq + 1 - a.window;
        return low > 0 ? (int)(low / kAttnTile) : 0;
    };
    {
        int64_t run = 0;
        for (int b0 = 0; b0 < a.B; b0 += kAttnThreads) {
            const int b = b0 + tid;
            int tiles = 0;
            if (b < a.B) {
                int len = a.lens[b];
                if (len < 0 || len > a.capacity) {
                    if (blockIdx.x == 0) record_status(a.status, RFP2_EBADID);
                    len = -1;
                }
                slen[b] = len;
                // a sequence without keys still has its rows written
                tiles = max(1, (len + kAttnTile - 1) / kAttnTile - tile_low(len));
            }
            int64_t incl = tiles;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += up;
            }
            if (b0) __syncthreads();
            if (lane == 31) small[warp] = incl;
            __syncthreads();
            int64_t before = 0, total = 0;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                before += w < warp ? small[w] : 0;
                total += small[w];
            }
            if (b < a.B) prefix[b] = run + before + incl - tiles;
            run += total;
        }
        if (tid == 0) prefix[a.B] = run;
        __syncthreads();
    }
    const int units_of = a.heads * a.column_tiles;
    const int64_t total = prefix[a.B] * units_of;
    // at least one tile a warp: a short stretch is not worth a join
    const int64_t parts = min((int64_t)gridDim.x, (total + kAttnWarps - 1) / kAttnWarps);
    if ((int64_t)blockIdx.x >= parts) return;
    const int64_t x0 = blockIdx.x * total / parts, x1 = (blockIdx.x + 1) * total / parts;

    AttnPlace first;
    {
        int lo = 0, hi = a.B;  // the last b with prefix[b] * units_of <= x0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] * units_of <= x0) lo = mid; else hi = mid;
        }
        first.b = lo;
        first.tiles = (int)(prefix[lo + 1] - prefix[lo]);
        const int64_t off = x0 - prefix[lo] * units_of;
        const int unit = (int)(off / first.tiles);
        first.t = (int)(off - (int64_t)unit * first.tiles);
        first.hk = unit / a.column_tiles;
        first.ct = unit - first.hk * a.column_tiles;
    }
    const auto next_unit = [&](AttnPlace &p) {
        if (++p.ct == a.column_tiles) {
            p.ct = 0;
            if (++p.hk == a.heads) {
                p.hk = 0;
                ++p.b;
                p.tiles = p.b < a.B ? (int)(prefix[p.b + 1] - prefix[p.b]) : 1;
            }
        }
    };

    // ---- the loads: this warp's tiles x0 + warp, + 8, ... ----
    const uint32_t ring = smem_addr(rings) + warp * STAGES * L::stage_bytes;
    AttnPlace lp = first;
    int64_t lx = x0 + warp;  // tile of the next load
    lp.t += warp;
    const auto settle = [&]() {
        while (lx < x1 && lp.t >= lp.tiles) {
            lp.t -= lp.tiles;
            next_unit(lp);
        }
    };
    int32_t next_page = 0;  // of key `lane` of the next tile, fetched ahead of its use
    int next_key = -1;
    const auto fetch_page = [&]() {
        next_key = -1;
        if (lx < x1 && lane < kAttnTile) {
            const int len = slen[lp.b];
            const int j = (tile_low(len) + lp.t) * kAttnTile + lane;
            if (j < len) {
                next_key = j;
                next_page = a.table[lp.b * a.table_stride +
                                    (a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size)];
            }
        }
    };
    settle();
    fetch_page();
    const auto load_tile = [&](int stage) {
        if (lx < x1) {
            const uint32_t k_at = ring + stage * L::stage_bytes, v_at = k_at + L::k_bytes,
                           s_at = v_at + L::v_bytes;
            // row of the cache arrays, or -1 (no such key), -2 (no such page)
            constexpr uint32_t kNoKey = 0xFFFFFFFFu, kNoPage = 0xFFFFFFFEu;
            uint32_t row = kNoKey;
            if (next_key >= 0) {
                if (next_page < 0 || next_page >= a.pages) {
                    row = kNoPage;
                    record_status(a.status, RFP2_EBADID);
                } else {
                    const uint32_t off = a.page_shift >= 0 ? next_key & (a.page_size - 1)
                                                           : next_key % a.page_size;
                    row = ((uint32_t)next_page * a.heads + lp.hk) * a.page_size + off;
                }
            }
            constexpr int CH = D / 16;
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const int id = lane + 32 * i, r = id / CH, c = id - r * CH;
                const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                const bool ok = src < kNoPage;
                const int64_t at = ok ? (int64_t)src * D + 16 * c : 0;
                cp_async16(k_at + r * L::k_stride + 16 * c, a.k_codes + at, ok ? 16 : 0);
                cp_async16(v_at + r * L::v_stride + 16 * c, a.v_codes + at, ok ? 16 : 0);
            }
            // scales: 2 x 16 rows of NB floats, in the widest words that divide a row
            constexpr int W = NB % 4 == 0 ? 4 : NB % 2 == 0 ? 2 : 1, PER = NB / W;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int id = lane + 32 * i, r2 = id / PER, c = id - r2 * PER;
                const uint32_t src = __shfl_sync(0xffffffffu, row, r2 & 15);
                const bool ok = src < kNoPage;
                const int64_t at = ok ? (int64_t)src * NB + W * c : 0;
                const uint32_t dst = s_at + (r2 * NB + W * c) * 4;
                if (src == kNoPage && r2 < 16) {
                    // a key whose page does not exist: its scores are NaN
                    float *p = reinterpret_cast<float *>(rings + (dst - smem_addr(rings)));
#pragma unroll
                    for (int e = 0; e < W; ++e) p[e] = CUDART_NAN_F;
                } else {
                    cp_async_small<4 * W>(dst, (r2 < 16 ? a.k_scales : a.v_scales) + at, ok ? 4 * W : 0);
                }
            }
            lx += kAttnWarps;
            lp.t += kAttnWarps;
            settle();
            fetch_page();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) load_tile(s);

    // ---- stretches of units ----
    int stage = 0;
    AttnPlace p = first;
    int64_t x = x0;
    while (x < x1) {
        const int64_t end_x = min(x1, x + (p.tiles - p.t));  // of this stretch
        const int len = slen[p.b], low = tile_low(len);

        // columns: this lane's two of each tile in the score layout
        int col_end[NT][2];
        int min_end = 0x7fffffff, max_end = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = min(p.ct * COLS + nt * 8 + 2 * t4 + e, a.columns - 1);
                col_end[nt][e] = len - a.nq + 1 + c / a.group;
            }
        {
            const int c0 = p.ct * COLS, c1 = min(c0 + COLS, a.columns) - 1;
            min_end = len - a.nq + 1 + c0 / a.group;
            max_end = len - a.nq + 1 + c1 / a.group;
        }
        const int64_t max_begin = a.window ? (int64_t)max_end - a.window : 0;

        // q of column g: values 32 b + 8 t4 .. + 7, scaled by a power of two
        uint32_t qf[NT][NB][2][PIECES][2];
        float col_scale[NT][2], block_scale[NT][2];
        bool far = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = p.ct * COLS + nt * 8 + g;
            float v[NB][8];
            float top = 0.0f;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[n][e] = 0.0f;
            if (c < a.columns) {
                const int i = c / a.group, h = p.hk * a.group + c - i * a.group;
                const int64_t at = p.b * a.qb + i * a.qt + h * a.qh + 8 * t4;
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    if (PIECES == 2) {
                        const float *src = static_cast<const float *>(a.q) + at + 32 * n;
                        if (a.q_words) {
                            load_values<float, 8>(src, v[n]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[n][e] = src[e];
                        }
                    } else if (a.dtype == RFP2_BF16) {
                        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + at + 32 * n;
                        if (a.q_words) {
                            load_values<__nv_bfloat16, 8>(src, v[n]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[n][e] = to_f32(src[e]);
                        }
                    } else {
                        const __half *src = static_cast<const __half *>(a.q) + at + 32 * n;
                        if (a.q_words) {
                            load_values<__half, 8>(src, v[n]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[n][e] = to_f32(src[e]);
                        }
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[n][e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^up brings the largest value to [2^14, 2^15); a zero row stays as it is
            const int up = top > 0.0f ? min(141 - (int)(__float_as_uint(top) >> 23), 126) : 0;
            const float by = __uint_as_float((uint32_t)(127 + up) << 23);
            const float back = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float u = v[n][4 * s + 2 * h] * by, w = v[n][4 * s + 2 * h + 1] * by;
                        const uint32_t hi = pack_f16(u, w);
                        qf[nt][n][s][0][h] = hi;
                        if constexpr (PIECES == 2) {
                            const float2 f = unpack_f16(hi);
                            qf[nt][n][s][1][h] = pack_f16(u - f.x, w - f.y);
                        }
                    }
            far |= up > 40 || up < -40;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                block_scale[nt][e] = __shfl_sync(0xffffffffu, back, 4 * (2 * t4 + e));
        }
        // q's power of two goes back in at the end, or, where it is so far from 1 that it has to meet
        // scales as far on the other side, into every block's sum
        far = __any_sync(0xffffffffu, far);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                col_scale[nt][e] = (far ? 1.0f : block_scale[nt][e]) * a.scale *
                                   (a.softcap > 0.0f ? 1.0f : 1.4426950408889634f);

        float o[NT][NB][2][4];          // [column tile][block][pair of values][accumulator]
        float ref[NT][2], sum[NT][2];   // r - 8, and this lane's share of the sum of p
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][n][m][e] = 0.0f;
            ref[nt][0] = ref[nt][1] = kNone;
            sum[nt][0] = sum[nt][1] = 0.0f;
        }

        // tiles of this stretch that are this warp's: (tile - x0) % 8 == warp
        int skip = (int)((warp - (x - x0)) & (kAttnWarps - 1));
        for (int64_t xt = x + skip; xt < end_x; xt += kAttnWarps) {
            cp_async_wait<STAGES - 2>();
            __syncwarp();
            load_tile(stage == 0 ? STAGES - 1 : stage - 1);
            const uint8_t *tile = rings + (warp * STAGES + stage) * L::stage_bytes;
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            const uint8_t *kt = tile, *vt = tile + L::k_bytes;
            const float *ks = reinterpret_cast<const float *>(vt + L::v_bytes), *vs = ks + kAttnTile * NB;
            const int key0 = (low + p.t + (int)(xt - x)) * kAttnTile;

            // scores of keys g and g + 8
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
            float top_d[2] = {0.0f, 0.0f};
            float dv[2][NB];
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint2 lo = *reinterpret_cast<const uint2 *>(kt + g * L::k_stride + 32 * n + 8 * t4);
                const uint2 hi = *reinterpret_cast<const uint2 *>(kt + (g + 8) * L::k_stride + 32 * n + 8 * t4);
                const float d0 = ks[g * NB + n], d1 = ks[(g + 8) * NB + n];
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[nt][e] = 0.0f;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const uint32_t w0 = (s ? lo.y : lo.x) ^ 0x80808080u, w1 = (s ? hi.y : hi.x) ^ 0x80808080u;
                    const uint32_t f[4] = {less_1152(__byte_perm(w0, 0x64646464u, 0x4140)),
                                           less_1152(__byte_perm(w1, 0x64646464u, 0x4140)),
                                           less_1152(__byte_perm(w0, 0x64646464u, 0x4342)),
                                           less_1152(__byte_perm(w1, 0x64646464u, 0x4342))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int piece = PIECES - 1; piece >= 0; --piece)
                            mma_f16(c[nt], f, qf[nt][n][s][piece][0], qf[nt][n][s][piece][1]);
                }
                if (far)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[nt][e] *= block_scale[nt][e & 1];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    sc[nt][0] += d0 * c[nt][0];
                    sc[nt][1] += d0 * c[nt][1];
                    sc[nt][2] += d1 * c[nt][2];
                    sc[nt][3] += d1 * c[nt][3];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    dv[k][n] = vs[(g + 8 * k) * NB + n];
                    // an infinite or NaN scale is no measure of range
                    top_d[k] = fmaxf(top_d[k], dv[k][n] <= 3.4e38f ? dv[k][n] : 0.0f);
                }
            }
            const float lg[2] = {fmaxf(log2_fast(top_d[0]), -110.0f), fmaxf(log2_fast(top_d[1]), -110.0f)};

            const bool whole = key0 + kAttnTile <= min_end && key0 >= max_begin;
            bool more = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float s = sc[nt][e] * col_scale[nt][e & 1];
                    if (a.softcap > 0.0f) s = a.softcap * tanhf(s / a.softcap) * 1.4426950408889634f;
                    if (!whole) {
                        const int j = key0 + g + 8 * (e >> 1), end = col_end[nt][e & 1];
                        if (j >= end || (a.window && j < end - a.window)) s = -CUDART_INF_F;
                    }
                    sc[nt][e] = s;
                    more |= s - ref[nt][e & 1] + lg[e >> 1] > kMost;
                }
            if (__any_sync(0xffffffffu, more)) {
                // a larger reference for the columns that need one
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(sc[nt][e] + lg[0], sc[nt][e + 2] + lg[1]) - kShift;
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, ref[nt][e]);
                        const float keep = exp2_fast(ref[nt][e] - m);
                        ref[nt][e] = m;
                        sum[nt][e] *= keep;
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                o[nt][n][h][e] *= keep;
                                o[nt][n][h][e + 2] *= keep;
                            }
                    }
            }
            float pr[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pr[nt][e] = exp2_fast(sc[nt][e] - ref[nt][e & 1]);
                    sum[nt][e & 1] += pr[nt][e] * kSumScale;
                }

            // values: out^T += V^T (p dV), keys 2 t4, + 1, + 8, + 9
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                uint32_t pb[NT][PIECES][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float u = pr[nt][2 * k] * dv[k][n], w = pr[nt][2 * k + 1] * dv[k][n];
                        if (!whole) {  // whatever the scale of a key out of sight is
                            if (sc[nt][2 * k] == -CUDART_INF_F) u = 0.0f;
                            if (sc[nt][2 * k + 1] == -CUDART_INF_F) w = 0.0f;
                        }
                        const uint32_t hi = pack_f16(u, w);
                        pb[nt][0][k] = transpose8x8(hi);
                        if constexpr (PIECES == 2) {
                            const float2 f = unpack_f16(hi);
                            pb[nt][1][k] = transpose8x8(pack_f16(u - f.x, w - f.y));
                        }
                    }
                const uint8_t *vp = vt + 2 * t4 * L::v_stride + 32 * n + 4 * g;
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = *reinterpret_cast<const uint32_t *>(vp + ((k & 1) + 8 * (k >> 1)) * L::v_stride);
#pragma unroll
                for (int h = 0; h < 2; ++h) {  // values 4 g + 2 h and 4 g + 2 h + 1 of the block
                    const uint32_t sel = h ? 0x7362 : 0x5140;
                    const uint32_t u = __byte_perm(w[0], w[1], sel) ^ 0x80808080u;
                    const uint32_t v = __byte_perm(w[2], w[3], sel) ^ 0x80808080u;
                    const uint32_t f[4] = {less_1152(__byte_perm(u, 0x64646464u, 0x4140)),
                                           less_1152(__byte_perm(u, 0x64646464u, 0x4342)),
                                           less_1152(__byte_perm(v, 0x64646464u, 0x4140)),
                                           less_1152(__byte_perm(v, 0x64646464u, 0x4342))};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (PIECES == 2) {
                            // the matrix unit cuts sums off; a long chain of them is kept in fp32 adds
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                            mma_f16(c, f, pb[nt][1][0], pb[nt][1][1]);
                            mma_f16(c, f, pb[nt][0][0], pb[nt][0][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][n][h][e] += c[e];
                        } else {
                            mma_f16(o[nt][n][h], f, pb[nt][0][0], pb[nt][0][1]);
                        }
                    }
                }
            }
        }

        // ---- the warps join ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = sum[nt][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    state_r[warp * COLS + nt * 8 + 2 * t4 + e] = ref[nt][e];
                    state_l[warp * COLS + nt * 8 + 2 * t4 + e] = l;
                }
            }
        __syncthreads();
        const auto top_of = [&](int c) {
            float m = kNone;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) m = fmaxf(m, state_r[w * COLS + c]);
            return m;
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float by = exp2_fast(ref[nt][e] - top_of(nt * 8 + 2 * t4 + e));
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        o[nt][n][h][e] *= by;
                        o[nt][n][h][e + 2] *= by;
                    }
            }

        const bool split = p.t != 0 || end_x - x != p.tiles;
        constexpr int SLOT = 2 * COLS + COLS * D;  // floats: references, sums, values
        const int64_t unit0 = x - p.t;             // first tile of the unit on the line
        float *slot = a.partials + (2 * (int64_t)blockIdx.x + (x != x0)) * SLOT;
        const auto store_row = [&](int c, int d, const float (&y)[4]) {
            const int cg = p.ct * COLS + c, i = cg / a.group;
            const int64_t at = (((int64_t)p.b * a.nq + i) * a.Hq + p.hk * a.group + cg - i * a.group) * D + d;
            if (PIECES == 2) {
                *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
            } else if (a.dtype == RFP2_BF16) {
                __nv_bfloat16 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = from_f32<__nv_bfloat16>(y[e]);
                uint2 u;
                memcpy(&u, v, 8);
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) = u;
            } else {
                __half v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = from_f32<__half>(y[e]);
                uint2 u;
                memcpy(&u, v, 8);
                *reinterpret_cast<uint2 *>(static_cast<__half *>(a.out) + at) = u;
            }
        };
        const auto store_lse = [&](int c, float m, float l) {
            const int cg = p.ct * COLS + c, i = cg / a.group;
            a.lse[((int64_t)p.b * a.nq + i) * a.Hq + p.hk * a.group + cg - i * a.group] =
                len < 0 ? CUDART_NAN_F : l == 0.0f ? -CUDART_INF_F : (m + kSumShift) * 0.6931471805599453f + logf(l);
        };
        const int live = min(COLS, a.columns - p.ct * COLS);
        constexpr int CHUNK = S::chunk;
#pragma unroll
        for (int d0 = 0; d0 < D; d0 += CHUNK) {
            if (d0) __syncthreads();
#pragma unroll
            for (int n = d0 / 32; n < NB && n < (d0 + CHUNK) / 32; ++n)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        *reinterpret_cast<float4 *>(join + (warp * COLS + nt * 8 + 2 * t4 + e) * S::row +
                                                    32 * n - d0 + 4 * g) =
                            make_float4(o[nt][n][0][e], o[nt][n][0][e + 2], o[nt][n][1][e], o[nt][n][1][e + 2]);
            __syncthreads();
            const int words = min(CHUNK, D - d0) / 4;
            for (int i = tid; i < live * words; i += kAttnThreads) {
                const int c = i / words, d = 4 * (i - c * words);
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f;
                const float m = top_of(c);
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    const float4 v = *reinterpret_cast<const float4 *>(join + (w * COLS + c) * S::row + d);
                    y[0] += v.x;
                    y[1] += v.y;
                    y[2] += v.z;
                    y[3] += v.w;
                    l += state_l[w * COLS + c] * exp2_fast(state_r[w * COLS + c] - m);
                }
                if (split) {
                    *reinterpret_cast<float4 *>(slot + 2 * COLS + c * D + d0 + d) = make_float4(y[0], y[1], y[2], y[3]);
                    if (d0 + d == 0) {
                        slot[c] = m;
                        slot[COLS + c] = l;
                    }
                } else {
                    const float inv = kSumScale / l;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = len < 0 ? CUDART_NAN_F : l == 0.0f ? 0.0f : y[e] * inv;
                    store_row(c, d0 + d, y);
                    if (a.lse && d0 + d == 0) store_lse(c, m, l);
                }
            }
        }
        if (split) {
            // CTAs of this unit: those that hold its first and its last tile, and between
            const int64_t c0 = ((unit0 + 1) * parts - 1) / total;
            const int64_t c1 = ((unit0 + p.tiles) * parts - 1) / total;
            __threadfence();
            __syncthreads();
            int *flag = reinterpret_cast<int *>(small);
            if (tid == 0) *flag = atomicAdd(a.counters + c0, 1) == (int)(c1 - c0);
            __syncthreads();
            if (*flag) {
                __threadfence();
                if (tid == 0) a.counters[c0] = 0;
                const int words = D / 4;
                const int64_t slot0 = 2 * c0 + (unit0 != c0 * total / parts);
                for (int i = tid; i < live * words; i += kAttnThreads) {
                    const int c = i / words, d = 4 * (i - c * words);
                    float m = kNone, l = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int64_t k = c0; k <= c1; ++k)
                        m = fmaxf(m, __ldcg(a.partials + (k == c0 ? slot0 : 2 * k) * SLOT + c));
                    for (int64_t k = c0; k <= c1; ++k) {
                        const float *from = a.partials + (k == c0 ? slot0 : 2 * k) * SLOT;
                        const float by = exp2_fast(__ldcg(from + c) - m);
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(from + 2 * COLS + c * D + d));
                        l += __ldcg(from + COLS + c) * by;
                        y[0] += v.x * by;
                        y[1] += v.y * by;
                        y[2] += v.z * by;
                        y[3] += v.w * by;
                    }
                    const float inv = kSumScale / l;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = l == 0.0f ? 0.0f : y[e] * inv;
                    store_row(c, d, y);
                    if (a.lse && d == 0) store_lse(c, m, l);
                }
            }
        }
        __syncthreads();  // the join buffer and the states are free again
        p.t = 0;
        next_unit(p);
        x = end_x;
    }
    cp_async_wait<0>();
}

// Launches one group of sequences; a.B <= kAttnMaxBatch.
template <int NB, int NT, int PIECES>
cudaError_t attn_launch(const AttnArgs &a, int sms, cudaStream_t stream) {
    static std::atomic<int> ready[64];  // by device: its shared memory limit is set
    const int device = current_device();
    if (device >= 64 || !ready[device].load(std::memory_order_relaxed)) {
        const cudaError_t e =
            set_smem_limit(attn_kernel<NB, NT, PIECES>, attn_smem<NB, NT>(kAttnMaxBatch));
        if (e != cudaSuccess) return e;
        if (device < 64) ready[device].store(1, std::memory_order_relaxed);
    }
    return launch(attn_kernel<NB, NT, PIECES>, dim3((unsigned)(sms * attn_ctas_per_sm<NB, NT>())),
                  dim3(kAttnThreads), attn_smem<NB, NT>(a.B), stream, true, a);
}

// Column tiles of 8 or, from 9 columns up, 16 (where the registers hold them).
template <int NB>
constexpr int attn_most_columns() { return NB <= 4 ? 16 : 8; }

template <int NB>
cudaError_t attn_by_columns(const AttnArgs &a, int sms, cudaStream_t stream) {
    if constexpr (attn_most_columns<NB>() == 16)
        if (a.columns > 8)
            return a.dtype == RFP2_F32 ? attn_launch<NB, 2, 2>(a, sms, stream)
                                       : attn_launch<NB, 2, 1>(a, sms, stream);
    return a.dtype == RFP2_F32 ? attn_launch<NB, 1, 2>(a, sms, stream)
                               : attn_launch<NB, 1, 1>(a, sms, stream);
}

// By blocks of 32 values a head; each is instantiated in one translation unit.
using AttnFn = cudaError_t (*)(const AttnArgs &, int, cudaStream_t);
cudaError_t attn_d32(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d64(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d96(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d128(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d160(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d192(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d224(const AttnArgs &a, int sms, cudaStream_t stream);
cudaError_t attn_d256(const AttnArgs &a, int sms, cudaStream_t stream);

}  // namespace rfp2
