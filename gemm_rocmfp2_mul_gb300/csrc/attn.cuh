// Decode attention over the paged Q8 cache: the kernel and its arguments.  The
// translation units attn_*.cu instantiate it by head size.
//
//   s_j = scale * sum_b dK[j, b] (sum over block b of q kq[j]),   softcap tanh(s / softcap)
//   out = sum_j p_j dV[j, b] vq[j] / sum_j p_j,  p_j = exp(s_j - max s),  lse = max s + ln sum_j p_j
//
// Bound by memory: each key of a head is 2 (D + D/8) bytes, read once for all
// its query heads and tokens ("columns").  Work is cut in tiles of 16 keys.  The
// tiles of all (sequence, key head, column tile) units lie on one line, with a
// gap before each unit that stands for its fixed cost, and the warps of the
// grid share the line out evenly whatever the lengths are.  A warp streams its
// stretch through its own ring in shared memory (cp.async), keeps its own
// softmax state and meets no barrier on the way; units that lie within its
// stretch it writes itself.  What it holds of units that reach beyond is joined
// at the end: within the CTA through shared memory, between CTAs through the
// workspace by the last of them to arrive, always in the order of the keys.
//
// Products run on 16-bit matrix instructions (16 keys x 8 columns x 16 values).
// Scores: codes are exact in f16, q goes in scaled by a power of two (one f16
// piece is exact for 16-bit q down to 2^-28 of its row's largest value; two leave
// 2^-22 of fp32 q; neither less than 2^-39 of the largest), and the block sums are
// scaled by dK in fp32.  Outputs: codes are exact in bf16 as well, and p dV goes in
// as bf16 pieces, which have fp32's range: however far apart the weights of the
// keys and the scales of a row's blocks are, each product keeps its own digits.
// Two pieces (the first 8 bits of p dV, and the rest rounded to 8) leave 2^-15 of
// it for 16-bit outputs, three are all 24 bits for fp32.  (f16 pieces, one for bf16
// outputs, took 350 us where these take 385, 55 where 60 and 40.5 where 44 below,
// but needed one exponent for all blocks of a key and lost what lay far below.)
//
// Measured (one GB300, back to back): 64 sequences of up to 32768 keys, 64 heads
// over 8 of 128, bf16: 385 us for 2.39 GB (6.2 TB/s; copy rate 6.7); one of 131072
// keys, 40 over 8: 60 us (5.0 TB/s); 16 of up to 8192, 32 over 8, fp32: 44 us (4.3
// TB/s); one of 1000 keys: 9.4 us, of 16: 4.5 us.  The start (three dependent reads)
// and the joins take about 8 us of a long call; on the way the instructions of three
// warps a scheduler set the pace, 607 a tile of 8 columns x 128 values, in 60 % of the
// issue slots.
#pragma once

#include <atomic>

#include "activation.cuh"

namespace rfp2 {

constexpr int kAttnTile = 16;        // keys
// A unit's fixed cost, in tiles.  1, 2 and 4: 38.4, 33.4 and 33.3 us for 7 sequences
// of 16 heads of 256 values, 26.8, 24.4 and 24.2 us for 53 of up to 926 keys.
constexpr int kAttnGap = 4;
// The shortest stretch of a warp, in tiles: 1 tile against 2, one sequence of 1000
// keys: 9.4 and 10.6 us.
constexpr int kAttnMinStretch = 1;
// Tiles a warp (gap included) up to which a unit stays in one CTA where the CTAs
// suffice: 8 heads of 256 keys 7.3 us in one CTA each and 8.7 joined, 512 keys 9.0
// and 9.1, 1000 keys 13.0 and 9.4.
constexpr int kAttnWholeUnit = 4;
// Bytes of the cache on their way to an SM, at most.  55 KB, 110 and 166, by the
// stages of 12 warps (64 sequences, 2.4 GB): 386 us, 386 and 388; 8 heads of 1000 keys:
// 9.5, 9.4 and 9.4; 53 sequences of up to 926: 23.8, 24.2 and 25.2.
constexpr int kAttnInFlight = 112 * 1024;
constexpr int kAttnMaxBatch = 1024;  // sequences of one launch
// Tiles whose weights are summed by themselves before they join the unit's sum: one
// by one, small weights round off beside what a large one has left (lse of 131072
// keys, 1700 tiles a warp: 4.5e-6 off, so 6e-7).
constexpr int kAttnSums = 32;

struct AttnArgs {
    const void *q;
    int64_t qb, qt, qh;
    const int8_t *k_codes, *v_codes;
    const float *k_scales, *v_scales;
    const int32_t *table, *lens;
    int64_t pages, table_stride, capacity;
    int B, nq, Hq, heads, group, columns, column_tiles;
    int page_size;
    int whole_pages;            // page_size % 16 == 0: a tile lies in one page
    int dtype, q_words;         // q_words: q can be read as 16-byte words
    // divisors of the launch, multiplied by: a division by a value only known at
    // run time is some 25 instructions on the way to the first load, and again at
    // every unit (12 x 5 tokens of 16 heads over 2, D = 64, pages of 48: 14.0 ->
    // 13.4 us; 7 x 16 heads of D = 256, pages of 33: 34.7 -> 33.3 us)
    FastDiv by_page, by_group, by_tiles;  // page_size, group, column_tiles
    float scale, softcap;
    int64_t window;
    void *out;
    float *lse;
    int *counters;
    float *partials;
    int32_t *status;
};

// A tile in shared memory.  K is read 8 bytes a lane, four keys a half-warp, V 4
// bytes a lane, keys two apart.  Rows of a multiple of 128 bytes have their
// 32-byte blocks permuted by the two bits in which those keys differ; others are
// padded, so that K's rows are an odd number of 32-byte steps apart and V's an
// odd number of 16-byte steps.  Neither read meets a bank twice.
template <int NB>
struct AttnLayout {
    static constexpr int D = 32 * NB;
    static constexpr bool permuted = NB % 4 == 0;
    static constexpr int k_stride = permuted || NB % 2 ? D : D + 32;
    static constexpr int v_stride = permuted ? D : D + 16;
    static constexpr int k_bytes = kAttnTile * k_stride, v_bytes = kAttnTile * v_stride;
    static constexpr int scale_bytes = kAttnTile * NB * 4;
    static constexpr int stage_bytes = k_bytes + v_bytes + 2 * scale_bytes;
    // block n of key r lies where block n ^ k_order(r), n ^ v_order(r) would
    static RFP2_DEV int k_order(int r) { return permuted ? r & 3 : 0; }
    static RFP2_DEV int v_order(int r) { return permuted ? r >> 1 & 3 : 0; }
};

// What the warps leave of a unit that reaches beyond their stretch.
struct AttnPiece {
    int present, starts;  // starts: holds the unit's first tile
    int b, hk, ct;
    int unit0;            // the unit's place on the line
};

// How q and p dV go into the products as pieces.  The kinds for up to four columns
// have second pieces as columns 4 .. 7 of the products.
constexpr int kHalf = 1;      // 16-bit activations: one piece of q, two of p dV
constexpr int kF32 = 2;       // two of q, three of p dV
constexpr int kPairHalf = 3;  // up to four columns
constexpr int kPairF32 = 4;

// Warps: the tile's work is a long chain, so as many as the registers hold.  By
// head size x columns (what a warp accumulates): 12 up to 128 values x 16 at 168
// registers, where q's fragments of 16 columns wait in shared memory (8: 436 us for 12's
// 386 of 64 sequences); beyond that 8.  Small ones run two CTAs of 8.  (Spilled to hold that: of 16 columns 16-20 bytes
// at 128 values, 24 at 256; of 8 columns of 256 values 8, fp32.)
constexpr int attn_warps(int NB, int NT) { return NB * NT <= 2 || NB > 4 ? 8 : 12; }
constexpr int attn_ctas_per_sm(int NB, int NT) { return NB * NT <= 2 ? 2 : 1; }
// Bytes of a warp's q fragments in shared memory: each lane's own, for two column
// tiles.
template <int NB, int NT, int PIECES>
constexpr int attn_q_bytes() { return NT == 2 ? NB * 2 * (PIECES == kF32 ? 2 : 1) * NT * 256 : 0; }

// The warps' sums of the scan, the pieces and their columns' states, and the
// line's prefix.
template <int WARPS, int NT>
constexpr int attn_small_bytes(int B) {
    return 128 + 2 * WARPS * ((int)sizeof(AttnPiece) + 2 * 8 * NT * 4) + (B + 1) * 4;
}
template <int NB, int NT, int PIECES>
constexpr int attn_stages() {
    constexpr int W = attn_warps(NB, NT);
    const int budget = (attn_ctas_per_sm(NB, NT) == 2 ? 113 : 227) * 1024;
    const int s = (budget - attn_small_bytes<W, NT>(kAttnMaxBatch) - W * attn_q_bytes<NB, NT, PIECES>()) /
                  (W * AttnLayout<NB>::stage_bytes);
    // the tiles on their way to an SM; the last stage is the one that is worked on
    const int wanted = 1 + kAttnInFlight / (W * attn_ctas_per_sm(NB, NT) * kAttnTile * NB * 72);
    return s < 2 || wanted < 2 ? 2 : s < wanted ? s : wanted;
}
template <int NB, int NT, int PIECES>
constexpr int attn_smem(int B) {
    constexpr int W = attn_warps(NB, NT);
    return W * (attn_stages<NB, NT, PIECES>() * AttnLayout<NB>::stage_bytes + attn_q_bytes<NB, NT, PIECES>()) +
           attn_small_bytes<W, NT>(B);
}
// Floats of one partial result: the columns' references and sums, and their
// values.
constexpr int attn_slot(int NB, int NT) { return 8 * NT * (2 + 32 * NB); }

RFP2_DEV void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
RFP2_DEV void cp_async_small(uint32_t dst, const void *src) {
    if constexpr (N == 16)
        cp_async16(dst, src);
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
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
// The same with bf16 in.
RFP2_DEV void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
RFP2_DEV uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
// Two bytes u = code + 128, bytes 0 and 2 of h, as two f16 of 2^-24 of the codes, exact: as the bits of an f16 a byte
// is u 2^-24.
RFP2_DEV uint32_t codes_f16(uint32_t h) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(0x00800080u));
    return d;
}
RFP2_DEV uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
// What is left of (lo, hi) beside the two f16 of h, as two f16.
RFP2_DEV uint32_t rest_f16(uint32_t h, float lo, float hi) {
    float u, v;
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " sub.rn.f32.f16 %0, a, %3;\n sub.rn.f32.f16 %1, b, %4;\n}\n"
        : "=f"(u), "=f"(v)
        : "r"(h), "f"(lo), "f"(hi));
    return pack_f16(-u, -v);
}
// Two codes, bytes 0 and 2 of h, as two bf16 of a 64th of them, exact: a byte u as the bits of a bf16 is u 2^-133 (up
// to the smallest normal binade they are linear), u = code + 128, and a fused product with 2^127 takes 2 off.
RFP2_DEV uint32_t codes_bf16(uint32_t h) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(d)
        : "r"((h & 0x00FF00FFu) ^ 0x00800080u), "r"(0x7F007F00u), "r"(0xC000C000u));
    return d;
}
// The first 8 bits of (lo, hi) as two bf16, and what is left of them, exact.
RFP2_DEV uint32_t first_bf16(float &lo, float &hi) {
    const uint32_t u = __float_as_uint(lo), w = __float_as_uint(hi);
    lo -= __uint_as_float(u & 0xFFFF0000u);
    hi -= __uint_as_float(w & 0xFFFF0000u);
    return __byte_perm(u, w, 0x7632);
}
RFP2_DEV uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
RFP2_DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A key's NB scales, in the widest words that divide its row.
template <int NB>
RFP2_DEV void load_scales(const float *p, float (&d)[NB]) {
    if constexpr (NB % 4 == 0) {
#pragma unroll
        for (int n = 0; n < NB; n += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + n);
            d[n] = v.x, d[n + 1] = v.y, d[n + 2] = v.z, d[n + 3] = v.w;
        }
    } else if constexpr (NB % 2 == 0) {
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(p + n);
            d[n] = v.x, d[n + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int n = 0; n < NB; ++n) d[n] = p[n];
    }
}

// A place on the line: unit (b, hk, ct) of `tiles` tiles that begins (with its
// gap) at `unit0`.
struct AttnPlace {
    int b, hk, ct, tiles, unit0;
};

// The line's share of each warp: `each` places, one more for the first `extra`.
struct AttnShare {
    uint32_t each, extra;
    RFP2_DEV int begin(uint32_t worker) const { return (int)(worker * each + min(worker, extra)); }
    RFP2_DEV uint32_t worker_of(uint32_t x) const {
        const uint32_t more = extra * (each + 1);
        return x < more ? x / (each + 1) : extra + (x - more) / each;
    }
};

template <int NB, int NT, int PIECES>
__global__ void __launch_bounds__(32 * attn_warps(NB, NT), attn_ctas_per_sm(NB, NT))
    attn_kernel(const AttnArgs a) {
    using L = AttnLayout<NB>;
    constexpr int WARPS = attn_warps(NB, NT), THREADS = 32 * WARPS;
    constexpr bool PAIR = PIECES == kPairHalf || PIECES == kPairF32;
    constexpr bool fp32 = PIECES == kF32 || PIECES == kPairF32;  // the activations
    constexpr int Q_PARTS = PIECES == kF32 ? 2 : 1, P_PARTS = PIECES == kPairHalf ? 1 : PIECES == kF32 ? 3 : 2;
    constexpr int PER = PAIR ? 4 : 8;  // columns of a tile
    static_assert(!PAIR || NT == 1, "");
    constexpr int D = L::D, STAGES = attn_stages<NB, NT, PIECES>(), COLS = 8 * NT, SLOT = attn_slot(NB, NT);
    static_assert(SLOT * 4 <= STAGES * L::stage_bytes, "a warp's partial result fits its ring");
    static_assert(STAGES >= 2 && WARPS <= 16, "");
    static_assert(attn_smem<NB, NT, PIECES>(kAttnMaxBatch) <= (attn_ctas_per_sm(NB, NT) == 2 ? 113 : 227) * 1024, "");
    // p = 2^(s - r), with r the largest s but for at most 4: 16 at most, and it goes with a 64th of the codes, so that
    // their product is a quarter of a value at most
    constexpr float kSlack = 4.0f;
    constexpr float kCodes = 64.0f;                // the products' codes are 64ths
    constexpr float kNone = -3.4e38f;              // the reference before any key
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *rings = smem;
    constexpr bool Q_SHARED = attn_q_bytes<NB, NT, PIECES>() > 0;
    uint2 *q_frags = reinterpret_cast<uint2 *>(rings + WARPS * STAGES * L::stage_bytes);  // [warps][fragments][lanes]
    int *small = reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(q_frags) +
                                         WARPS * attn_q_bytes<NB, NT, PIECES>());  // 32
    AttnPiece *pieces = reinterpret_cast<AttnPiece *>(small + 32);                  // [warps][head, tail]
    float *piece_r = reinterpret_cast<float *>(pieces + 2 * WARPS);                 // [pieces][COLS]
    float *piece_l = piece_r + 2 * WARPS * COLS;
    int *prefix = reinterpret_cast<int *>(piece_l + 2 * WARPS * COLS);  // [B + 1]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    // this lane's columns of tile nt in the score layout, and whether it is the one that writes them
    const auto column_of = [&](int nt, int e) { return nt * 8 + ((2 * t4 + e) & (PER - 1)); };
    const bool writes = !PAIR || t4 < 2;
    // 16-byte word w of column c of a piece lies where word w ^ slot_order(c) would: so its writers, eight
    // lanes in four columns, meet no bank twice
    const auto slot_order = [](int c) { return c & 6; };
    pdl_wait();
    pdl_launch_dependents();

    // ---- the line: each sequence's length on it for one unit, and their prefix ----
    const auto length_of = [&](int b) {  // -1: not a length
        const int len = a.lens[b];
        return len < 0 || len > a.capacity ? -1 : len;
    };
    const auto first_key = [&](int len) {  // that any query sees
        return a.window == 0 ? 0 : (int)max((int64_t)0, (int64_t)len - a.nq + 1 - a.window);
    };
    const auto tile_low = [&](int len) { return first_key(len) / kAttnTile; };
    const auto cost_of = [&](int b) {
        const int len = length_of(b);
        if (len < 0 && blockIdx.x == 0) record_status(a.status, RFP2_EBADID);
        // a sequence without keys has one tile too: its rows are written
        return kAttnGap + max(1, (len + kAttnTile - 1) / kAttnTile - tile_low(len));
    };
    if (lane < 2) pieces[2 * warp + lane].present = 0;
    const int units_of = a.heads * a.column_tiles;
    bool whole_units = false;  // a CTA for every unit
    if (a.B <= 32) {
        // every warp by itself
        const int cost = lane < a.B ? cost_of(lane) : 0;
        whole_units = a.B * units_of <= (int)gridDim.x &&
                      __reduce_max_sync(0xffffffffu, cost) <= kAttnWholeUnit * WARPS;
        int incl = cost;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += up;
        }
        if (lane < a.B) prefix[lane + 1] = incl;
        if (lane == 0) prefix[0] = 0;
        __syncwarp();
    } else {
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += THREADS) {
            const int b = b0 + tid;
            int incl = b < a.B ? cost_of(b) : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += up;
            }
            if (b0) __syncthreads();
            if (lane == 31) small[warp] = incl;
            __syncthreads();
            int before = 0, all = 0;
            for (int w = 0; w < WARPS; ++w) {
                before += w < warp ? small[w] : 0;
                all += small[w];
            }
            if (b < a.B) prefix[b + 1] = run + before + incl;
            run += all;
        }
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
    }
    const int total = prefix[a.B] * units_of;
    // Some tiles for each warp: shorter stretches are not worth their joins.  And where there are fewer
    // units than CTAs, each of a few tiles a warp, a unit stays in one CTA: those tiles cost less than a
    // join across CTAs.
    const int parts = whole_units ? a.B * units_of
                                  : min((int)gridDim.x, (total - 1) / (kAttnMinStretch * WARPS) + 1);
    if ((int)blockIdx.x >= parts) return;
    const int worker = blockIdx.x * WARPS + warp;
    AttnShare share;
    AttnPlace first;
    int y0, y1;
    const auto place_unit = [&](int b, int unit) {
        const int cost = prefix[b + 1] - prefix[b];
        first.b = b;
        first.tiles = cost - kAttnGap;
        first.unit0 = prefix[b] * units_of + unit * cost;
        first.hk = a.by_tiles(unit);
        first.ct = unit - first.hk * a.column_tiles;
        return cost;
    };
    if (whole_units) {
        const int b = blockIdx.x / units_of, cost = place_unit(b, blockIdx.x - b * units_of);
        // from the first tile on: the gap costs nothing here
        share.each = (uint32_t)(cost - kAttnGap) / WARPS;
        share.extra = cost - kAttnGap - share.each * WARPS;
        y0 = first.unit0 + kAttnGap + share.begin(warp);
        y1 = first.unit0 + kAttnGap + share.begin(warp + 1);
    } else {
        share.each = (uint32_t)total / (uint32_t)(parts * WARPS);
        share.extra = total - share.each * parts * WARPS;
        y0 = share.begin(worker);
        y1 = share.begin(worker + 1);
        int lo = 0, hi = a.B;  // the last b with prefix[b] * units_of <= y0
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] * units_of <= y0) lo = mid; else hi = mid;
        }
        place_unit(lo, (uint32_t)(y0 - prefix[lo] * units_of) / (uint32_t)(prefix[lo + 1] - prefix[lo]));
    }
    const auto next_unit = [&](AttnPlace &p) {
        p.unit0 += p.tiles + kAttnGap;
        if (++p.ct == a.column_tiles) {
            p.ct = 0;
            if (++p.hk == a.heads) {
                p.hk = 0;
                ++p.b;
                p.tiles = p.b < a.B ? prefix[p.b + 1] - prefix[p.b] - kAttnGap : 1;
            }
        }
    };
    // this warp's tiles [from, to) of a unit
    const auto tiles_from = [&](const AttnPlace &p) {
        return max(0, y0 - p.unit0 - kAttnGap);
    };
    const auto tiles_to = [&](const AttnPlace &p) {
        return max(0, min(p.tiles, y1 - p.unit0 - kAttnGap));
    };

    // ---- the loads, STAGES - 1 tiles ahead ----
    const uint32_t ring = smem_addr(rings) + warp * STAGES * L::stage_bytes;
    AttnPlace lp = first;
    int lt = 0, lt_end = 0, l_len = 0, l_low = 0;  // tile of the next load; of its unit
    bool loading = true;
    // Pages of the tiles to come, those of the `block` tiles from page_at on, and the ones after them on
    // their way.  Where a tile lies in one page, lane i holds that of tile page_at + i; else that of the
    // i-th key from tile page_at on.
    const int block = a.whole_pages ? 32 : 2, key_step = a.whole_pages ? kAttnTile : 1;
    int32_t page = -1, page_after = -1;
    int page_at = 0;
    const auto pages_from = [&](int t) {
        const int j = (l_low + t) * kAttnTile + lane * key_step;
        return j < l_len ? a.table[lp.b * a.table_stride + a.by_page(j)] : -1;
    };
    // enters units until one has tiles in this stretch
    const auto enter = [&]() {
        while (true) {
            if (lp.unit0 + kAttnGap >= y1) {
                loading = false;
                return;
            }
            lt = tiles_from(lp);
            lt_end = tiles_to(lp);
            if (lt < lt_end) break;
            next_unit(lp);
        }
        l_len = length_of(lp.b);
        l_low = tile_low(l_len);
        page_at = lt;
        page = pages_from(lt);
        page_after = lt + block < lt_end ? pages_from(lt + block) : -1;
    };
    enter();
    // a unit's rows of q on their way while the unit before is worked on
    const auto prefetch_q = [&](const AttnPlace &p) {
        const int size = fp32 ? 4 : 2, lines = fp32 ? 2 * NB : NB;  // of 64 bytes: one address at least of each 128
        const int c0 = p.ct * COLS, live = min(COLS, a.columns - c0);
        for (int k = lane; k < live * lines; k += 32) {
            const int cl = (fp32 ? k >> 1 : k) / NB, c = c0 + cl, i = a.by_group(c), h = p.hk * a.group + c - i * a.group;
            const int64_t at = p.b * a.qb + i * a.qt + h * a.qh;
            const char *src = static_cast<const char *>(a.q) + at * size + (k - cl * lines) * 64;
            asm volatile("prefetch.global.L1 [%0];" ::"l"(src));
        }
    };
    const auto load_tile = [&](int stage) {
        if (loading) {
            const uint32_t k_at = ring + stage * L::stage_bytes, v_at = k_at + L::k_bytes,
                           s_at = v_at + L::v_bytes;
            constexpr int CH = D / 16;
            // scales: rows of NB floats, in the widest words that divide a row
            constexpr int W = NB % 4 == 0 ? 4 : NB % 2 == 0 ? 2 : 1, PER = NB / W;
            const int key0 = (l_low + lt) * kAttnTile;
            // of 16-byte word c of key r
            const auto k_place = [&](int r, int c) { return r * L::k_stride + 16 * (c ^ L::k_order(r) << 1); };
            const auto v_place = [&](int r, int c) { return r * L::v_stride + 16 * (c ^ L::v_order(r) << 1); };
            if (lt - page_at == block) {
                page = page_after;
                page_at = lt;
                page_after = lt + block < lt_end ? pages_from(lt + block) : -1;
            }
            if (a.whole_pages) {
                const int32_t next_page = __shfl_sync(0xffffffffu, page, lt - page_at);
                // sixteen rows that follow one another; those past the sequence's end are masked later
                if (key0 >= l_len) {
                    // an empty sequence: nothing to read, and its place is masked
                } else if (next_page < 0 || next_page >= a.pages) {
                    record_status(a.status, RFP2_EBADID);
                    float *p = reinterpret_cast<float *>(rings + (s_at - smem_addr(rings)));
#pragma unroll
                    for (int i = 0; i < (kAttnTile * NB + 31) / 32; ++i)
                        if (lane + 32 * i < kAttnTile * NB) p[lane + 32 * i] = CUDART_NAN_F;
                } else {
                    const uint32_t off = key0 - a.by_page(key0) * a.page_size;
                    const uint32_t row = ((uint32_t)next_page * a.heads + lp.hk) * a.page_size + off;
                    const int8_t *kp = a.k_codes + (int64_t)row * D + 16 * lane;
                    const int8_t *vp = a.v_codes + (int64_t)row * D + 16 * lane;
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
                        const int id = lane + 32 * i, r = id / CH, c = id - r * CH;
                        cp_async16(k_at + k_place(r, c), kp + 512 * i);
                        cp_async16(v_at + v_place(r, c), vp + 512 * i);
                    }
                    const float *ks = a.k_scales + (int64_t)row * NB, *vs = a.v_scales + (int64_t)row * NB;
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int id = lane + 32 * i, half = id >= 16 * PER, at = W * (id - half * 16 * PER);
                        cp_async_small<4 * W>(s_at + 4 * W * id, (half ? vs : ks) + at);
                    }
                }
            } else {
                // row of the cache arrays of key `lane`, or -1 (no such key, or out of sight: its page may be
                // another's by now), -2 (no such page)
                constexpr uint32_t kNoKey = 0xFFFFFFFFu, kNoPage = 0xFFFFFFFEu;
                uint32_t row = kNoKey;
                const int j = key0 + (lane & (kAttnTile - 1));
                const int32_t own_page = __shfl_sync(0xffffffffu, page, (lt - page_at) * kAttnTile + (lane & (kAttnTile - 1)));
                if (j < l_len && j >= first_key(l_len)) {
                    if (own_page < 0 || own_page >= a.pages) {
                        row = kNoPage;
                        record_status(a.status, RFP2_EBADID);
                    } else {
                        const uint32_t off = j - a.by_page(j) * a.page_size;
                        row = ((uint32_t)own_page * a.heads + lp.hk) * a.page_size + off;
                    }
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int id = lane + 32 * i, r = id / CH, c = id - r * CH;
                    const uint32_t src = __shfl_sync(0xffffffffu, row, r);
                    if (src < kNoPage) {
                        const int64_t at = (int64_t)src * D + 16 * c;
                        cp_async16(k_at + k_place(r, c), a.k_codes + at);
                        cp_async16(v_at + v_place(r, c), a.v_codes + at);
                    }
                }
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int id = lane + 32 * i, r2 = id / PER, c = id - r2 * PER;
                    const uint32_t src = __shfl_sync(0xffffffffu, row, r2 & 15);
                    const uint32_t dst = s_at + (r2 * NB + W * c) * 4;
                    if (src == kNoPage) {
                        // a key whose page does not exist: its scores are NaN
                        float *p = reinterpret_cast<float *>(rings + (dst - smem_addr(rings)));
#pragma unroll
                        for (int e = 0; e < W; ++e) p[e] = CUDART_NAN_F;
                    } else if (src != kNoKey) {
                        cp_async_small<4 * W>(dst, (r2 < 16 ? a.k_scales : a.v_scales) + (int64_t)src * NB + W * c);
                    }
                }
            }
            if (++lt == lt_end) {
                next_unit(lp);
                enter();
                if (loading) prefetch_q(lp);
            }
        }
        cp_async_commit();
    };

    // ---- outputs: four values d .. d + 3 of column c of a unit, and its lse ----
    const auto row_of = [&](int b, int hk, int cg) {
        const int i = a.by_group(cg);
        return ((int64_t)b * a.nq + i) * a.Hq + hk * a.group + cg - i * a.group;
    };
    const auto store_four = [&](int64_t row, int d, const float (&y)[4]) {
        const int64_t at = row * D + d;
        if (fp32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
            uint2 u;
            if (a.dtype == RFP2_BF16) {
                __nv_bfloat16 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = from_f32<__nv_bfloat16>(y[e]);
                memcpy(&u, v, 8);
            } else {
                __half v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = from_f32<__half>(y[e]);
                memcpy(&u, v, 8);
            }
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = u;
        }
    };
    const auto lse_of = [&](float m, float l) {
        return l == 0.0f ? -CUDART_INF_F : m * 0.6931471805599453f + logf(l);
    };

    // four values d .. d + 3 of column c of a unit that is joined: references and sums m and l
    const auto finish = [&](const AttnPiece &u, int c, int d, float (&y)[4], float m, float l) {
        const float inv = l == 0.0f ? 0.0f : kCodes / l;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] *= inv;
        const int64_t row = row_of(u.b, u.hk, u.ct * COLS + c);
        store_four(row, d, y);
        if (a.lse && d == 0) a.lse[row] = lse_of(m, l);
    };

    // ---- the units of this stretch ----
    const float cap_out = a.softcap * 1.4426950408889634f;
    // tanhf for 16-bit types too, 0.4 us of 13.4 for 12 x 5 tokens: the lse of few keys shows an error of
    // 2e-7 of the cap, as 1 - 2 / (e^2x + 1) has it near 0
    const float cap_in = fminf(1.0f / a.softcap, 3.402823466e38f);
    // Queries of any size on keys of any size: 2^-24 of the codes and q below 2^15 make a block's sum 8 at most, so that
    // no scale of fp32's takes a score's sum out of its range; what q was scaled by comes off first, these last.
    const float to_score = 16777216.0f * a.scale * (a.softcap > 0.0f ? 1.0f : 1.4426950408889634f);
    int stage = 0;
    bool filled = false;
    for (AttnPlace p = first; p.unit0 + kAttnGap < y1; next_unit(p)) {
        const int from = tiles_from(p), to = tiles_to(p);
        if (from >= to) continue;
        const int len = length_of(p.b), low = tile_low(len);

        // columns: this lane's two of each tile in the score layout
        int col_end[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = min(p.ct * COLS + column_of(nt, e), a.columns - 1);
                col_end[nt][e] = len - a.nq + 1 + (int)a.by_group(c);
            }
        const int c_last = min(p.ct * COLS + COLS, a.columns) - 1;
        const int min_end = len - a.nq + 1 + (int)a.by_group(p.ct * COLS);
        const int64_t max_begin = a.window ? len - a.nq + 1 + (int)a.by_group(c_last) - a.window : 0;

        // q of column g: values 32 n + 8 t4 .. + 7, scaled by a power of two
        uint32_t qf[Q_SHARED ? 1 : NB][2][Q_PARTS][2];
        uint2 *q_mine = q_frags + warp * (attn_q_bytes<NB, NT, PIECES>() / 8) + lane;
        const auto q_place = [](int nt, int n, int s, int part) { return (((nt * NB + n) * 2 + s) * Q_PARTS + part) * 32; };
        float col_scale[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int c = p.ct * COLS + nt * 8 + (g & (PER - 1));
            float v[NB][8];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[n][e] = 0.0f;
            if (c < a.columns) {
                const int i = a.by_group(c), h = p.hk * a.group + c - i * a.group;
                const int64_t at = p.b * a.qb + i * a.qt + h * a.qh + 8 * t4;
                if (fp32) {
                    const float *src = static_cast<const float *>(a.q) + at;
                    if (a.q_words) {
#pragma unroll
                        for (int n = 0; n < NB; ++n) load_values<float, 8>(src + 32 * n, v[n]);
                    } else {
#pragma unroll
                        for (int n = 0; n < NB; ++n)
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[n][e] = src[32 * n + e];
                    }
                } else {
                    const uint16_t *src = static_cast<const uint16_t *>(a.q) + at;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        uint16_t u[8];
                        if (a.q_words) {
                            const uint4 w = *reinterpret_cast<const uint4 *>(src + 32 * n);
                            memcpy(u, &w, 16);
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) u[e] = src[32 * n + e];
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[n][e] = a.dtype == RFP2_BF16 ? __uint_as_float((uint32_t)u[e] << 16)
                                                           : __half2float(__ushort_as_half(u[e]));
                    }
                }
            }
            if (!filled) {
                // the first tiles, behind the first unit's q: what comes later queues behind them
#pragma unroll 1
                for (int s = 0; s < STAGES - 1; ++s) load_tile(s);
                filled = true;
            }
            float top = 0.0f;
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[n][e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^up brings the largest value to [2^14, 2^15); a zero row stays as it is
            const int up = top > 0.0f ? min(141 - (int)(__float_as_uint(top) >> 23), 126) : 0;
            const float by = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int s = 0; s < 2; ++s)
{
                    uint32_t part[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float u = v[n][4 * s + 2 * h] * by, w = v[n][4 * s + 2 * h + 1] * by;
                        const uint32_t hi = pack_f16(u, w);
                        part[0][h] = hi;
                        if constexpr (PIECES == kPairF32) part[0][h] = g < 4 ? hi : rest_f16(hi, u, w);
                        if constexpr (Q_PARTS == 2) part[1][h] = rest_f16(hi, u, w);
                    }
#pragma unroll
                    for (int i = 0; i < Q_PARTS; ++i) {
                        if constexpr (Q_SHARED) {
                            q_mine[q_place(nt, n, s, i)] = make_uint2(part[i][0], part[i][1]);
                        } else {
                            qf[n][s][i][0] = part[i][0];
                            qf[n][s][i][1] = part[i][1];
                        }
                    }
                }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                col_scale[nt][e] = __uint_as_float(
                    (uint32_t)(127 - __shfl_sync(0xffffffffu, up, 4 * column_of(0, e))) << 23);
        }

        float o[NT][NB][2][4];          // [column tile][block][pair of values][accumulator]
        float ref[NT][2], sum[NT][2];   // r, and this lane's share of the sum of p
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

#pragma unroll 1
        for (int t = from; t < to;) {
            const int stop = min(to, t + kAttnSums);
            float part[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) part[nt][0] = part[nt][1] = 0.0f;
#pragma unroll 1
            for (; t < stop; ++t) {
                cp_async_wait<STAGES - 2>();
                __syncwarp();
                load_tile(stage == 0 ? STAGES - 1 : stage - 1);
                const uint8_t *kt = rings + (warp * STAGES + stage) * L::stage_bytes, *vt = kt + L::k_bytes;
                const float *ks = reinterpret_cast<const float *>(vt + L::v_bytes), *vs = ks + kAttnTile * NB;
                stage = stage + 1 == STAGES ? 0 : stage + 1;
                const int key0 = (low + t) * kAttnTile;

                // scales of keys g and g + 8
                float dk[2][NB], dv[2][NB];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    load_scales<NB>(ks + (g + 8 * k) * NB, dk[k]);
                    load_scales<NB>(vs + (g + 8 * k) * NB, dv[k]);
                }

                // scores of keys g and g + 8
                float sc[NT][4];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int at = 32 * (n ^ L::k_order(g)) + 8 * t4;
                    const uint2 lo = *reinterpret_cast<const uint2 *>(kt + g * L::k_stride + at);
                    const uint2 hi = *reinterpret_cast<const uint2 *>(kt + (g + 8) * L::k_stride + at);
                    float c[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[nt][e] = 0.0f;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t w0 = (s ? lo.y : lo.x) ^ 0x80808080u, w1 = (s ? hi.y : hi.x) ^ 0x80808080u;
                        const uint32_t f[4] = {codes_f16(__byte_perm(w0, 0u, 0x4140)),
                                               codes_f16(__byte_perm(w1, 0u, 0x4140)),
                                               codes_f16(__byte_perm(w0, 0u, 0x4342)),
                                               codes_f16(__byte_perm(w1, 0u, 0x4342))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int piece = Q_PARTS - 1; piece >= 0; --piece) {
                                if constexpr (Q_SHARED) {
                                    const uint2 q = q_mine[q_place(nt, n, s, piece)];
                                    mma_f16(c[nt], f, q.x, q.y);
                                } else {
                                    mma_f16(c[nt], f, qf[n][s][piece][0], qf[n][s][piece][1]);
                                }
                            }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[nt][e] = n ? sc[nt][e] + dk[e >> 1][n] * c[nt][e] : dk[e >> 1][n] * c[nt][e];
                }

                if constexpr (PIECES == kPairF32)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[0][e] += __shfl_xor_sync(0xffffffffu, sc[0][e], 2);

                const bool whole = key0 + kAttnTile <= min_end && key0 >= max_begin;
                bool more = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[nt][e] = sc[nt][e] * col_scale[nt][e & 1] * to_score;
                if (a.softcap > 0.0f)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[nt][e] = cap_out * tanhf(sc[nt][e] * cap_in);
                if (!whole) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = key0 + g + 8 * (e >> 1), end = col_end[nt][e & 1];
                            if (j >= end || (a.window && j < end - a.window)) sc[nt][e] = -CUDART_INF_F;
                        }
                    // a value's scale that is not finite counts where its key is seen, and there alone
                    bool odd = false;
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        odd |= !(fabsf(dv[0][n]) <= 3.402823466e38f) || !(fabsf(dv[1][n]) <= 3.402823466e38f);
                    if (__any_sync(0xffffffffu, odd))
#pragma unroll
                        for (int n = 0; n < NB; ++n) {
                            const bool bad[2] = {!(fabsf(dv[0][n]) <= 3.402823466e38f),
                                                 !(fabsf(dv[1][n]) <= 3.402823466e38f)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const bool seen = (bad[0] && sc[nt][e] != -CUDART_INF_F) ||
                                                      (bad[1] && sc[nt][e + 2] != -CUDART_INF_F);
                                    // by any of the lanes of this column
                                    if (__ballot_sync(0xffffffffu, seen) & 0x11111111u << t4)
#pragma unroll
                                        for (int h = 0; h < 2; ++h) o[nt][n][h][e] = o[nt][n][h][e + 2] = CUDART_NAN_F;
                                }
                            if (bad[0]) dv[0][n] = 0.0f;
                            if (bad[1]) dv[1][n] = 0.0f;
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) more |= sc[nt][e] - ref[nt][e & 1] > kSlack;
                if (__any_sync(0xffffffffu, more)) {
                    // a larger reference for the columns that need one
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float m = fmaxf(sc[nt][e], sc[nt][e + 2]);
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            m = fmaxf(m, ref[nt][e]);
                            const float keep = exp2_fast(ref[nt][e] - m);
                            ref[nt][e] = m;
                            sum[nt][e] *= keep;
                            part[nt][e] *= keep;
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
                        part[nt][e & 1] += pr[nt][e];
                    }

                // values: out^T += V^T (p dV), keys 2 t4, + 1, + 8, + 9
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    // p dV in the layout that the products take it in
                    uint32_t pb[NT][P_PARTS][2];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float u = pr[nt][2 * k] * dv[k][n], w = pr[nt][2 * k + 1] * dv[k][n];
                            const uint32_t hi = first_bf16(u, w);
                            if constexpr (PIECES == kHalf) {
                                pb[nt][0][k] = transpose8x8(hi);
                                pb[nt][1][k] = transpose8x8(pack_bf16(u, w));
                            } else if constexpr (PIECES == kPairHalf) {
                                pb[nt][0][k] = transpose8x8(t4 < 2 ? hi : pack_bf16(u, w));
                            } else {
                                const uint32_t mid = first_bf16(u, w), lo = first_bf16(u, w);
                                if constexpr (PIECES == kF32) {
                                    pb[nt][0][k] = transpose8x8(hi);
                                    pb[nt][1][k] = transpose8x8(mid);
                                    pb[nt][2][k] = transpose8x8(lo);
                                } else {
                                    pb[nt][0][k] = transpose8x8(t4 < 2 ? hi : mid);
                                    pb[nt][1][k] = transpose8x8(t4 < 2 ? lo : 0u);
                                }
                            }
                        }
                    const uint8_t *vp = vt + 2 * t4 * L::v_stride + 32 * (n ^ L::v_order(2 * t4)) + 4 * g;
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = *reinterpret_cast<const uint32_t *>(vp + ((k & 1) + 8 * (k >> 1)) * L::v_stride);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // values 4 g + 2 h and 4 g + 2 h + 1 of the block
                        const uint32_t at0 = h ? 0x0602 : 0x0400, at1 = h ? 0x0703 : 0x0501;
                        const uint32_t f[4] = {
                            codes_bf16(__byte_perm(w[0], w[1], at0)), codes_bf16(__byte_perm(w[0], w[1], at1)),
                            codes_bf16(__byte_perm(w[2], w[3], at0)), codes_bf16(__byte_perm(w[2], w[3], at1))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            // the matrix unit cuts its sums off: 1.4e-7 of them a tile, were they kept there.  (As the
                            // accumulators of the products: 368 us of 64 sequences, so 384.)
                            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                            for (int i = P_PARTS - 1; i >= 0; --i) mma_bf16(c, f, pb[nt][i][0], pb[nt][i][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[nt][n][h][e] += c[e];
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) sum[nt][e] += part[nt][e];
        }

        // ---- the end of the unit, or of the stretch ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 4);
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 8);
                sum[nt][e] += __shfl_xor_sync(0xffffffffu, sum[nt][e], 16);
            }
        if constexpr (PAIR)
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[0][n][h][e] += __shfl_xor_sync(0xffffffffu, o[0][n][h][e], 2);
        if (from == 0 && to == p.tiles) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int cg = p.ct * COLS + column_of(nt, e);
                    if (!writes || cg >= a.columns) continue;
                    const int64_t row = row_of(p.b, p.hk, cg);
                    const float l = sum[nt][e], inv = l == 0.0f ? 0.0f : kCodes / l;
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        float y[4] = {o[nt][n][0][e] * inv, o[nt][n][0][e + 2] * inv, o[nt][n][1][e] * inv,
                                      o[nt][n][1][e + 2] * inv};
                        if (len < 0) y[0] = y[1] = y[2] = y[3] = CUDART_NAN_F;
                        store_four(row, 32 * n + 4 * g, y);
                    }
                    if (a.lse && g == 0) a.lse[row] = len < 0 ? CUDART_NAN_F : lse_of(ref[nt][e], l);
                }
        } else {
            // a head (the unit ends here) goes to the workspace: the ring is in use.  A tail is the
            // stretch's last: it goes to the ring, which its loads have left.
            const bool tail = to != p.tiles;
            float *slot;
            if (tail) {
                cp_async_wait<0>();
                __syncwarp();
                slot = reinterpret_cast<float *>(rings + warp * STAGES * L::stage_bytes);
            } else {
                slot = a.partials + (2 * gridDim.x + worker) * (int64_t)SLOT;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = column_of(nt, e);
                    if (!writes) continue;
                    if (g == 0) {
                        piece_r[(2 * warp + tail) * COLS + c] = ref[nt][e];
                        piece_l[(2 * warp + tail) * COLS + c] = sum[nt][e];
                    }
#pragma unroll
                    for (int n = 0; n < NB; ++n)
                        *reinterpret_cast<float4 *>(slot + c * D + 4 * ((8 * n + g) ^ slot_order(c))) =
                            make_float4(o[nt][n][0][e], o[nt][n][0][e + 2], o[nt][n][1][e], o[nt][n][1][e + 2]);
                }
            if (lane == 0) {
                AttnPiece &x = pieces[2 * warp + tail];
                x.starts = from == 0;
                x.b = p.b;
                x.hk = p.hk;
                x.ct = p.ct;
                x.unit0 = p.unit0;
                x.present = 1;
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // ---- the CTA's pieces: those of one unit follow one another, a head is its last ----
    constexpr int WORDS = COLS * D / 4;
    const uint32_t present = __ballot_sync(0xffffffffu, lane < 2 * WARPS && pieces[min(lane, 2 * WARPS - 1)].present);
    if (present == 0) return;
    uint32_t ends = present & 0x55555555u;         // heads, and a last tail
    ends |= present & (0x80000000u >> __clz(present));
    const int groups = __popc(ends);
    const auto members_of = [&](int j) {  // pieces of group j, as bits
        uint32_t rest = ends, below = 0;
        for (int k = 0; k < j; ++k) {
            below = 2u * (rest & -rest) - 1u;
            rest &= rest - 1;
        }
        return present & (2u * (rest & -rest) - 1u) & ~below;
    };
    const AttnPiece *head_unit = pieces + __ffs(present) - 1;                 // of the first group
    const AttnPiece *tail_unit = pieces + __ffs(members_of(groups - 1)) - 1;  // of the last
    const bool split0 = !head_unit->starts;
    const bool split1 = (31 - __clz(present)) % 2 == 1 && !(split0 && groups == 1);
    for (int k = tid; k < groups * WORDS; k += THREADS) {
        const int j = k / WORDS, c = (k - j * WORDS) / (D / 4), d = 4 * (k % (D / 4));
        const uint32_t members = members_of(j), tails = members & ~0x55555555u, head = members & 0x55555555u;
        const AttnPiece &u = pieces[__ffs(members) - 1];
        if (c >= a.columns - u.ct * COLS) continue;
        const int at = d ^ 4 * slot_order(c);
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f}, l = 0.0f, m = kNone, r[WARPS];
        float4 hv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int hw = head ? __ffs(head) - 1 : 0;
        if (head) {
            hv = *reinterpret_cast<const float4 *>(
                a.partials + (2 * gridDim.x + blockIdx.x * WARPS + (hw >> 1)) * (int64_t)SLOT + c * D + at);
            m = piece_r[hw * COLS + c];
        }
        const float hr = m;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            r[w] = tails >> (2 * w + 1) & 1u ? piece_r[(2 * w + 1) * COLS + c] : kNone;
            m = fmaxf(m, r[w]);
        }
        const auto add = [&](const float4 &v, float by) {
            y[0] += v.x * by;
            y[1] += v.y * by;
            y[2] += v.z * by;
            y[3] += v.w * by;
        };
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            if (tails >> (2 * w + 1) & 1u) {
                const float by = exp2_fast(r[w] - m);
                l += piece_l[(2 * w + 1) * COLS + c] * by;
                add(*reinterpret_cast<const float4 *>(rings + w * STAGES * L::stage_bytes + (c * D + at) * 4), by);
            }
        if (head) {
            const float by = exp2_fast(hr - m);
            l += piece_l[hw * COLS + c] * by;
            add(hv, by);
        }
        if (u.starts && head) {
            finish(u, c, d, y, m, l);
        } else {
            // a unit of several CTAs
            float *mine = a.partials + (2 * (int64_t)blockIdx.x + u.starts) * SLOT;
            const float inv = l == 0.0f ? 0.0f : kCodes / l;
            *reinterpret_cast<float4 *>(mine + 2 * COLS + c * D + d) =
                make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
            if (d == 0) *reinterpret_cast<float2 *>(mine + 2 * c) = make_float2(m, l);
        }
    }
    if (!split0 && !split1) return;

    // ---- units of several CTAs: the first group, if it did not start here, and the last, if it does
    // not end here.  The last CTA of each to arrive joins it. ----
    int *arrived = small, *from_cta = small + 4;  // [2][2]: joins, CTAs; [2]
    __syncthreads();
    if (lane == 0 && warp < 2) {
        int joins = 0, n = 0;
        if (warp == 0 ? split0 : split1) {
            const AttnPiece *u = warp == 0 ? head_unit : tail_unit;
            const int t0 = u->unit0 + kAttnGap, tiles = prefix[u->b + 1] - prefix[u->b] - kAttnGap;
            const int c0 = share.worker_of(t0) / WARPS, c1 = share.worker_of(t0 + tiles - 1) / WARPS;
            n = c1 - c0 + 1;
            __threadfence();  // the CTA's parts, before it is counted
            joins = atomicAdd(a.counters + c0, 1) == n - 1;
            if (joins) {
                __threadfence();  // the other CTAs' parts, after they are
                a.counters[c0] = 0;
            }
            from_cta[warp] = c0;
        }
        arrived[2 * warp] = joins;
        arrived[2 * warp + 1] = n;
    }
    __syncthreads();
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        if (!arrived[2 * which]) continue;
        const AttnPiece &u = which == 0 ? *head_unit : *tail_unit;
        const int n = arrived[2 * which + 1], live = min(COLS, a.columns - u.ct * COLS);
        // the CTAs' parts, each with its own sum divided out, which weighs it.  Of the first CTA its second
        // slot, of the others their first
        const float *parts0 = a.partials + (2 * from_cta[which] + 1) * (int64_t)SLOT;
        const auto part_of = [&](int i) { return parts0 + (i ? (2 * i - 1) * (int64_t)SLOT : 0); };
        for (int k = tid; k < live * (D / 4); k += THREADS) {
            const int c = k / (D / 4), d = 4 * (k - c * (D / 4));
            float m = kNone, l = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            constexpr int AHEAD = 16;  // parts whose loads travel together
#pragma unroll 1
            for (int i0 = 0; i0 < n; i0 += AHEAD) {
                float4 v[AHEAD];
                float2 r[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    r[i] = make_float2(kNone, 0.0f);
                    v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i0 + i < n) {
                        const float *from = part_of(i0 + i);
                        r[i] = __ldcg(reinterpret_cast<const float2 *>(from) + c);
                        v[i] = __ldcg(reinterpret_cast<const float4 *>(from + 2 * COLS + c * D + d));
                    }
                }
                float top = m;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) top = fmaxf(top, r[i].x);
                const float keep = exp2_fast(m - top);
                m = top;
                l *= keep;
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] *= keep;
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const float by = r[i].y * exp2_fast(r[i].x - m);
                    l += by;
                    y[0] += v[i].x * by;
                    y[1] += v[i].y * by;
                    y[2] += v[i].z * by;
                    y[3] += v[i].w * by;
                }
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= inv;
            const int64_t row = row_of(u.b, u.hk, u.ct * COLS + c);
            store_four(row, d, y);
            if (a.lse && d == 0) a.lse[row] = lse_of(m, l);
        }
    }
}

// Launches one group of sequences; a.B <= kAttnMaxBatch.
template <int NB, int NT, int PIECES>
cudaError_t attn_launch(const AttnArgs &a, int sms, cudaStream_t stream) {
    static std::atomic<int> ready[64];  // by device: its shared memory limit is set
    const int device = current_device();
    if (device >= 64 || !ready[device].load(std::memory_order_relaxed)) {
        const cudaError_t e =
            set_smem_limit(attn_kernel<NB, NT, PIECES>, attn_smem<NB, NT, PIECES>(kAttnMaxBatch));
        if (e != cudaSuccess) return e;
        if (device < 64) ready[device].store(1, std::memory_order_relaxed);
    }
    return launch(attn_kernel<NB, NT, PIECES>, dim3((unsigned)(sms * attn_ctas_per_sm(NB, NT))),
                  dim3(32 * attn_warps(NB, NT)), attn_smem<NB, NT, PIECES>(a.B), stream, true, a);
}

// Column tiles of 8 or, from 9 columns up, 16: a tile's codes are converted once
// for all of them.  (Of heads past 128 values, fp32's two pieces for 16 columns
// would not fit beside the ring.)
inline int attn_most_columns(int D, int dtype, int columns) {
    return columns > 8 && (D <= 128 || dtype != RFP2_F32) ? 16 : 8;
}

template <int NB>
cudaError_t attn_by_columns(const AttnArgs &a, int sms, cudaStream_t stream) {
    const bool two = attn_most_columns(32 * NB, a.dtype, a.columns) == 16;
    if (a.dtype != RFP2_F32) {
        if (a.columns <= 4) return attn_launch<NB, 1, kPairHalf>(a, sms, stream);
        return two ? attn_launch<NB, 2, kHalf>(a, sms, stream) : attn_launch<NB, 1, kHalf>(a, sms, stream);
    }
    if (a.columns <= 4) return attn_launch<NB, 1, kPairF32>(a, sms, stream);
    if constexpr (NB <= 4)
        if (two) return attn_launch<NB, 2, kF32>(a, sms, stream);
    return attn_launch<NB, 1, kF32>(a, sms, stream);
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
