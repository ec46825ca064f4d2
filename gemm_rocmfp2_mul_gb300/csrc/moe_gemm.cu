// The routed experts' products for any number of tokens:
//   z = W[e] x + bias[e];  y = z, or act(z[gate rows]) * z[up rows];  a row of y for each (token, slot) pair.
//
// Two launches:
//  1. plan (one CTA): the pairs sorted by expert, and each expert's run cut into tiles of at most 256 tokens.
//  2. the product on the tensor cores: units of a tile and 256 weight rows (128 gate rows and the 128 up rows
//     that go with them).
//
// Measured (one GB300, GPU time a call): 8192 tokens to 2 of 8 experts of 14336 x 4096, gated: 1160-1305 us by how
// long the chip has been busy, 1.47-1.66 PFLOP/s (0.76-0.86 of cuBLAS's burst rate, which has no weights to decode;
// 0.77 is what rfp2_gemm has); 2047 to 8 of 256 of 1536 x 2048, gated: 254 us; 16 to 8 of 256 of 768 x 2048: 38 us.
// Wide tiles are bound by the shared-memory port, narrow ones by a stage's way around.
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "rfp2_decode.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace rfp2 {
namespace {

constexpr int kTileTokens = 256;  // of a tile at most, and 64 at least where tiles are narrow
constexpr int kMaxExperts = 1024;
constexpr int64_t kMaxPairs = 1 << 24;
constexpr int kPlanThreads = 1024;

// Workspace: header (tiles, pairs with an expert, pairs), the pairs by expert (those without one last),
// and the tiles.
struct Plan {
    int *header;
    int *pairs;
    int4 *tiles;  // expert, first place in pairs, tokens
};

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
int64_t most_tiles(int64_t P, int64_t E) { return P / 64 + std::min(P, E); }  // of any width
size_t plan_bytes(int64_t P, int64_t E) {
    return 256 + align256((size_t)P * 4) + align256((size_t)most_tiles(P, E) * 16);
}
Plan carve_plan(void *ws, int64_t P) {
    uint8_t *p = static_cast<uint8_t *>(ws);
    return {reinterpret_cast<int *>(p), reinterpret_cast<int *>(p + 256),
            reinterpret_cast<int4 *>(p + 256 + align256((size_t)P * 4))};
}

// Exclusive sum of (a, b) over the CTA's threads, and their totals.
RFP2_DEV int2 scan_pairs(int2 v, int2 *sums, int2 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s.x, off), y = __shfl_up_sync(0xffffffffu, s.y, off);
        if (lane >= off) s.x += x, s.y += y;
    }
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int2 w = sums[lane];
        const int2 own = w;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, w.x, off), y = __shfl_up_sync(0xffffffffu, w.y, off);
            if (lane >= off) w.x += x, w.y += y;
        }
        sums[lane] = make_int2(w.x - own.x, w.y - own.y);
        if (lane == 31) sums[32] = w;
    }
    __syncthreads();
    total = sums[32];
    return make_int2(sums[warp].x + s.x - v.x, sums[warp].y + s.y - v.y);
}

// Each warp counts a stretch of the pairs by expert in a row of shared memory of its own, the rows become
// places, and each warp puts its stretch there.  Lanes that meet in one expert are in no fixed order, which
// changes nothing: a column's sums do not depend on its place in a tile.  (Ranks by matching lanes, in a
// fixed order, took 35 us of 16376 pairs over 256 experts.)
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const int32_t *__restrict__ ids, int P, int E, int warps,
                                                               int tile, Plan plan, int32_t *status) {
    extern __shared__ int count[];  // [warps][E + 1], the last for pairs without an expert
    __shared__ int2 sums[33];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bins = E + 1;
    for (int i = tid; i < warps * bins; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    const int chunk = ((P + warps - 1) / warps + 31) / 32 * 32;
    const int from = min(P, warp * chunk), to = warp < warps ? min(P, from + chunk) : from;
    int *mine = count + warp * bins;
    // the ids are fetched eight words at a time, all on their way together
    constexpr int kAhead = 8;
    int id[kAhead];
    const auto fetch = [&](int p0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int p = p0 + 32 * i + lane;
            id[i] = p < to ? ids[p] : 0;
        }
    };
    for (int p0 = from; p0 < to; p0 += 32 * kAhead) {
        fetch(p0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (p0 + 32 * i >= to) break;
            const bool in = p0 + 32 * i + lane < to;
            const int b = !in ? -1 : (unsigned)id[i] < (unsigned)E ? id[i] : E;
            if (b == E && id[i] != -1) record_status(status, RFP2_EBADID);
            if (b >= 0) atomicAdd(&mine[b], 1);
        }
    }
    __syncthreads();
    // thread e: the places of expert e's pairs and tiles
    int n = 0;
    if (tid < E)
        for (int w = 0; w < warps; ++w) n += count[w * bins + tid];
    const int tiles = (n + tile - 1) / tile;
    int2 total;
    const int2 at = scan_pairs(make_int2(n, tiles), sums, total);
    if (tid < E) {
        int place = at.x;
        for (int w = 0; w < warps; ++w) {
            const int c = count[w * bins + tid];
            count[w * bins + tid] = place;
            place += c;
        }
        // tiles of one expert are as good as equal
        const int each = tiles ? (n + tiles - 1) / tiles : 0;
        for (int i = 0; i < tiles; ++i)
            plan.tiles[at.y + i] = make_int4(tid, at.x + i * each, min(each, n - i * each), 0);
    }
    if (tid == 0) {
        plan.header[0] = total.y;
        plan.header[1] = total.x;
        plan.header[2] = P;
        int place = total.x;
        for (int w = 0; w < warps; ++w) {
            const int c = count[w * bins + E];
            count[w * bins + E] = place;
            place += c;
        }
    }
    __syncthreads();
    for (int p0 = from; p0 < to; p0 += 32 * kAhead) {
        if (to - from > 32 * kAhead) fetch(p0);  // a short stretch is still there
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (p0 + 32 * i >= to) break;
            const int p = p0 + 32 * i + lane;
            const int b = p >= to ? -1 : (unsigned)id[i] < (unsigned)E ? id[i] : E;
            if (b >= 0) plan.pairs[atomicAdd(&mine[b], 1)] = p;
        }
    }
}

struct GemmArgs {
    const __nv_bfloat16 *X;
    const float *bias;
    __nv_bfloat16 *Y;
    const int32_t *ids;
    Plan plan;
    int M, K, each, out;
    FastDiv by_top_k;
};

// Both activations are gate / (1 + exp(-v)): v = gate, or twice tanh's argument.  With h = exp(-|v| / 2) they are
// gate s / (1 + h^2) s, where s is 1 for v >= 0 and h below: the divisor stays within [1, 2], where a reciprocal
// needs no care for its range, and act(gate) * up is formed before it would underflow (h is 0 from |v| = 174 on).
// The approximate exponential and reciprocal are off by 2^-21 (2 + |v|) of the result at most, which is rounded to
// bf16; with exact ones the epilogue held the MMAs up (1363 us of the first case above and 277 of the second).
RFP2_DEV float activated(int activation, float gate, float up) {
    const float v = activation == RFP2_ACT_SILU ? gate : 1.5957691216057308f * fmaf(0.044715f * gate * gate, gate, gate);
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(-0.72134752044448170f * fabsf(v)));  // log2(e) / 2
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.0f)));
    const float s = v < 0.0f ? h : 1.0f;
    return gate * s * r * (up * s);
}

// The rows of pairs without an expert: zeros for -1, NaN for another id.  A warp a row, in words of 16 bytes (a row
// is a multiple of 16 values); warp `of` of `warps` takes every warps-th row, and 32 of them have their places and
// ids on their way together.  By a warp that has no other work, beside the products: 57344 of 65536 rows of 7168 take
// 0.2 ms, as a plain fill does.  (Single values, written by the epilogue ahead of its first tile, took 5.5 ms, in
// which the MMAs waited; of arrays that fill the memory nearly the time limit of their waits.)
RFP2_DEV void fill_rest(const GemmArgs &a, int of, int warps) {
    const int lane = threadIdx.x & 31;
    const int first = a.plan.header[1], rest = a.plan.header[2] - first, words = a.out / 8;
    for (int i0 = of; i0 < rest; i0 += 32 * warps) {
        const int i = i0 + lane * warps;
        int p = 0;
        uint32_t fill = 0;
        if (i < rest) {
            p = a.plan.pairs[first + i];
            fill = a.ids[p] == -1 ? 0u : 0x7FFF7FFFu;
        }
        const int n = min(32, (rest - i0 + warps - 1) / warps);
        for (int j = 0; j < n; ++j) {
            const uint32_t f = __shfl_sync(0xffffffffu, fill, j);
            uint4 *row = reinterpret_cast<uint4 *>(a.Y + (int64_t)__shfl_sync(0xffffffffu, p, j) * a.out);
            for (int w = lane; w < words; w += 32) row[w] = make_uint4(f, f, f, f);
        }
    }
}

// ---- the product --------------------------------------------------------------
constexpr int kRows = 128;   // weight rows of a CTA (TMEM lanes), 256 of a pair (UMMA M)
constexpr int kStep = 64;    // K of a stage: one 128-byte swizzle row
constexpr int kUmmaK = 16;   // K of an instruction
constexpr int kABytes = kRows * kStep * 2;
constexpr int kBoxRowBytes = 80;  // eight 10-byte blocks: four steps of K
constexpr int kBoxBytes = kRows * kBoxRowBytes;
constexpr int kBoxes = 4;
constexpr int kGroups = 4;      // decoders: group i takes steps i, i + 4, ...
constexpr int kGroupWarps = 4;  // a weight row a thread
constexpr int kDecodeWarps = kGroups * kGroupWarps;
constexpr int kLoadWarps = 4;  // gather the tokens: warp i of them steps i, i + 4, ...
constexpr int kThreads = (6 + kDecodeWarps + kLoadWarps) * 32;
constexpr uint32_t kTmemCols = 512;  // two accumulators of 256 columns
// By the most tokens of a tile: a stage is a slice of 64 of K of both operands, and a narrow tile leaves room for
// more of them.  A stage's way around (tokens' loads, both SMs' arrivals, MMAs, their commit) takes about 2500
// cycles however narrow it is, so that the number of stages sets the pace there.
template <int TILE>
struct Cfg {
    static constexpr int kBBytes = TILE / 2 * kStep * 2;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = TILE == 64 ? 9 : TILE == 128 ? 7 : 5;
    static constexpr size_t kRingOff = (size_t)kStages * kStageBytes;
    static constexpr size_t kBarOff = kRingOff + (size_t)kBoxes * kBoxBytes;
    static constexpr size_t kSmemBytes = 1024 + kBarOff + 256;
    static constexpr int kLoads = TILE / 2 / 4;  // copies of a lane for a step, at most
    static_assert(kSmemBytes <= 227 * 1024 && (2 * kStages + 4 + 2 * kBoxes) * 8 + 8 <= 256, "shared memory");
};

// Has the phase with `parity` completed?  (No waiting.)
RFP2_DEV bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// mbar_wait, which reads the GPU's timer once a probe has failed, after probes without it.
RFP2_DEV bool wait_for(uint64_t *bar, uint32_t parity) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        uint32_t ok;  // sleeps for up to 20 us at a time: probes would take the decoders' issue slots
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
    }
    return mbar_wait(bar, parity);
}

// The 16 weights of a half block (code word c) to eight words of two bf16 values, exactly: level / 2 is one of
// +-2 and +-0.5, whose low bytes are 0, and its product with twice the scale (`twice`, in both halves of a word)
// has four significant bits.  Codes are spread to a nibble each, so that one byte permute finds the high bytes
// of four neighbours and another puts two of them in place; spreads and products run beside those on the FMA
// pipe.  (Decoding is what a narrow tile's step takes: 40 integer instructions a half before, 20 now.)
RFP2_DEV void decode_half(uint32_t c, uint32_t twice, uint32_t (&o)[8]) {
    constexpr uint32_t kHigh = 0x403FBFC0u;  // high bytes of -2, -0.5, 0.5, 2
    const __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162 *>(&twice);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t y = prmt(c, 0u, h ? 0x4342 : 0x4140);  // four codes in the low byte of each half word
        y += 15u * (y & 0x00F000F0u);
        y += 3u * (y & 0x0C0C0C0Cu);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t high = prmt(kHigh, 0u, q ? y >> 16 : y);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t pair = prmt(high, 0u, p ? 0x3424 : 0x1404);
                const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&pair), t);
                o[4 * h + 2 * q + p] = *reinterpret_cast<const uint32_t *>(&v);
            }
        }
    }
}
// Twice the scale of a UE4M3 byte in both halves of a word: its bits at a bf16's exponent and top of mantissa
// are the scale times 2^-119 (a subnormal for E = 0), and all products are exact.
RFP2_DEV uint32_t twice_scale(uint32_t byte) {
    const uint32_t bits = byte * 0x00100010u, up = 0x7B807B80u;  // 2^120
    const __nv_bfloat162 v =
        __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&bits), *reinterpret_cast<const __nv_bfloat162 *>(&up));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A unit of work of a CTA pair: a tile of tokens and a block of 256 weight rows.
struct Unit {
    int4 tile;
    int block, width;  // columns of the MMA: the tile's tokens, rounded up to 32
};
RFP2_DEV Unit unit_at(const GemmArgs &a, int u, int blocks) {
    Unit r;
    const int t = u / blocks;
    r.tile = a.plan.tiles[t];
    r.block = u - t * blocks;
    r.width = (r.tile.z + 31) & ~31;
    return r;
}

RFP2_DEV void copy16(uint32_t smem_dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(src) : "memory");
}
RFP2_DEV void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Persistent over CTA pairs (clusters of two): pair p takes units p, p + pairs, ...  The weights are the MMAs'
// A operand, so that a tile has as many columns as it has tokens.  In each CTA
//   warps 0, 23-25 gather their CTA's half of the tile's tokens into the B half of a ring of stages, swizzled,
//                 16 bytes a lane and copy, a step of K a warp at a time;
//   warp 6        streams the packed rows of its 128 weight rows, 256 of K to a box, into a ring of boxes;
//   warps 7-22    decode them exactly to bf16 into the A half of the stages, a row a thread;
//   warp 1        (even CTA) issues M = 256 pair MMAs over both CTAs' stages; (odd CTA) writes the rows of pairs
//                 without an expert;
//   warps 2-5     read one of two accumulators back while the MMAs fill the other: a lane has a weight row, a
//                 register a token.
// Gated: lanes 0-15 of a warp have gate rows, lanes 16-31 the up rows that go with them, and a shuffle brings
// the two together.  Every wait is bounded; tensor memory is always freed.
template <int ACT, int TILE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap wmap, const GemmArgs a, int32_t *status) {
    constexpr bool kGated = ACT != RFP2_ACT_NONE;
    constexpr int kStages = Cfg<TILE>::kStages, kStageBytes = Cfg<TILE>::kStageBytes, kLoads = Cfg<TILE>::kLoads;
    constexpr int kOut = kGated ? kRows / 2 : kRows;  // outputs of a CTA's rows
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = smem + Cfg<TILE>::kRingOff;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Cfg<TILE>::kBarOff);  // (even CTA) a stage of both CTAs is there
    uint64_t *empty = full + kStages;       // its MMAs are done
    uint64_t *accf = empty + kStages;       // [2] an accumulator is complete
    uint64_t *acce = accf + 2;              // [2] (even CTA) it has been read back
    uint64_t *pfull = acce + 2;             // a box is there
    uint64_t *pempty = pfull + kBoxes;      // it has been decoded
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(pempty + kBoxes);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int nk = a.K / kStep;

    if (threadIdx.x == 0) {
        prefetch_tensor_map(&wmap);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2 * (1 + kGroupWarps));  // both CTAs' tokens and decoders
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], 8);
        }
        for (int s = 0; s < kBoxes; ++s) {
            mbar_init(&pfull[s], 1);
            mbar_init(&pempty[s], kDecodeWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    pdl_wait();  // the plan comes from the launch before, X and W perhaps from earlier ones
    const int blocks = (a.out + 2 * kOut - 1) / (2 * kOut);
    const int units = a.plan.header[0] * blocks;

    const auto goes_on = [&](bool there) { return warp_goes_on(there, abort_flag, status); };

    if (warp == 0 || warp >= 7 + kDecodeWarps) {
        // ---- gathers: lane l copies chunk l % 8 of rows l / 8, l / 8 + 4, ...  Each warp waits for its own copies
        // before it hands the stage over; the other three have theirs on their way meanwhile.
        const int wl = warp == 0 ? 0 : warp - 6 - kDecodeWarps, at = lane >> 3;
        const uint32_t base = smem_addr(smem) + kABytes + at * 128;
        const uint32_t even = base + (((lane & 7) ^ at) << 4), odd = base + (((lane & 7) ^ (at + 4)) << 4);  // rows % 8
        const uint32_t full0 = cluster_map(&full[0], 0), pitch = (uint32_t)a.K * 2;
        int gbase = 0;
        bool ok = true;
        for (int u = pair; u < units && ok; u += npairs, gbase += nk) {
            const Unit un = unit_at(a, u, blocks);
            const int half = un.width / 2;
            int row[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                // columns past the tile's tokens repeat its last
                const int c = min((int)rank * half + 4 * i + at, un.tile.z - 1);
                if (4 * i < half) row[i] = a.plan.pairs[un.tile.y + c];
            }
            if (!a.each)
#pragma unroll
                for (int i = 0; i < kLoads; ++i) row[i] = (int)a.by_top_k(row[i]);
            for (int kb = wl; kb < nk; kb += kLoadWarps) {
                const int g = gbase + kb, s = g % kStages;
                if (!goes_on(!*abort_flag && (g < kStages || wait_for(&empty[s], ((g / kStages) - 1) & 1)))) {
                    ok = false;
                    break;
                }
                // (few instructions a copy, and none for the rows that a narrow tile lacks: the decoders keep the
                // schedulers busy)
                const uint8_t *x = reinterpret_cast<const uint8_t *>(a.X + kb * kStep + (lane & 7) * 8);
                const uint32_t to0 = even + s * kStageBytes, to1 = odd + s * kStageBytes;
#pragma unroll
                for (int j = 0; j < kLoads; j += 4) {
                    if (4 * j >= half) break;  // half is a multiple of 16 rows
#pragma unroll
                    for (int i = j; i < j + 4; ++i)
                        copy16((i & 1 ? to1 : to0) + i * 512, x + (uint64_t)(uint32_t)row[i] * pitch);
                }
                copies_wait();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(full0 + 8u * s);
            }
        }
    } else if (warp == 1 && rank == 0) {
        // ---- MMAs: the whole warp waits, one lane issues (operands stay warp-uniform)
        // The warp's own instructions are on the critical path: the next stage is looked at while this one's MMAs are
        // issued, and nothing but a vote stands between a stage that is there and its MMAs.
        int it = 0, s = 0;
        uint32_t phase = 0;
        bool ok = true, ready = false;
        int width = pair < units ? unit_at(a, pair, blocks).width : 0;
        const uint64_t adesc0 = smem_desc_sw128(smem_addr(smem)), bdesc0 = smem_desc_sw128(smem_addr(smem) + kABytes);
        for (int u = pair; u < units && ok; u += npairs, ++it) {
            const int b = it & 1;
            if (!goes_on(!*abort_flag && (it < 2 || wait_for(&acce[b], ((it >> 1) - 1) & 1)))) break;
            tc_fence_after();
            const uint32_t idesc = idesc_bf16_f32(2 * kRows, width);
            const uint32_t d = tmem + (uint32_t)(b * kTileTokens);
            if (u + npairs < units) width = unit_at(a, u + npairs, blocks).width;
            for (int kb = 0; kb < nk; ++kb) {
                if (!__all_sync(0xffffffffu, ready)) {
                    if (!goes_on(!*abort_flag && wait_for(&full[s], phase))) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_after();
                const int s1 = s + 1 == kStages ? 0 : s + 1;
                const uint32_t phase1 = s1 ? phase : phase ^ 1;
                ready = mbar_test(&full[s1], phase1);
                if (elect_one()) {
                    const uint64_t at = (uint64_t)((s * kStageBytes) >> 4);
#pragma unroll
                    for (int k = 0; k < kStep / kUmmaK; ++k)
                        umma_bf16_pair(d, adesc0 + at + 2 * k, bdesc0 + at + 2 * k, idesc, (kb > 0 || k > 0) ? 1u : 0u);
                    umma_commit_pair_both(&empty[s]);
                }
                s = s1;
                phase = phase1;
            }
            if (elect_one()) umma_commit_pair_both(&accf[b]);  // complete, or idle after an abort
            __syncwarp();
        }
    } else if (warp == 1) {
        fill_rest(a, pair, npairs);  // (the odd CTA has no MMAs to issue)
    } else if (warp >= 2 && warp < 6) {
        // ---- epilogue
        const int q = warp & 3;  // lanes 32 q ... of the accumulators
        const uint32_t acce0 = cluster_map(&acce[0], 0);
        int it = 0;
        for (int u = pair; u < units; u += npairs, ++it) {
            const int b = it & 1;
            const Unit un = unit_at(a, u, blocks);
            const int m = (2 * un.block + (int)rank) * kOut + (kGated ? q * 16 + (lane & 15) : q * 32 + lane);
            float bias = 0.0f;
            if (a.bias && m < a.out) bias = a.bias[(int64_t)un.tile.x * a.M + m + (kGated && lane >= 16 ? a.out : 0)];
            if (!goes_on(!*abort_flag && wait_for(&accf[b], (it >> 1) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < un.width; c0 += 32) {
                uint32_t r[32];
                tmem_ld_32cols(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(b * kTileTokens + c0), r);
                const int mine = a.plan.pairs[un.tile.y + min(c0 + lane, un.tile.z - 1)];
                tmem_ld_wait();
                const int n = un.tile.z - c0;
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    if constexpr (kGated) {
                        // lanes 0-15 finish column c, lanes 16-31 column c + 1
                        const bool low = lane < 16;
                        const float own = __uint_as_float(low ? r[c] : r[c + 1]) + bias;
                        const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(low ? r[c + 1] : r[c]) + bias, 16);
                        const int p = __shfl_sync(0xffffffffu, mine, c + (lane >> 4));
                        const float y = activated(ACT, low ? own : other, low ? other : own);
                        if (c + (lane >> 4) < n && m < a.out) a.Y[(int64_t)p * a.out + m] = __float2bfloat16(y);
                    } else {
                        // even lanes take two rows of column c, odd lanes of column c + 1
                        const bool odd = lane & 1;
                        const float own = __uint_as_float(odd ? r[c + 1] : r[c]) + bias;
                        const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(odd ? r[c] : r[c + 1]) + bias, 1);
                        const int p = __shfl_sync(0xffffffffu, mine, c + odd);
                        const __nv_bfloat162 y = __floats2bfloat162_rn(odd ? other : own, odd ? own : other);
                        if (c + odd < n && m < a.out)  // out is even, so both rows are there or neither
                            *reinterpret_cast<__nv_bfloat162 *>(a.Y + (int64_t)p * a.out + (m & ~1)) = y;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acce0 + 8u * b);
        }
    } else if (warp == 6 && lane == 0) {
        // ---- packed boxes, in the decoders' order; gated: 64 gate rows, then 64 up rows
        int n = 0;
        bool ok = true;
        for (int u = pair; u < units && ok; u += npairs) {
            const Unit un = unit_at(a, u, blocks);
            const int row = un.tile.x * a.M + (2 * un.block + (int)rank) * kOut;
            for (int kq = 0; kq < nk / 4; ++kq, ++n) {
                const int s = n % kBoxes;
                if (*abort_flag || (n >= kBoxes && !wait_for(&pempty[s], ((n / kBoxes) - 1) & 1))) {
                    record_status(status, RFP2_ETIMEOUT);
                    *abort_flag = 1;
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&pfull[s], kBoxBytes);
                uint8_t *to = ring + (size_t)s * kBoxBytes;
                tma_load_2d(to, &wmap, kq * kBoxRowBytes, row, &pfull[s]);
                tma_load_2d(to + kBoxBytes / 2, &wmap, kq * kBoxRowBytes, row + (kGated ? a.out : kRows / 2), &pfull[s]);
            }
        }
        for (int i = max(0, n - kBoxes); i < n; ++i)  // none in flight when the CTA retires
            if (!wait_for(&pfull[i % kBoxes], (i / kBoxes) & 1)) record_status(status, RFP2_ETIMEOUT);
    } else if (warp >= 7 && warp < 7 + kDecodeWarps) {
        // ---- decoders: two blocks of a row at byte 20 gi of its 80-byte box row, in a window of 32 bytes
        const int gi = (warp - 7) / kGroupWarps;
        const int quarter = (warp - 7) % kGroupWarps;
        const int row = quarter * 32 + lane;  // of the A operand
        const int from = kGated ? (lane < 16 ? quarter * 16 + lane : 64 + quarter * 16 + lane - 16) : row;  // of the box
        const int wq = (20 * gi & 15) >> 2;
        const uint32_t full0 = cluster_map(&full[0], 0);
        int gbase = 0, nd = 0;
        bool ok = true;
        for (int u = pair; u < units && ok; u += npairs, gbase += nk) {
            for (int kb = gi; kb < nk; kb += kGroups, ++nd) {
                const int gd = gbase + kb, s = gd % kStages, ps = nd % kBoxes;
                bool there = !*abort_flag && wait_for(&pfull[ps], (nd / kBoxes) & 1);
                // decoded before the wait for a free stage, so that only the stores come after it
                uint32_t o[4][8];
                if (there) {
                    const uint4 *win = reinterpret_cast<const uint4 *>(ring + (size_t)ps * kBoxBytes + from * kBoxRowBytes + ((20 * gi) & ~15));
                    const uint4 q0 = win[0], q1 = win[1];
                    const uint32_t wv[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
                    uint32_t w[5];
#pragma unroll
                    for (int i = 0; i < 5; ++i)
                        w[i] = wq == 0 ? wv[i] : wq == 1 ? wv[i + 1] : wq == 2 ? wv[i + 2] : wv[i + 3];
                    // block 0: codes w0, w1, scales in the low half of w2; block 1: from byte 10
                    const uint32_t code[4] = {w[0], w[1], __funnelshift_r(w[2], w[3], 16), __funnelshift_r(w[3], w[4], 16)};
                    const uint32_t scales[4] = {w[2] & 0xFFu, w[2] >> 8 & 0xFFu, w[4] >> 16 & 0xFFu, w[4] >> 24};
#pragma unroll
                    for (int h = 0; h < 4; ++h) decode_half(code[h], twice_scale(scales[h]), o[h]);
                }
                if (gd >= kStages) there = there && wait_for(&empty[s], ((gd / kStages) - 1) & 1);
                if (!goes_on(there)) {
                    ok = false;
                    break;
                }
                uint8_t *to = smem + (size_t)s * kStageBytes + row * 128;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    *reinterpret_cast<uint4 *>(to + (((2 * h) ^ (row & 7)) << 4)) = make_uint4(o[h][0], o[h][1], o[h][2], o[h][3]);
                    *reinterpret_cast<uint4 *>(to + (((2 * h + 1) ^ (row & 7)) << 4)) = make_uint4(o[h][4], o[h][5], o[h][6], o[h][7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_remote(full0 + 8u * s);
                    mbar_arrive(&pempty[ps]);
                }
            }
        }
    }
    if (warp == 0 && lane == 0) {
        // Neither CTA leaves before the commits of the last stages have arrived here.
        const int n = (units - pair + npairs - 1) / npairs * nk;
        for (int i = max(0, n - kStages); i < n; ++i)
            if (!wait_for(&empty[i % kStages], (i / kStages) & 1)) record_status(status, RFP2_ETIMEOUT);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

using ProductFn = void (*)(CUtensorMap, GemmArgs, int32_t *);

struct Product {
    ProductFn fn;
    size_t smem;
};
template <int TILE>
Product product_of(int activation) {
    return {activation == RFP2_ACT_NONE   ? product_kernel<RFP2_ACT_NONE, TILE>
            : activation == RFP2_ACT_SILU ? product_kernel<RFP2_ACT_SILU, TILE>
                                          : product_kernel<RFP2_ACT_GELU, TILE>,
            Cfg<TILE>::kSmemBytes};
}
Product product_of(int activation, int tile) {
    return tile == 64 ? product_of<64>(activation) : tile == 128 ? product_of<128>(activation) : product_of<256>(activation);
}

// Tokens of a tile at most: an expert that has more has its weights decoded again, so the mean (of P pairs over E
// experts) fits in once or twice.  Against tiles of up to 256 for all: 16 tokens to 8 of 256 experts 39.5 -> 38.4
// us, 2047 tokens 281 -> 277.
int tile_of(int64_t P, int64_t E) { return P <= 32 * E ? 64 : P <= 64 * E ? 128 : 256; }

// Sets the kernels up on a device; returns how many pairs it holds at a time (0: an error).
int pairs_of(int dev) {
    static std::mutex mu;
    static int held[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 64 && held[dev]) return held[dev];
    int pairs = 0;
    if (set_smem_limit(plan_kernel, 32 * (kMaxExperts + 1) * 4) != cudaSuccess) return 0;
    for (int i = 0; i < 9; ++i) {
        const Product p = product_of(i % 3, 64 << i / 3);
        if (set_smem_limit(p.fn, (int)p.smem) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = p.smem;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void *>(p.fn), &cfg) != cudaSuccess || n <= 0) return 0;
        pairs = pairs ? std::min(pairs, n) : n;
    }
    if (dev < 64) held[dev] = pairs;
    return pairs;
}

}  // namespace
}  // namespace rfp2

using namespace rfp2;

extern "C" size_t rfp2_moe_gemm_workspace_bytes(int64_t T, int64_t top_k, int64_t E) {
    if (T <= 0 || top_k <= 0 || E <= 0 || T > kMaxPairs / top_k) return 0;
    return plan_bytes(T * top_k, E);
}

extern "C" rfp2_status rfp2_moe_gemm(const uint8_t *W, int64_t E, int64_t M, int64_t K, const int32_t *ids, int64_t T,
                                     int64_t top_k, const uint16_t *X, int each, const float *bias, int activation,
                                     uint16_t *Y, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                     rfp2_stream_t stream) {
    if (T < 0 || activation < RFP2_ACT_NONE || activation > RFP2_ACT_GELU) return RFP2_EINVAL;
    if (E < 1 || E > kMaxExperts || M < 1 || K < 1 || top_k < 1 || T > kMaxPairs / top_k || M > (1 << 30) || E * M > (1 << 30) ||
        K > (1 << 20) || T * top_k > (1ll << 40) / M)
        return RFP2_ESHAPE;
    const bool gated = activation != RFP2_ACT_NONE;
    if (K % 256 != 0 || M % (gated ? 32 : 16) != 0) return RFP2_EUNSUPPORTED;
    if (T == 0) return RFP2_OK;
    if (!W || !ids || !X || !Y) return RFP2_EINVAL;
    const int64_t P = T * top_k;
    if (!workspace || workspace_bytes < plan_bytes(P, E)) return RFP2_EWORKSPACE;
    if (!aligned(W, 16) || !aligned(ids, 4) || !aligned(X, 16) || !aligned(bias, 4) || !aligned(Y, 16) ||
        !aligned(workspace, 256))
        return RFP2_EALIGN;
    const int64_t out = gated ? M / 2 : M;
    const Rows in[] = {{W, 1, E * M * (K / 32) * 10, 0}, {ids, 1, P * 4, 0}, {X, 1, (each ? P : T) * K * 2, 0}, {bias, 1, E * M * 4, 0}};
    const Rows y(Y, 1, P * out * 2, 0), ws(workspace, 1, (int64_t)plan_bytes(P, E), 0);
    bool meet = y.meet(ws);
    for (const Rows &r : in) meet |= r.meet(y) || r.meet(ws);
    if (meet) return RFP2_EINVAL;
    const int pairs = pairs_of(current_device());
    CUtensorMap wmap;
    const uint64_t row_bytes = (uint64_t)(K / 32) * 10;
    if (pairs <= 0 ||
        !encode_tensor_map_2d(&wmap, W, CU_TENSOR_MAP_DATA_TYPE_UINT8, row_bytes, (uint64_t)(E * M), row_bytes, kBoxRowBytes,
                              kRows / 2, CU_TENSOR_MAP_SWIZZLE_NONE))
        return RFP2_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    GemmArgs a;
    a.X = reinterpret_cast<const __nv_bfloat16 *>(X);
    a.bias = bias;
    a.Y = reinterpret_cast<__nv_bfloat16 *>(Y);
    a.ids = ids;
    a.plan = carve_plan(workspace, P);
    a.M = (int)M;
    a.K = (int)K;
    a.by_top_k = FastDiv((uint32_t)top_k);
    a.each = each;
    a.out = (int)out;
    const int tile = tile_of(P, E), warps = (int)std::min<int64_t>(32, (P + 31) / 32);
    cudaError_t e = launch(plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)warps * (E + 1) * 4, s, true, ids, (int)P,
                           (int)E, warps, tile, a.plan, dev_status);
    if (e != cudaSuccess) return RFP2_ECUDA;
    // at most a pair for every unit there can be
    const int64_t blocks = (out + (gated ? kRows : 2 * kRows) - 1) / (gated ? kRows : 2 * kRows);
    const dim3 grid((unsigned)(2 * std::min<int64_t>(pairs, most_tiles(P, E) * blocks)));
    const Product k = product_of(activation, tile);
    return from_cuda(launch(k.fn, grid, dim3(kThreads), k.smem, s, true, wmap, a, dev_status));
}
