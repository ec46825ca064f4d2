// The routed experts' products for any number of tokens:
//   z = W[e] x + bias[e];  y = z, or act(z[gate rows]) * z[up rows];  a row of y for each (token, slot) pair.
//
// Two launches:
//  1. plan (one CTA): the pairs sorted by expert, and each expert's run cut into tiles of tokens.
//  2. the product: units of (tile, block of weight rows).
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "expand.cuh"
#include "rfp2_decode.cuh"

namespace rfp2 {
namespace {

constexpr int kTileTokens = 256;
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
int64_t most_tiles(int64_t P, int64_t E) { return P / kTileTokens + std::min(P, E); }
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
// places, and each warp puts its stretch there: every pair's place is a function of the ids alone.
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const int32_t *__restrict__ ids, int P, int E, int warps,
                                                               Plan plan, int32_t *status) {
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
    const auto bin_of = [&](int p) {
        const int e = ids[p];
        return e >= 0 && e < E ? e : E;
    };
    for (int p0 = from; p0 < to; p0 += 32) {
        const int p = p0 + lane;
        const int b = p < to ? bin_of(p) : -1;
        if (b == E && ids[p] != -1) record_status(status, RFP2_EBADID);
        const unsigned same = __match_any_sync(0xffffffffu, b);
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    // thread e: the places of expert e's pairs and tiles
    int n = 0;
    if (tid < E)
        for (int w = 0; w < warps; ++w) n += count[w * bins + tid];
    const int tiles = (n + kTileTokens - 1) / kTileTokens;
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
    for (int p0 = from; p0 < to; p0 += 32) {
        const int p = p0 + lane;
        const int b = p < to ? bin_of(p) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, b);
        if (b >= 0) plan.pairs[mine[b] + __popc(same & ((1u << lane) - 1))] = p;
        __syncwarp();
        if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
        __syncwarp();
    }
}

struct GemmArgs {
    const uint8_t *W;
    const __nv_bfloat16 *X;
    const float *bias;
    __nv_bfloat16 *Y;
    const int32_t *ids;
    Plan plan;
    int E, M, K, top_k, each, activation, out;
};

RFP2_DEV float activated(int activation, float gate, float up) {
    if (activation == RFP2_ACT_SILU) return gate / (1.0f + expf(-gate)) * up;
    const float t = tanhf(0.7978845608028654f * fmaf(0.044715f * gate * gate, gate, gate));
    return 0.5f * gate * (1.0f + t) * up;
}

// The rows of pairs without an expert: zeros for -1, NaN for another id.
RFP2_DEV void fill_rest(const GemmArgs &a, int64_t thread, int64_t threads) {
    const int first = a.plan.header[1], rest = a.plan.header[2] - first;
    for (int64_t i = thread; i < (int64_t)rest * a.out; i += threads) {
        const int p = a.plan.pairs[first + i / a.out];
        a.Y[(int64_t)p * a.out + i % a.out] = __float2bfloat16(a.ids[p] == -1 ? 0.0f : CUDART_NAN_F);
    }
}

// The plain form on CUDA cores: 32 output columns x 32 tokens of a tile at a time, 64 of K per step.
constexpr int kRows = 32, kCols = 32, kStep = 64, kThreads = 256;

__global__ void __launch_bounds__(kThreads) product_kernel(const GemmArgs a) {
    __shared__ float w[2][kRows][kStep + 1], x[kCols][kStep + 1];
    pdl_wait();
    pdl_launch_dependents();
    fill_rest(a, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
    const int ntiles = a.plan.header[0], blocks = (a.out + kRows - 1) / kRows;
    const int parts = a.activation == RFP2_ACT_NONE ? 1 : 2;
    const int row = threadIdx.x >> 3, col0 = (threadIdx.x & 7) * 4;
    for (int64_t u = blockIdx.x; u < (int64_t)ntiles * blocks; u += gridDim.x) {
        const int4 tile = a.plan.tiles[u / blocks];
        const int row0 = (int)(u % blocks) * kRows;
        for (int c0 = 0; c0 < tile.z; c0 += kCols) {
            float sum[2][4] = {};
            for (int k0 = 0; k0 < a.K; k0 += kStep) {
                for (int i = threadIdx.x; i < kCols * kStep; i += kThreads) {
                    const int c = i / kStep, k = i % kStep;
                    float v = 0.0f;
                    if (c0 + c < tile.z) {
                        const int p = a.plan.pairs[tile.y + c0 + c];
                        v = __bfloat162float(a.X[(int64_t)(a.each ? p : p / a.top_k) * a.K + k0 + k]);
                    }
                    x[c][k] = v;
                }
                for (int i = threadIdx.x; i < parts * kRows * (kStep / 16); i += kThreads) {
                    const int h = i % (kStep / 16), r = i / (kStep / 16) % kRows, part = i / (kStep / 16) / kRows;
                    const int m = row0 + r;
                    const int half = k0 / 16 + h;
                    const uint8_t *b = a.W + ((int64_t)tile.x * a.M + part * a.out + m) * (a.K / 32 * 10) + half / 2 * 10;
                    for (int j = 0; j < 16; ++j) {
                        float v = 0.0f;
                        if (m < a.out) {
                            float s0, s1;
                            decode_scale_pair(b[8] | b[9] << 8, s0, s1);
                            const int c = b[(half & 1) * 4 + j / 4] >> (2 * (j % 4)) & 3;
                            v = (half & 1 ? s1 : s0) * (c == 0 ? -4.0f : c == 1 ? -1.0f : c == 2 ? 1.0f : 4.0f);
                        }
                        w[part][r][h * 16 + j] = v;
                    }
                }
                __syncthreads();
                for (int k = 0; k < kStep; ++k)
                    for (int part = 0; part < parts; ++part)
#pragma unroll
                        for (int c = 0; c < 4; ++c) sum[part][c] = fmaf(w[part][row][k], x[col0 + c][k], sum[part][c]);
                __syncthreads();
            }
            const int m = row0 + row;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c0 + col0 + c >= tile.z || m >= a.out) continue;
                const float *bias = a.bias ? a.bias + (int64_t)tile.x * a.M + m : nullptr;
                float z = sum[0][c] + (bias ? bias[0] : 0.0f);
                if (parts == 2) z = activated(a.activation, z, sum[1][c] + (bias ? bias[a.out] : 0.0f));
                a.Y[(int64_t)a.plan.pairs[tile.y + c0 + col0 + c] * a.out + m] = __float2bfloat16(z);
            }
        }
    }
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
    if (E < 1 || E > kMaxExperts || M < 1 || K < 1 || top_k < 1 || T > kMaxPairs / top_k || E * M > (1 << 30) ||
        M > (1 << 30) || K > (1 << 20))
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
    static std::mutex mu;
    static bool configured[64] = {};
    const int dev = current_device();
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev >= 64 || !configured[dev]) {
            if (set_smem_limit(plan_kernel, 32 * (kMaxExperts + 1) * 4) != cudaSuccess) return RFP2_ECUDA;
            if (dev < 64) configured[dev] = true;
        }
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    GemmArgs a;
    a.W = W;
    a.X = reinterpret_cast<const __nv_bfloat16 *>(X);
    a.bias = bias;
    a.Y = reinterpret_cast<__nv_bfloat16 *>(Y);
    a.ids = ids;
    a.plan = carve_plan(workspace, P);
    a.E = (int)E;
    a.M = (int)M;
    a.K = (int)K;
    a.top_k = (int)top_k;
    a.each = each;
    a.activation = activation;
    a.out = (int)out;
    const int warps = (int)std::min<int64_t>(32, (P + 31) / 32);
    cudaError_t e = launch(plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)warps * (E + 1) * 4, s, true, ids, (int)P,
                           (int)E, warps, a.plan, dev_status);
    if (e != cudaSuccess) return RFP2_ECUDA;
    return from_cuda(launch(product_kernel, dim3(4 * sm_count(dev)), dim3(kThreads), 0, s, true, a));
}
