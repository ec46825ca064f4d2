// Decode attention over the paged Q8 cache: the entry point, its checks and the
// choice of kernel (attn.cuh).
#include <algorithm>

#include "attn.cuh"

using namespace rfp2;

namespace {

// A call's queries: rows of D values, `qb`, `qt` and `qh` values apart.
struct Queries {
    uintptr_t at;
    int64_t B, nq, Hq, D, qb, qt, qh;
    int size;
    bool contiguous() const {
        return (Hq == 1 || qh == D) && (nq == 1 || qt == Hq * D) && (B == 1 || qb == nq * Hq * D);
    }
    // Does any row share memory with [from, from + bytes)?
    bool meet(uintptr_t from, int64_t bytes) const {
        const auto apart = [&](int64_t low, int64_t high) {  // values before the first row, and after
            return (int64_t)(from - at) >= high * size || (int64_t)(from + bytes - at) <= low * size;
        };
        const int64_t b = (B - 1) * qb, t = (nq - 1) * qt, h = (Hq - 1) * qh;
        if (apart(std::min<int64_t>(b, 0) + std::min<int64_t>(t, 0) + std::min<int64_t>(h, 0),
                  std::max<int64_t>(b, 0) + std::max<int64_t>(t, 0) + std::max<int64_t>(h, 0) + D))
            return false;
        // between the rows, perhaps
        for (int64_t i = 0; i < B * nq; ++i)
            for (int64_t j = 0; j < Hq; ++j) {
                const int64_t row = i / nq * qb + i % nq * qt + j * qh;
                if (!apart(row, row + D)) return true;
            }
        return false;
    }
};

}  // namespace

extern "C" size_t rfp2_attn_decode_workspace_bytes(int64_t B, int64_t nq, int64_t Hq,
                                                   int64_t heads, int64_t D) {
    if (B < 1 || nq < 1 || Hq < 1 || heads < 1 || Hq % heads != 0 || D < 32 || D > 256) return 0;
    // partial results: two a CTA and one a warp, of as many columns as a tile may have
    const int NB = (int)(D / 32), NT = nq * (Hq / heads) > 8 ? 2 : 1;
    const size_t ctas = (size_t)sm_count(current_device()) * attn_ctas_per_sm(NB, NT);
    return RFP2_ATTN_ZERO_BYTES + ctas * (2 + attn_warps(NB, NT)) * attn_slot(NB, NT) * 4;
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
        nq > 65536 / Hq || B > (1 << 24) || D < 32 || D > 256 || D % 32 != 0 || pages < 1 ||
        page_size < 1 || page_size >= (1ll << 32) / heads ||
        pages >= (1ll << 32) / (heads * page_size) || table_width < 1 ||
        table_stride < table_width || page_size > (1ll << 30) ||
        table_width > (1ll << 30) / page_size)
        return RFP2_ESHAPE;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !table || !lens || !out)
        return RFP2_EINVAL;
    if (!workspace || workspace_bytes < rfp2_attn_decode_workspace_bytes(B, nq, Hq, heads, D))
        return RFP2_EWORKSPACE;
    if (!aligned(q, size) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(table, 4) ||
        !aligned(lens, 4) || !aligned(k_codes, 16) || !aligned(k_scales, 16) ||
        !aligned(v_codes, 16) || !aligned(v_scales, 16) || !aligned(workspace, 256))
        return RFP2_EALIGN;
    // Each row of q is read before the same row of out is written, and at any time to another's.
    const uintptr_t q_at = reinterpret_cast<uintptr_t>(q), out_at = reinterpret_cast<uintptr_t>(out),
                    lse_at = reinterpret_cast<uintptr_t>(lse);
    const int64_t rows = B * nq * Hq;
    const Queries queries = {q_at, B, nq, Hq, D, q_batch_stride, q_token_stride, q_head_stride, size};
    if (!(q_at == out_at && queries.contiguous()) && queries.meet(out_at, rows * D * size)) return RFP2_EINVAL;
    if (lse && (queries.meet(lse_at, rows * 4) || (lse_at < out_at + rows * D * size && out_at < lse_at + rows * 4)))
        return RFP2_EINVAL;
    AttnArgs a;
    a.qb = q_batch_stride;
    a.qt = q_token_stride;
    a.qh = q_head_stride;
    a.k_codes = k_codes;
    a.k_scales = k_scales;
    a.v_codes = v_codes;
    a.v_scales = v_scales;
    a.pages = pages;
    a.table_stride = table_stride;
    a.capacity = table_width * page_size;
    a.nq = (int)nq;
    a.Hq = (int)Hq;
    a.heads = (int)heads;
    a.group = (int)(Hq / heads);
    a.columns = (int)(nq * a.group);
    const int most = attn_most_columns((int)D, dtype, a.columns);
    a.column_tiles = (a.columns + most - 1) / most;
    a.page_size = (int)page_size;
    a.by_page = FastDiv((uint32_t)page_size);
    a.by_group = FastDiv((uint32_t)a.group);
    a.by_tiles = FastDiv((uint32_t)a.column_tiles);
    a.whole_pages = page_size % kAttnTile == 0;
    a.dtype = dtype;
    const int64_t words = 16 / size;
    a.q_words = aligned(q, 16) && a.qb % words == 0 && a.qt % words == 0 && a.qh % words == 0;
    a.scale = scale;
    // a cap so far off moves no score below 2^48; its reciprocal's products would be subnormal
    a.softcap = softcap < 0x1p60f ? softcap : 0.0f;
    a.window = std::min<int64_t>(window, 1ll << 30);
    a.counters = static_cast<int *>(workspace);
    a.partials = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + RFP2_ATTN_ZERO_BYTES);
    a.status = dev_status;
    constexpr int64_t kLine = (1ll << 31) - 1 - kAttnGap;  // the kernel adds a gap to its places
    const int64_t line = (a.capacity / kAttnTile + 1 + kAttnGap) * a.heads * a.column_tiles;
    if (line > kLine) return RFP2_ESHAPE;
    static const AttnFn kinds[] = {attn_d32,  attn_d64,  attn_d96,  attn_d128,
                                   attn_d160, attn_d192, attn_d224, attn_d256};
    const int sms = std::min(sm_count(current_device()), RFP2_ATTN_ZERO_BYTES / 8);
    // a launch keeps its sequences' places on the line, 32-bit numbers, in shared memory
    for (int64_t b0 = 0; b0 < B; b0 += a.B) {
        a.B = (int)std::min<int64_t>({B - b0, kAttnMaxBatch, kLine / line});
        a.q = static_cast<const uint8_t *>(q) + b0 * q_batch_stride * size;
        a.table = table + b0 * table_stride;
        a.lens = lens + b0;
        a.out = static_cast<uint8_t *>(out) + b0 * nq * Hq * D * size;
        a.lse = lse ? lse + b0 * nq * Hq : nullptr;
        const cudaError_t e = kinds[D / 32 - 1](a, sms, reinterpret_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return RFP2_ECUDA;
    }
    return RFP2_OK;
}
