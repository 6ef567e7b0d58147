// kvq_mass.cu -- C entry points of the attention mass: the weight that each
// cached token gets in attention, summed over heads and query tokens.
#include "kvq_mass.cuh"

namespace kvq {
namespace {

constexpr int64_t kMaxLen = int64_t(1) << 30;  // cached tokens of a sequence
constexpr int64_t kMaxTree = 1024;             // drafted tokens of a sequence, as in kvq_tree_mask

// Bytes of `rows` rows of `width` floats.
int64_t span(int64_t rows, int64_t width, int64_t stride) { return rows > 0 ? ((rows - 1) * stride + width) * 4 : 0; }

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_mass_workspace(int64_t n_seq, int64_t rows, int64_t max_len) {
    if (n_seq <= 0 || rows <= 0 || max_len <= 0 || mass_tiles(rows) == 1) return 0;
    return size_t(n_seq) * size_t(mass_tiles(rows)) * size_t(mass_part_stride(max_len)) * sizeof(float);
}

extern "C" kvq_status kvq_attend_mass(kvq_layout layout, int page_bits, const void *q_bf16, int64_t q_token_stride,
                                      int64_t q_head_stride, int64_t n_seq, int64_t q_len, int64_t heads, const float *lse,
                                      const uint8_t *pool, int64_t pool_pages, const int32_t *page_table,
                                      int64_t table_rows, int64_t table_width, int64_t table_stride, const int32_t *req,
                                      const int32_t *kv_len, const uint64_t *mask, float scale, float *mass, int64_t mass_row_count,
                                      int64_t mass_width, int64_t mass_row_stride, const int32_t *rows, const float *prev,
                                      int64_t prev_row_stride, float decay, void *workspace, size_t workspace_bytes,
                                      int32_t *err, struct CUstream_st *stream) {
    if (layout != KVQ_LAYOUT_V41 && layout != KVQ_LAYOUT_V41_FP4) return KVQ_ERR_INVALID_ARG;
    if (page_bits < 1 || page_bits > 16) return KVQ_ERR_INVALID_ARG;
    if (!page_bits_supported(page_bits)) return KVQ_ERR_UNSUPPORTED;
    if (n_seq < 0 || q_len < 1 || heads < 1 || mass_row_count < 0 || mass_width < 0) return KVQ_ERR_INVALID_ARG;
    if (q_len > (int64_t(1) << 20) || heads > (int64_t(1) << 10) || n_seq > 0xFFFF || n_seq * q_len > (int64_t(1) << 24))
        return KVQ_ERR_UNSUPPORTED;
    if (mask && q_len > kMaxTree) return KVQ_ERR_UNSUPPORTED;
    if (!aligned(mask, 8)) return KVQ_ERR_INVALID_ARG;
    if (!(scale - scale == 0.f) || (prev && !(decay - decay == 0.f))) return KVQ_ERR_INVALID_ARG;  // NaN or infinite
    if (!pool || !aligned(pool, 16) || pool_pages <= 0) return KVQ_ERR_INVALID_ARG;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if (table_rows < 0 || table_width < 0 || table_stride < table_width) return KVQ_ERR_INVALID_ARG;
    if (n_seq == 0) return KVQ_OK;
    if (!q_bf16 || !aligned(q_bf16, 16) || !lse || !aligned(lse, 4)) return KVQ_ERR_INVALID_ARG;
    if (n_seq * q_len > 1 && (q_token_stride < 0 || q_token_stride % 8)) return KVQ_ERR_INVALID_ARG;
    if (heads > 1 && (q_head_stride < 0 || q_head_stride % 8)) return KVQ_ERR_INVALID_ARG;
    if (table_rows > 0 && table_width > 0 && !page_table) return KVQ_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || (req && !aligned(req, 4)) || (rows && !aligned(rows, 4))) return KVQ_ERR_INVALID_ARG;
    if (!kv_len || !aligned(kv_len, 4)) return KVQ_ERR_INVALID_ARG;
    if ((!req && n_seq > table_rows) || (!rows && n_seq > mass_row_count)) return KVQ_ERR_INVALID_ARG;
    if (mass_row_count > 0 && mass_width > 0 && !mass) return KVQ_ERR_INVALID_ARG;
    if (!aligned(mass, 4) || !aligned(prev, 4)) return KVQ_ERR_INVALID_ARG;
    if (mass_row_count > 1 && (mass_row_stride < mass_width || (prev && prev_row_stride < mass_width))) return KVQ_ERR_INVALID_ARG;
    if (prev && !(prev == mass && (mass_row_count <= 1 || prev_row_stride == mass_row_stride))) {
        const uintptr_t m = reinterpret_cast<uintptr_t>(mass), p = reinterpret_cast<uintptr_t>(prev);
        if (m < p + uintptr_t(span(mass_row_count, mass_width, prev_row_stride)) &&
            p < m + uintptr_t(span(mass_row_count, mass_width, mass_row_stride)))
            return KVQ_ERR_INVALID_ARG;
    }
    // no sequence is longer than kMaxLen, the table's row or the weights' row
    if (table_width > (kMaxLen >> page_bits)) table_width = kMaxLen >> page_bits;
    int64_t max_len = table_width << page_bits;
    if (mass_width < max_len) max_len = mass_width;
    const size_t need = kvq_mass_workspace(n_seq, q_len * heads, max_len);
    if (need && (!workspace || !aligned(workspace, 16) || workspace_bytes < need)) return KVQ_ERR_INVALID_ARG;

    MassArgs a = {};
    a.q = static_cast<const uint16_t *>(q_bf16);
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.n_seq = n_seq;
    a.q_len = int(q_len);
    a.heads = int(heads);
    a.pool = pool;
    a.pool_limit = pool_pages;
    a.page_bits = page_bits;
    a.table = page_table;
    a.table_rows = table_rows;
    a.table_stride = table_stride;
    a.max_len = max_len;
    a.req = req;
    a.kv_len = kv_len;
    a.mask = mask;
    a.mask_words = int((q_len + 63) / 64);
    a.lse = lse;
    a.scale = scale;
    const double c = double(scale) * 1.4426950408889634;
    a.c = float(c);
    a.c_off = float(a.c != 0.f ? c / double(a.c) - 1.0 : 0.0);
    a.mass = mass;
    a.mass_stride = mass_row_stride;
    a.prev = prev;
    a.prev_stride = prev_row_stride;
    a.rows = rows;
    a.n_rows = mass_row_count;
    a.decay = decay;
    a.part = static_cast<float *>(workspace);
    a.part_stride = mass_part_stride(max_len);
    a.err = err;
    a.wait_tries = attend_wait_tries();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return layout == KVQ_LAYOUT_V41 ? launch_mass_v41(a, s) : launch_mass_fp4(a, s);
}
