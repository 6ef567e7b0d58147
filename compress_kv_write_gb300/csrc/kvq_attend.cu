// kvq_attend.cu -- C entry points of the latent attention over the paged V41 /
// V41_FP4 pool, by page table (kvq_attend), with a tree of drafted tokens at its
// end (kvq_attend_tree), or by selected slots (kvq_attend_slots).
#include <atomic>

#include "kvq_attend.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

kvq_status launch_attend(int layout, const AttendArgs &a, bool slots, cudaStream_t s) {
    return layout == KVQ_LAYOUT_V41 ? launch_attend_v41(a, slots, s) : launch_attend_fp4(a, slots, s);
}

// Tries of the waits inside the kernels: 2^20 take some seconds where nothing happens.
constexpr uint32_t kMostWaitTries = 1u << 24;
std::atomic<uint32_t> g_wait_tries{kWaitTries};

constexpr int64_t kMaxTree = 1024;  // drafted tokens of a sequence, as in kvq_tree_mask
constexpr int64_t kMaxLen = int64_t(1) << 30;  // cached tokens of a sequence: positions and block sums fit an int

// What both entry points share: layout, pool, query, output and workspace.
kvq_status check_common(int layout, int page_bits, const void *q, int64_t q_tok, int64_t q_head, int64_t n_seq,
                        int64_t q_len, int64_t heads, const uint8_t *pool, int64_t pool_limit, float scale,
                        const void *out, int out_dtype, int64_t out_tok, int64_t out_head, const float *lse,
                        const void *ws, size_t ws_bytes, const int32_t *err) {
    if (layout != KVQ_LAYOUT_V41 && layout != KVQ_LAYOUT_V41_FP4) return KVQ_ERR_INVALID_ARG;
    if (page_bits < 1 || page_bits > 16) return KVQ_ERR_INVALID_ARG;
    if (!page_bits_supported(page_bits)) return KVQ_ERR_UNSUPPORTED;
    if (out_dtype != KVQ_BF16 && out_dtype != KVQ_F32) return KVQ_ERR_INVALID_ARG;
    if (n_seq < 0 || q_len < 1 || heads < 1) return KVQ_ERR_INVALID_ARG;
    if (q_len > (int64_t(1) << 20) || heads > (int64_t(1) << 10) || n_seq > (int64_t(1) << 24) ||
        n_seq * q_len > (int64_t(1) << 24))
        return KVQ_ERR_UNSUPPORTED;
    if (!(scale - scale == 0.f)) return KVQ_ERR_INVALID_ARG;  // NaN or infinite
    if (!pool || !aligned(pool, 16) || pool_limit <= 0) return KVQ_ERR_INVALID_ARG;
    if (err && !aligned(err, 4)) return KVQ_ERR_INVALID_ARG;
    if (n_seq == 0) return KVQ_OK;
    // the stride of an axis of one element is never used
    const int64_t unit = out_dtype == KVQ_BF16 ? 8 : 4;  // elements of 16 bytes
    if (!q || !aligned(q, 16) || !out || !aligned(out, 16)) return KVQ_ERR_INVALID_ARG;
    if (n_seq * q_len > 1 && (q_tok < 0 || q_tok % 8 || out_tok < kD || out_tok % unit)) return KVQ_ERR_INVALID_ARG;
    if (heads > 1 && (q_head < 0 || q_head % 8 || out_head < kD || out_head % unit)) return KVQ_ERR_INVALID_ARG;
    if (n_seq * q_len > 1 && heads > 1) {  // rows that do not overlap: one stride spans the other axis
        const bool by_token = out_tok >= out_head;
        const int64_t inner = by_token ? out_head : out_tok, outer = by_token ? out_tok : out_head;
        if (outer - kD < inner * ((by_token ? heads : n_seq * q_len) - 1)) return KVQ_ERR_INVALID_ARG;
    }
    if (lse && !aligned(lse, 4)) return KVQ_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < kvq_attend_workspace(q_len * heads)) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

// kvq_attend, and with a mask kvq_attend_tree.
kvq_status attend_pages(int layout, int page_bits, const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                        int64_t n_seq, int64_t q_len, int64_t heads, const uint8_t *pool, int64_t pool_pages,
                        const int32_t *page_table, int64_t table_rows, int64_t table_width, int64_t table_stride,
                        const int32_t *req, const int32_t *kv_len, const uint64_t *mask, bool tree, float scale, void *out,
                        int out_dtype, int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                        size_t workspace_bytes, int32_t *err, cudaStream_t stream) {
    kvq_status st = check_common(layout, page_bits, q_bf16, q_token_stride, q_head_stride, n_seq, q_len, heads, pool,
                                 pool_pages, scale, out, out_dtype, out_token_stride, out_head_stride, lse, workspace,
                                 workspace_bytes, err);
    if (st != KVQ_OK || n_seq == 0) return st;
    if (table_rows < 0 || table_width < 0 || table_stride < table_width) return KVQ_ERR_INVALID_ARG;
    if (table_rows > 0 && table_width > 0 && !page_table) return KVQ_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || (req && !aligned(req, 4))) return KVQ_ERR_INVALID_ARG;
    if (!kv_len || !aligned(kv_len, 4)) return KVQ_ERR_INVALID_ARG;
    if (tree && (!mask || !aligned(mask, 8))) return KVQ_ERR_INVALID_ARG;
    if (!req && n_seq > table_rows) return KVQ_ERR_INVALID_ARG;
    // no sequence is longer than kMaxLen, however wide the table
    if (table_width > (kMaxLen >> page_bits)) table_width = kMaxLen >> page_bits;

    AttendArgs a = {};
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
    a.max_len = table_width << page_bits;
    a.req = req;
    a.kv_len = kv_len;
    a.mask = mask;
    a.mask_words = int((q_len + 63) / 64);
    a.scale = scale;
    a.out = out;
    a.out_tok = out_token_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.ws = static_cast<uint8_t *>(workspace);
    a.err = err;
    a.out_bf16 = out_dtype == KVQ_BF16;
    a.wait_tries = attend_wait_tries();
    if (tree) return layout == KVQ_LAYOUT_V41 ? launch_attend_tree_v41(a, stream) : launch_attend_tree_fp4(a, stream);
    return launch_attend(layout, a, false, stream);
}

}  // namespace

uint32_t attend_wait_tries() { return g_wait_tries.load(std::memory_order_relaxed); }

}  // namespace kvq

using namespace kvq;

extern "C" uint32_t kvq_attend_wait_limit(uint32_t tries) {
    return g_wait_tries.exchange(tries < kMostWaitTries ? tries : kMostWaitTries, std::memory_order_relaxed);
}

extern "C" size_t kvq_attend_workspace(int64_t rows) {
    if (rows <= 0) return 0;
    return kMaxAttendCtas * (sizeof(int2) + 2 * size_t(attend_rows(rows)) * kPartRow * sizeof(float));
}

extern "C" kvq_status kvq_attend(kvq_layout layout, int page_bits, const void *q_bf16, int64_t q_token_stride,
                                 int64_t q_head_stride, int64_t n_seq, int64_t q_len, int64_t heads,
                                 const uint8_t *pool, int64_t pool_pages, const int32_t *page_table,
                                 int64_t table_rows, int64_t table_width, int64_t table_stride, const int32_t *req,
                                 const int32_t *kv_len, float scale, void *out, kvq_dtype out_dtype,
                                 int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                 size_t workspace_bytes, int32_t *err, struct CUstream_st *stream) {
    return attend_pages(layout, page_bits, q_bf16, q_token_stride, q_head_stride, n_seq, q_len, heads, pool, pool_pages,
                        page_table, table_rows, table_width, table_stride, req, kv_len, nullptr, false, scale, out, out_dtype,
                        out_token_stride, out_head_stride, lse, workspace, workspace_bytes, err,
                        reinterpret_cast<cudaStream_t>(stream));
}

extern "C" kvq_status kvq_attend_tree(kvq_layout layout, int page_bits, const void *q_bf16, int64_t q_token_stride,
                                 int64_t q_head_stride, int64_t n_seq, int64_t q_len, int64_t heads,
                                 const uint8_t *pool, int64_t pool_pages, const int32_t *page_table,
                                 int64_t table_rows, int64_t table_width, int64_t table_stride, const int32_t *req,
                                 const int32_t *kv_len, const uint64_t *mask, float scale, void *out, kvq_dtype out_dtype,
                                 int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                 size_t workspace_bytes, int32_t *err, struct CUstream_st *stream) {
    if (q_len > kMaxTree) return KVQ_ERR_UNSUPPORTED;
    return attend_pages(layout, page_bits, q_bf16, q_token_stride, q_head_stride, n_seq, q_len, heads, pool, pool_pages,
                        page_table, table_rows, table_width, table_stride, req, kv_len, mask, true, scale, out, out_dtype,
                        out_token_stride, out_head_stride, lse, workspace, workspace_bytes, err,
                        reinterpret_cast<cudaStream_t>(stream));
}

extern "C" kvq_status kvq_attend_slots(kvq_layout layout, int page_bits, const void *q_bf16, int64_t q_token_stride,
                                       int64_t q_head_stride, int64_t n_tokens, int64_t heads, const uint8_t *pool,
                                       int64_t pool_slots, const void *slots, kvq_index_dtype slot_dtype,
                                       int64_t n_sel, int64_t slots_stride, float scale, void *out,
                                       kvq_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride,
                                       float *lse, void *workspace, size_t workspace_bytes, int32_t *err,
                                       struct CUstream_st *stream) {
    kvq_status st = check_common(layout, page_bits, q_bf16, q_token_stride, q_head_stride, n_tokens, 1, heads, pool,
                                 pool_slots, scale, out, out_dtype, out_token_stride, out_head_stride, lse, workspace,
                                 workspace_bytes, err);
    if (st != KVQ_OK) return st;
    if ((pool_slots & ((int64_t(1) << page_bits) - 1)) != 0) return KVQ_ERR_INVALID_ARG;
    if (slot_dtype != KVQ_I32 && slot_dtype != KVQ_I64) return KVQ_ERR_INVALID_ARG;
    if (n_sel < 0 || slots_stride < 0 || n_sel > kMaxLen) return KVQ_ERR_INVALID_ARG;
    if (n_tokens == 0) return KVQ_OK;
    if (n_sel > 0 && (!slots || !aligned(slots, slot_dtype == KVQ_I64 ? 8 : 4))) return KVQ_ERR_INVALID_ARG;

    AttendArgs a = {};
    a.q = static_cast<const uint16_t *>(q_bf16);
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.n_seq = n_tokens;
    a.q_len = 1;
    a.heads = int(heads);
    a.pool = pool;
    a.pool_limit = pool_slots;
    a.page_bits = page_bits;
    a.max_len = n_sel;
    a.slots = slots;
    a.slots_stride = slots_stride;
    a.scale = scale;
    a.out = out;
    a.out_tok = out_token_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.ws = static_cast<uint8_t *>(workspace);
    a.err = err;
    a.slots64 = slot_dtype == KVQ_I64;
    a.out_bf16 = out_dtype == KVQ_BF16;
    a.wait_tries = attend_wait_tries();
    return launch_attend(layout, a, true, reinterpret_cast<cudaStream_t>(stream));
}
