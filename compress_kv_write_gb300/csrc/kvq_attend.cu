// kvq_attend.cu -- latent attention over the paged V41 / V41_FP4 pool, by
// page table (kvq_attend) or by selected slots (kvq_attend_slots).
//
// One warp per query row.  Lane l owns dims 16l .. 16l+15 (half a quant
// block) of the row, of every decoded token and of the output; a token's score
// is a warp sum, and the softmax is online (running max and sum).
#include <math.h>

#include "kvq_attend.cuh"

namespace kvq {
namespace {

constexpr int kAtWarps = 8;

template <Layout L>
__device__ __forceinline__ void decode16(const uint8_t *pool, int64_t slot, int page_bits, int lane, float (&k)[16]) {
    using T = LayoutTraits<L>;
    const int64_t page = slot >> page_bits, row = slot & ((int64_t(1) << page_bits) - 1);
    const uint8_t *base = pool + page * (int64_t(kTokenBytes<L>) << page_bits);
    const uint8_t *codes = base + row * T::kCodeBytes;
    const uint32_t sb = __ldg(base + (int64_t(T::kCodeBytes) << page_bits) + row * T::kScaleBytes + lane / 2);
    if constexpr (L == Layout::V41) {
        const uint4 c = __ldg(reinterpret_cast<const uint4 *>(codes) + lane);
        const float s = ue8m0_to_f32(sb);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = e4m3x2_to_f32x2((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
            k[2 * i] = f.x * s;
            k[2 * i + 1] = f.y * s;
        }
    } else {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(codes) + lane);
        const float s = e4m3x2_to_f32x2(sb).x;
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = e2m1x2_to_f32x2((w[i / 4] >> (8 * (i & 3))) & 0xFFu);
            k[2 * i] = f.x * s;
            k[2 * i + 1] = f.y * s;
        }
    }
}

template <Layout L, bool kSlots>
__global__ void __launch_bounds__(kAtWarps * 32) attend_row_kernel(const AttendArgs a, bool slots64, bool out_bf16) {
    const int lane = threadIdx.x & 31;
    const int64_t row = int64_t(blockIdx.x) * kAtWarps + (threadIdx.x >> 5);
    const int64_t per = int64_t(a.q_len) * a.heads;
    if (row >= a.n_seq * per) return;
    const int64_t seq = row / per;
    const int j = int((row % per) / a.heads), head = int(row % a.heads);
    const int64_t tok = seq * a.q_len + j;
    pdl_wait();

    int64_t visible = a.max_len, trow = seq;
    if constexpr (!kSlots) {
        if (a.req) trow = a.req[seq];
        int64_t len = a.kv_len[seq];
        if (trow < 0 || trow >= a.table_rows) {
            if (lane == 0) raise_err(a.err, KVQ_DEVERR_STATE);
            len = 0;
        } else if (len < 0 || len > a.max_len) {
            if (lane == 0) raise_err(a.err, KVQ_DEVERR_LEN);
            len = 0;
        }
        visible = len - (a.q_len - 1 - j);
    }
    float q[16], acc[16];
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(a.q + tok * a.q_tok + head * a.q_head + lane * 16);
        const uint4 u[2] = {__ldg(p), __ldg(p + 1)};
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            q[2 * i] = bf16_lo(w[i]);
            q[2 * i + 1] = bf16_hi(w[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    const float c = a.scale * kLog2e;
    for (int64_t t = 0; t < visible; ++t) {
        int64_t slot;
        if constexpr (kSlots) {
            slot = slots64 ? static_cast<const int64_t *>(a.slots)[seq * a.slots_stride + t]
                           : int64_t(static_cast<const int32_t *>(a.slots)[seq * a.slots_stride + t]);
            if (slot < 0 || slot >= a.pool_limit) {
                if (slot != -1 && lane == 0) raise_err(a.err, KVQ_DEVERR_SLOT);
                continue;
            }
        } else {
            const int64_t page = a.table[trow * a.table_stride + (t >> a.page_bits)];
            if (page < 0 || page >= a.pool_limit) {
                if (lane == 0) raise_err(a.err, KVQ_DEVERR_PAGE);
                continue;
            }
            slot = (page << a.page_bits) + (t & ((int64_t(1) << a.page_bits) - 1));
        }
        float k[16];
        decode16<L>(a.pool, slot, a.page_bits, lane, k);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s *= c;
        const float mn = fmaxf(m, s);
        const float al = mn == -INFINITY ? 1.f : exp2f(m - mn);
        const float p = mn == -INFINITY ? s * 0.f : exp2f(s - mn);
        l = l * al + p;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = fmaf(p, k[i], acc[i] * al);
        m = mn;
    }
    const float r = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = tok * a.out_tok + head * a.out_head + lane * 16;
    if (out_bf16) {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            o[i] = make_uint4(pack_bf16x2(acc[8 * i] * r, acc[8 * i + 1] * r), pack_bf16x2(acc[8 * i + 2] * r, acc[8 * i + 3] * r),
                              pack_bf16x2(acc[8 * i + 4] * r, acc[8 * i + 5] * r), pack_bf16x2(acc[8 * i + 6] * r, acc[8 * i + 7] * r));
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = make_float4(acc[4 * i] * r, acc[4 * i + 1] * r, acc[4 * i + 2] * r, acc[4 * i + 3] * r);
    }
    if (a.lse && lane == 0) a.lse[tok * a.heads + head] = (m + log2f(l)) * 0.6931471805599453f;
}

template <bool kSlots>
kvq_status launch_attend(int layout, const AttendArgs &a, bool slots64, bool out_bf16, cudaStream_t s) {
    const int64_t rows = a.n_seq * a.q_len * a.heads;
    const int64_t blocks = (rows + kAtWarps - 1) / kAtWarps;
    if (blocks > 0x7FFFFFFF) return KVQ_ERR_INVALID_ARG;
    return with_layout(layout, [&](auto Lc) {
        return launch_pdl(attend_row_kernel<decltype(Lc)::value, kSlots>, dim3(unsigned(blocks)), dim3(kAtWarps * 32),
                          s, a, slots64, out_bf16);
    });
}

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
    if (lse && !aligned(lse, 4)) return KVQ_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 16) || ws_bytes < kvq_attend_workspace(q_len * heads)) return KVQ_ERR_INVALID_ARG;
    return KVQ_OK;
}

}  // namespace
}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_attend_workspace(int64_t rows) { return rows > 0 ? 16 : 0; }

extern "C" kvq_status kvq_attend(kvq_layout layout, int page_bits, const void *q_bf16, int64_t q_token_stride,
                                 int64_t q_head_stride, int64_t n_seq, int64_t q_len, int64_t heads,
                                 const uint8_t *pool, int64_t pool_pages, const int32_t *page_table,
                                 int64_t table_rows, int64_t table_width, int64_t table_stride, const int32_t *req,
                                 const int32_t *kv_len, float scale, void *out, kvq_dtype out_dtype,
                                 int64_t out_token_stride, int64_t out_head_stride, float *lse, void *workspace,
                                 size_t workspace_bytes, int32_t *err, struct CUstream_st *stream) {
    kvq_status st = check_common(layout, page_bits, q_bf16, q_token_stride, q_head_stride, n_seq, q_len, heads, pool,
                                 pool_pages, scale, out, out_dtype, out_token_stride, out_head_stride, lse, workspace,
                                 workspace_bytes, err);
    if (st != KVQ_OK || n_seq == 0) return st;
    if (table_rows < 0 || table_width < 0 || table_stride < table_width) return KVQ_ERR_INVALID_ARG;
    if (table_rows > 0 && table_width > 0 && !page_table) return KVQ_ERR_INVALID_ARG;
    if (!aligned(page_table, 4) || (req && !aligned(req, 4))) return KVQ_ERR_INVALID_ARG;
    if (!kv_len || !aligned(kv_len, 4)) return KVQ_ERR_INVALID_ARG;
    if (!req && n_seq > table_rows) return KVQ_ERR_INVALID_ARG;
    // kv_len is int32: no sequence is longer, however wide the table
    if (table_width > (int64_t(0x7FFFFFFF) >> page_bits)) table_width = int64_t(0x7FFFFFFF) >> page_bits;

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
    a.scale = scale;
    a.out = out;
    a.out_tok = out_token_stride;
    a.out_head = out_head_stride;
    a.lse = lse;
    a.ws = static_cast<uint8_t *>(workspace);
    a.err = err;
    return launch_attend<false>(layout, a, false, out_dtype == KVQ_BF16, reinterpret_cast<cudaStream_t>(stream));
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
    if (n_sel < 0 || slots_stride < 0 || n_sel > 0x7FFFFFFF - 128) return KVQ_ERR_INVALID_ARG;
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
    return launch_attend<true>(layout, a, slot_dtype == KVQ_I64, out_dtype == KVQ_BF16,
                               reinterpret_cast<cudaStream_t>(stream));
}
