/*
 * kvq.h -- C ABI of the GB300 (sm_103a) KV-cache write path for
 * DeepSeek-V4-style serving: block quantisation of new K rows into a paged
 * pool (optionally pooled by a ratio-r softmax compressor, RMS-normalised and
 * rotated), the once-per-step full->SWA slot translation, and the paged
 * dequant back to a bf16 workspace; and of what a decode step does around it:
 * attention over the pool (also of a tree of drafted tokens), the weight that
 * it gives each token and eviction by it, rotary positions, and the norm.
 *
 * Sources (page title, section):
 *  [P1] "[sglang] DeepSeek V4.1 Paged KV Cache: V41 and FP4 formats"
 *       (sglang#39123): section 1 kv_layout.cuh (V41 / V41_FP4 layouts,
 *       PagedKV, store_row), section 2 c1.cuh/c2.cuh (ratio compressors,
 *       kv_page_bytes), section 4 dequant_k_cache.py, the store-latency
 *       table (store, store + RoPE, fused K norm + RoPE, c1, c2).
 *  [P2] "[sglang] Hoist DSv4 draft-extend SWA write locs" (sglang#34890):
 *       section 1 (translate once per step into a preallocated int32
 *       buffer, zero the tail, no buffer when n exceeds it), section 2.
 *  [P3] "[vLLM] DeepSeek V4 Sparse FP8 Compressor kernel" (vllm#44161):
 *       section 2 (per-element online-softmax pooling), section 3 (RoPE,
 *       bf16 cast, per-32-value absmax and fp8 scale).
 *
 * Conventions for every entry point:
 *  - All array pointers are DEVICE pointers owned by the caller.  The library
 *    allocates nothing, frees nothing and never synchronises.
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and
 *    launched with programmatic dependent launch enabled: a kernel waits for
 *    its predecessor on the stream before its first global read.
 *  - Arguments are checked on the host before anything is launched; a
 *    failing check returns a status and enqueues no work.
 *  - Problems only the device can see (an index outside its table) set bits
 *    in `*err` (when err is not NULL; atomic OR, KVQ_DEVERR_*) and skip that
 *    row or page; the caller zeroes *err and reads it after its own sync.
 *    Kernels never trap.
 *  - Row data are 512 dims ("head dim"); RoPE rotates the last 64 dims
 *    (448..511) as interleaved pairs (448+2i, 449+2i); a quant block is 32
 *    consecutive dims, 16 blocks per token.
 *  - Slots in one call must be distinct (scatter targets do not overlap);
 *    with repeated slots the surviving row is unspecified.
 */
#ifndef KVQ_H
#define KVQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st; /* = cudaStream_t */

typedef enum {
    KVQ_OK = 0,
    KVQ_ERR_INVALID_ARG = 1, /* null / misaligned pointer, bad size or enum */
    KVQ_ERR_UNSUPPORTED = 2, /* valid request with no compiled instance    */
    KVQ_ERR_CAPACITY = 3,    /* n > out_capacity in kvq_translate_loc      */
    KVQ_ERR_LAUNCH = 4       /* the CUDA launch itself failed              */
} kvq_status;

/* [P1] section 1.  V41: 512 e4m3 codes + 16 ue8m0 scales = 528 B/token.
 * V41_FP4: 256 B of e2m1 codes (two per byte, even dim in the low nibble)
 * + 16 e4m3 scales + 16 B of zero padding = 288 B/token. */
typedef enum { KVQ_LAYOUT_V41 = 1, KVQ_LAYOUT_V41_FP4 = 2 } kvq_layout;
typedef enum { KVQ_F32 = 0, KVQ_BF16 = 1 } kvq_dtype;
typedef enum { KVQ_I32 = 0, KVQ_I64 = 1 } kvq_index_dtype;
enum { KVQ_FLAG_ROPE = 1, KVQ_FLAG_NORM = 2 };
enum { KVQ_ROPE_HALF = 1, KVQ_ROPE_INVERSE = 2 }; /* flags of kvq_rope */

/* bits of the device error word */
enum {
    KVQ_DEVERR_SLOT = 1,  /* a slot outside [0, pool_slots) (row skipped)        */
    KVQ_DEVERR_POS = 2,   /* a RoPE position outside [0, cos_sin_rows) (skipped) */
    KVQ_DEVERR_PAGE = 4,  /* a page-table entry outside [0, pool_pages) (skipped)*/
    KVQ_DEVERR_LOC = 8,   /* a full slot outside the translation table (-> -1)   */
    KVQ_DEVERR_WAIT = 16, /* an attention kernel gave up a bounded wait: the rows */
                          /* and lse that it worked on are NaN                    */
    KVQ_DEVERR_STATE = 32,   /* a request index outside [0, n_state) or a count   */
                             /* outside [0, ratio): that request is skipped; in   */
                             /* the calls over pages a row outside its table; in  */
                             /* kvq_tree_mask a parent that is no earlier token   */
    KVQ_DEVERR_LEN = 64      /* a kv_len outside [0, table_width pages] or above  */
                             /* 2^30 (the sequence counts as empty)               */
};

/* Bytes one token occupies: 528 (V41) or 288 (V41_FP4); 0 for a bad layout.
 * [P1] section 1 and "Why is this good" 1. */
size_t kvq_bytes_per_token(kvq_layout layout);

/* Bytes of one page of 2^page_bits tokens: all code rows, then all scale
 * rows ([P1] section 2, kv_page_bytes).  0 for a bad layout / page_bits. */
size_t kvq_page_bytes(kvq_layout layout, int page_bits);

/* 1 if page_bits is supported (the page size is a compile-time constant of the
 * store, compress and dequant kernels), else 0. */
int kvq_page_bits_supported(int page_bits);

/* Full -> SWA slot translation, hoisted to once per step ([P2] sections 1-2).
 *   full_loc     [n] int32 or int64 (loc_dtype): slots of the full pool.
 *   full_to_swa  [full_slots] int32: the SWA slot of each full slot.
 *   out          [out_capacity] int32: out[i] = full_to_swa[full_loc[i]] for
 *                i < n, and out[n:out_capacity] = 0.
 * n > out_capacity returns KVQ_ERR_CAPACITY and enqueues nothing (the
 * caller then translates into a buffer of its own, as the eager fallback
 * does).  A full_loc[i] outside [0, full_slots) writes -1 there and sets
 * KVQ_DEVERR_LOC. */
kvq_status kvq_translate_loc(const void *full_loc, kvq_index_dtype loc_dtype, int64_t n,
                             const int32_t *full_to_swa, int64_t full_slots,
                             int32_t *out, int64_t out_capacity,
                             int32_t *err, struct CUstream_st *stream);

/* Quantise n new rows and scatter them into the paged pool ([P1] section 1
 * store_row, the store / store + RoPE / fused K norm + RoPE kernels).
 *   x            [n, x_row_stride] fp32 or bf16 (x_dtype); the first 512
 *                elements of each row are used; 16-byte aligned rows.
 *   loc          [n] int32 or int64: destination slot of each row.
 *   flags        KVQ_FLAG_NORM: y = x * rsqrt(mean(x^2) + eps) * norm_weight
 *                (norm_weight [512] fp32); KVQ_FLAG_ROPE: rotate dims
 *                448..511 by row pos[i] of cos_sin ([cos_sin_rows, 64] fp32,
 *                32 cosines then 32 sines).  Norm runs before RoPE, all in
 *                fp32, and the result is rounded to bf16 before quantising;
 *                without flags the input is quantised as given.
 *   pool         [pool_slots / 2^page_bits pages] of kvq_page_bytes each;
 *                pool_slots a multiple of 2^page_bits.
 * V41: per 32 dims, scale byte = (amax exponent field - 8) clamped at 0,
 * code = e4m3_satfinite(x * 2^(127 - byte)).  V41_FP4: scale =
 * e4m3(amax / 6), code = e2m1_satfinite(x * rcp(scale)) (a zero scale gives
 * zero codes). */
kvq_status kvq_store(kvq_layout layout, int page_bits, unsigned flags,
                     const void *x, kvq_dtype x_dtype, int64_t n, int64_t x_row_stride,
                     const void *loc, kvq_index_dtype loc_dtype,
                     const float *norm_weight, float eps,
                     const float *cos_sin, int64_t cos_sin_rows, const int32_t *pos,
                     uint8_t *pool, int64_t pool_slots,
                     int32_t *err, struct CUstream_st *stream);

/* Ratio-r softmax compressor + store ([P1] section 2 c1/c2; [P3] sections
 * 2-3, C4A / C128A).  Group g pools rows g*ratio .. g*ratio+ratio-1:
 *   out[d] = sum_t softmax_t(scores[t, d]) * values[t, d]   (per dim d),
 * then (KVQ_FLAG_ROPE) rotates dims 448..511 by row group_pos[g] of cos_sin,
 * rounds to bf16 and quantises into slot loc[g] as kvq_store does.
 *   values, scores  [n_groups * ratio, 512] fp32, contiguous, 16-B aligned.
 *   loc             [n_groups] int32 (already translated slots).
 *   ratio           1, 2, 4 or 128.  KVQ_FLAG_NORM is not accepted. */
kvq_status kvq_compress(kvq_layout layout, int page_bits, int ratio, unsigned flags,
                        const float *values, const float *scores, int64_t n_groups,
                        const float *cos_sin, int64_t cos_sin_rows, const int32_t *group_pos,
                        const int32_t *loc, uint8_t *pool, int64_t pool_slots,
                        int32_t *err, struct CUstream_st *stream);

/* Decode-time ratio-r compressor ([P1] section 2, flash_c1/c2_decode_kernel;
 * [P3] section 2, the online max / sum softmax): each call brings ONE new row
 * per request, and the softmax pool of the request's unfinished group is
 * carried between calls as online state.
 *   values, scores  [n, 512] fp32: request i's new row.
 *   state           [n_state, 3, 512] fp32, caller-owned, per request slot:
 *                   running max m, sum of exp(s - m) and sum of
 *                   exp(s - m) * v of the rows seen so far, per dim.
 *   count           [n_state] int32: rows of the open group (0 .. ratio-1);
 *                   start at 0 with any state contents.
 *   req             [n] int32: state slot of request i (NULL: slot i).
 * When request i's row is the group's ratio-th, the pooled row acc / sum is
 * rotated by row group_pos[i] of cos_sin (KVQ_FLAG_ROPE), rounded to bf16,
 * quantised and stored into slot loc[i] exactly as kvq_compress does, and
 * count returns to 0; otherwise only state and count change and the values
 * of loc[i] and group_pos[i] are ignored.  The kernel reads both arrays
 * before it knows the count (to overlap their latency), so they must hold n
 * readable entries on every call.  A bad request index or count sets
 * KVQ_DEVERR_STATE and skips that request.  Requests in one call must use
 * distinct state slots.  KVQ_FLAG_NORM is not accepted. */
kvq_status kvq_compress_decode(kvq_layout layout, int page_bits, int ratio, unsigned flags,
                               const float *values, const float *scores, int64_t n,
                               float *state, int32_t *count, const int32_t *req, int64_t n_state,
                               const float *cos_sin, int64_t cos_sin_rows, const int32_t *group_pos,
                               const int32_t *loc, uint8_t *pool, int64_t pool_slots,
                               int32_t *err, struct CUstream_st *stream);

/* Paged dequant to a bf16 workspace ([P1] section 4, dequant_k_cache.py).
 *   page_table  [n_tokens / 2^page_bits] int32: physical page of each
 *               logical page; n_tokens must be a multiple of 2^page_bits.
 *   out_bf16    [n_tokens, out_row_stride] bf16 (stride >= 512, rows 16-B
 *               aligned): row t = decode(page_table[t >> page_bits], row
 *               t & (2^page_bits - 1)).  V41: e4m3 * 2^(byte - 127);
 *               V41_FP4: e2m1 * e4m3 scale; both exact in bf16.
 * An entry outside [0, pool_pages) sets KVQ_DEVERR_PAGE and leaves that
 * page's rows untouched. */
kvq_status kvq_dequant(kvq_layout layout, int page_bits,
                       const uint8_t *pool, int64_t pool_pages,
                       const int32_t *page_table, int64_t n_tokens,
                       void *out_bf16, int64_t out_row_stride,
                       int32_t *err, struct CUstream_st *stream);

/* Dequant of selected tokens to bf16 rows: the consumer side of [P1] section
 * 4 (dequant_k_cache.py) restricted to the tokens a sparse attention picks
 * (the FlashMLA sparse-FP8 reader of [P3]).
 *   slots       [n] int32 or int64 (slot_dtype): pool slot of output row i.
 *   out_bf16    [n, out_row_stride] bf16 (stride >= 512, rows 16-B aligned):
 *               row i = decode(slot slots[i]), exact in bf16 as in kvq_dequant.
 * Slot -1 is padding and writes a zero row.  Any other slot outside
 * [0, pool_slots) sets KVQ_DEVERR_SLOT and leaves row i untouched. */
kvq_status kvq_dequant_slots(kvq_layout layout, int page_bits,
                             const uint8_t *pool, int64_t pool_slots,
                             const void *slots, kvq_index_dtype slot_dtype, int64_t n,
                             void *out_bf16, int64_t out_row_stride,
                             int32_t *err, struct CUstream_st *stream);

/* Bytes of workspace a kvq_attend / kvq_attend_slots call needs whose rows
 * per sequence (q_len * heads; for kvq_attend_slots heads) are `rows`: the
 * partial results of work that is split over CTAs.  It depends on nothing
 * else; 0 when rows is not positive.  The contents need no initialisation
 * and mean nothing after the call; calls that may run at the same time need
 * workspaces of their own (captured graphs too, unless they run in turn). */
size_t kvq_attend_workspace(int64_t rows);

/* How often a wait inside the kernels of kvq_attend, kvq_attend_slots,
 * kvq_attend_tree and kvq_attend_mass (for another warp's part of the work)
 * tries before the call gives up with KVQ_DEVERR_WAIT; the default is 2^20,
 * which takes some seconds, far beyond any wait of a sound call.  Sets
 * the limit of the process's later calls (at most 2^24; a captured call keeps
 * the one it was captured with) and returns the one before.  With 0 every call
 * gives up, which is how a program can test what it does then. */
uint32_t kvq_attend_wait_limit(uint32_t tries);

/* Latent attention over a paged pool: the reader of the rows that kvq_store
 * and kvq_compress write.  Every head of a query token attends over the same
 * row k[t] (512 values) of a cached token, as key and as value:
 *   s[t] = scale * sum_d q[d] * k[t][d],  p = softmax(s) over the visible t,
 *   out[d] = sum_t p[t] * k[t][d],        lse = log(sum_t exp(s[t])).
 * Sequence i has q_len query tokens, rows i*q_len .. i*q_len + q_len - 1 of
 * q, and kv_len[i] cached tokens, its own query tokens among them; query
 * token j sees the first kv_len[i] - (q_len - 1 - j) of them (causal).  A
 * query token that sees none gets a zero row and lse = -inf.
 *   q            bf16, element (token, head, d) at token * q_token_stride +
 *                head * q_head_stride + d; 16-B aligned rows.  A stride of 0
 *                repeats a row.
 *   pool         16-B aligned.
 *   page_table   [table_rows, table_stride] int32, the first table_width of
 *                a row used: physical page of each logical page.
 *   req          [n_seq] int32: table row of sequence i (NULL: row i, and
 *                n_seq <= table_rows).
 *   kv_len       [n_seq] int32, 0 .. table_width * 2^page_bits, at most 2^30.
 *   scale        finite.
 *   out          bf16 or fp32 (out_dtype), strides like q's (16-B aligned
 *                rows that do not overlap each other or an input).
 *   lse          [n_seq * q_len, heads] fp32, natural log, or NULL.
 *   workspace    kvq_attend_workspace(q_len * heads) bytes, 16-B aligned.
 * Scores, softmax statistics and sums are fp32; the products' operands are
 * fp16.  A query row is scaled by a power of two that brings its largest value
 * to [2^14, 2^15): exact down to 2^-28 of that value.  A V41_FP4 row is exact
 * as it is.  A V41 row is decoded relative to a power of two of its own that
 * brings its largest scale to 2^7 (the scores and weights take it back):
 * values above 2^-36 of the row's largest are exact, smaller ones off by at
 * most 2^-40 of it, and a block whose scale is 2^-32 of the row's largest or
 * less counts as zeros.  (A row whose largest scale is below 2^-40 counts as
 * if it were 2^-40.)  A softmax weight, for V41 times its row's power of two, is
 * rounded to fp16: relative 2^-11, or, for weights of 2^-14 of the largest and
 * less, by an amount that all of a CTA's tokens together bring to no more than
 * 2^-13 of the largest weight (of n > 2^26 tokens, n 2^-39): a long tail of
 * small weights keeps its share.  The softmax sum takes the weights in fp32.
 * The tensor cores round their sums down; no more than 256 blocks of 64 tokens
 * are summed there before they are added to the rest, rounded to nearest.
 * Scores have to stay within fp32.
 * The result does not depend on anything but the arguments and the number of
 * SMs (no atomics on data).
 * The causal bound moves by one cached row a query token.  Over a pool that
 * kvq_compress wrote, where a row stands for several tokens, pass every query
 * token as a sequence of its own (q_len 1, req for the shared table row) with
 * the kv_len that it sees.
 * At most 2^20 query tokens a sequence, 1,024 heads and 2^24 query tokens in
 * all; more, or more blocks of 64 tokens a CTA than an int holds (taken from
 * table_width, whatever the lengths), is KVQ_ERR_UNSUPPORTED.
 * A visible token whose row holds a NaN or an infinity makes the rows that
 * see it NaN, and no others; what masked tokens hold does not matter, nor does
 * the pool's first row where it is no one's.  A query row that holds a NaN or
 * an infinity is NaN itself, and its lse, where it sees a token.
 * A bad kv_len (KVQ_DEVERR_LEN) or req (KVQ_DEVERR_STATE) makes the sequence
 * an empty one; a table entry outside [0, pool_pages) (KVQ_DEVERR_PAGE) masks
 * its tokens.  Entries past a sequence's kv_len are not read. */
kvq_status kvq_attend(kvq_layout layout, int page_bits,
                      const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                      int64_t n_seq, int64_t q_len, int64_t heads,
                      const uint8_t *pool, int64_t pool_pages,
                      const int32_t *page_table, int64_t table_rows, int64_t table_width,
                      int64_t table_stride, const int32_t *req, const int32_t *kv_len, float scale,
                      void *out, kvq_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride,
                      float *lse, void *workspace, size_t workspace_bytes,
                      int32_t *err, struct CUstream_st *stream);

/* Masks and positions of trees of drafted tokens, for kvq_attend_tree.
 *   parent    [n_seq, parent_stride] int32, the first q_len of a row used:
 *             the token that token j follows, one drafted before it (< j), or
 *             -1: the sequence's last token before the tree.  Anything else
 *             counts as -1 and sets KVQ_DEVERR_STATE.  q_len: at most 1024.
 *   mask      [n_seq, q_len, ceil(q_len / 64)] 64-bit words: bit k % 64 of
 *             word k / 64 of token j is set where k is j or one of its
 *             ancestors.
 *   pos       [n_seq, q_len] int32, or NULL: max(0, kv_len[i] - q_len + depth
 *             of j), the depth being the number of its ancestors (kv_len NULL:
 *             the depth alone).
 *   kv_len    [n_seq] int32, or NULL: here a length in positions, the drafted
 *             tokens included.  Of a cache that was cut (kvq_evict_move) that
 *             is what the sequence would have without the cut: with the cut
 *             length, which the attention takes, drafted tokens would be placed
 *             before keys that they follow. */
kvq_status kvq_tree_mask(const int32_t *parent, int64_t n_seq, int64_t q_len, int64_t parent_stride,
                         const int32_t *kv_len, uint64_t *mask, int32_t *pos, int32_t *err,
                         struct CUstream_st *stream);

/* kvq_attend for a tree of drafted tokens, verified in one step: the last
 * q_len of a sequence's kv_len[i] cached tokens are its query tokens (already
 * stored, in the order of q), and query token j sees all tokens before them
 * and, of them, token k where bit k % 64 of word k / 64 of mask[i][j] is set
 * (its own too).  Any mask is accepted.  Of a sequence with kv_len[i] < q_len
 * the first q_len - kv_len[i] drafted tokens are not there, whatever the mask.
 *   mask      [n_seq, q_len, ceil(q_len / 64)] 64-bit words, 8-B aligned.
 *   q_len     at most 1024.
 * All else is as in kvq_attend, among it that a softmax weight is rounded to
 * fp16 for the outputs' products (not for their sum and lse).  fp32 outputs are
 * off by some 2^-12 of their scale for it; bf16 ones are a neighbouring value of
 * what fp32 weights give in 2 to 6 places of a hundred, and no further off. */
kvq_status kvq_attend_tree(kvq_layout layout, int page_bits,
                           const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                           int64_t n_seq, int64_t q_len, int64_t heads,
                           const uint8_t *pool, int64_t pool_pages,
                           const int32_t *page_table, int64_t table_rows, int64_t table_width,
                           int64_t table_stride, const int32_t *req, const int32_t *kv_len, const uint64_t *mask,
                           float scale, void *out, kvq_dtype out_dtype, int64_t out_token_stride,
                           int64_t out_head_stride, float *lse, void *workspace, size_t workspace_bytes,
                           int32_t *err, struct CUstream_st *stream);

/* kvq_attend over selected tokens: query token i attends over the tokens in
 * slots slots[i * slots_stride + 0 .. n_sel - 1] (int32 or int64), the ones
 * kvq_dequant_slots would gather.  Slot -1 is padding, anywhere in the list;
 * any other slot outside [0, pool_slots) sets KVQ_DEVERR_SLOT and is masked.
 * A slot that is listed twice counts twice.  n_sel: at most 2^30.  workspace:
 * kvq_attend_workspace(heads) bytes. */
kvq_status kvq_attend_slots(kvq_layout layout, int page_bits,
                            const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                            int64_t n_tokens, int64_t heads,
                            const uint8_t *pool, int64_t pool_slots,
                            const void *slots, kvq_index_dtype slot_dtype, int64_t n_sel,
                            int64_t slots_stride, float scale,
                            void *out, kvq_dtype out_dtype, int64_t out_token_stride, int64_t out_head_stride,
                            float *lse, void *workspace, size_t workspace_bytes,
                            int32_t *err, struct CUstream_st *stream);

/* Bytes of workspace a kvq_attend_mass call needs: n_seq sequences of `rows`
 * = q_len * heads query rows over at most max_len tokens (table_width pages of
 * them, or mass_width where that is less).  0 up to 128 rows, 4 bytes a
 * sequence, token and 128 rows beyond.  As kvq_attend_workspace otherwise. */
size_t kvq_mass_workspace(int64_t n_seq, int64_t rows, int64_t max_len);

/* The weight that each cached token gets in kvq_attend, or with a mask in
 * kvq_attend_tree, summed over the query rows that see it (all heads of all
 * q_len query tokens):
 *   w[t] = sum over these rows of exp(scale * sum_d q[d] k[t][d] - lse[row]),
 *   mass[t] = decay * prev[t] + w[t], or, where prev is NULL, w[t],
 * for the tokens t < kv_len[i] of sequence i; what lies behind them in mass
 * stays as it is.  With prev = mass the weights of one step after another add
 * up, the older ones worth `decay` as much each step (a token that is new in
 * the cache has a 0 in prev).
 *   q, pool, page_table, req, kv_len, scale   as in kvq_attend, the call's own.
 *   lse        [n_seq * q_len, heads] fp32: what the attention left.  A row
 *              whose lse is -inf has no weight.
 *   mask       as in kvq_attend_tree (q_len at most 1024), or NULL: causal.
 *   mass       [mass_rows, mass_row_stride] fp32, the first mass_width of a
 *              row used; row rows[i] (NULL: row i) is sequence i's.  Sequences
 *              of a call have rows of their own: what two write to one row is
 *              unspecified.
 *   prev       rows like mass's, by the same index: mass itself with its
 *              stride, or apart from it, or NULL.
 *   n_seq      at most 65535; with T = n_seq * ceil(q_len * heads / 128) and B
 *              = ceil(tokens of the table's width, or mass_width where that is
 *              less, / 128): T * (B + 2) below 2^31, above it the call is
 *              KVQ_ERR_UNSUPPORTED.
 *   workspace  kvq_mass_workspace bytes, 16-B aligned (NULL where that is 0).
 * Products and what counts as nothing are as for kvq_attend's scores.  The
 * tensor cores round a score's sums towards zero; they are kept short (a score
 * of up to 32 rows in four sums; of more rows, less a number near the scores
 * that count), which leaves weights off by some 2^-24 of lse, and by nothing
 * where a row's products sum exactly.
 * The exponent's own roundings are relative to score - lse up to |lse| = 2^28;
 * beyond, where fp32 hardly tells one weight from another, none is NaN for it.
 * Sums are fp32, in one order whatever the lengths (no atomics on data).
 * A token whose row holds a NaN or an infinity, and a query row that does or
 * whose lse is NaN, make the weights that they share in NaN, and no others.
 * A bad kv_len (KVQ_DEVERR_LEN; mass_width is a limit too), req or row
 * (KVQ_DEVERR_STATE) makes the sequence an empty one; a token behind a bad
 * table entry (KVQ_DEVERR_PAGE) has w[t] = 0.  A call that gives up a wait
 * (KVQ_DEVERR_WAIT) leaves NaN in the weights that it worked on. */
kvq_status kvq_attend_mass(kvq_layout layout, int page_bits,
                           const void *q_bf16, int64_t q_token_stride, int64_t q_head_stride,
                           int64_t n_seq, int64_t q_len, int64_t heads, const float *lse,
                           const uint8_t *pool, int64_t pool_pages,
                           const int32_t *page_table, int64_t table_rows, int64_t table_width,
                           int64_t table_stride, const int32_t *req, const int32_t *kv_len, const uint64_t *mask,
                           float scale, float *mass, int64_t mass_rows, int64_t mass_width, int64_t mass_row_stride,
                           const int32_t *rows, const float *prev, int64_t prev_row_stride, float decay,
                           void *workspace, size_t workspace_bytes, int32_t *err, struct CUstream_st *stream);

/* RMS norm of a row plus its residual, quantised like a V41 row: the input
 * of the projections whose K rows kvq_store takes.
 *   z = x + residual (fp32; residual NULL: z = x), residual_out = z rounded
 *   to x_dtype, y = z * rsqrt(mean(z^2) + eps) * weight (fp32), then per 32
 *   values scale byte = (amax exponent field - 8) clamped at 0 and code =
 *   e4m3_satfinite(y * 2^(127 - byte)), as V41 blocks are written.
 *   x, residual   [n, stride] fp32 or bf16 (x_dtype), the first dim elements
 *                 of a row used; 16-B aligned rows.
 *   dim           a multiple of 32, at most 16384.
 *   weight        [dim] fp32, 16-B aligned.
 *   residual_out  rows like x's; given exactly when residual is; it may be
 *                 residual itself, or x, with that one's row stride; rows
 *                 that overlap an input's otherwise are refused.
 *   codes         [n, codes_stride] bytes, codes_stride a multiple of 8,
 *                 8-B aligned.
 *   scales        [n, scales_stride] bytes, dim / 32 used a row.
 * codes and scales overlap no other array. */
kvq_status kvq_norm_quant(const void *x, kvq_dtype x_dtype, int64_t n, int64_t dim, int64_t x_row_stride,
                          const void *residual, int64_t residual_row_stride,
                          void *residual_out, int64_t residual_out_row_stride,
                          const float *weight, float eps,
                          uint8_t *codes, int64_t codes_stride, uint8_t *scales, int64_t scales_stride,
                          struct CUstream_st *stream);

/* The table of cosines and sines that kvq_store, the compressors and kvq_rope
 * read: row r, of rot_dim floats, is amplitude * cos((first + r) * freq[i]),
 * i = 0 .. rot_dim / 2 - 1, and then as many sines.
 *   freq      [rot_dim / 2] fp64, radians a position; the frequencies of a
 *             context that is longer than the model's own are scaled by the
 *             caller.  One that is not finite, or 2^52 turns and more, makes
 *             its columns NaN.
 *   rot_dim   even, at most 1024 (64 for kvq_store).
 *   first     >= 0; first + rows at most 2^31 - 1.
 *   table     [rows, rot_dim] fp32, contiguous, 16-B aligned.
 * Values are off by at most 2^-22 |amplitude|, at every position and for every
 * finite frequency below that limit: the phase is held modulo 2^64 of a turn. */
kvq_status kvq_rope_table(const double *freq, int64_t rot_dim, int64_t first, int64_t rows, float amplitude,
                          float *table, struct CUstream_st *stream);

/* Rotary positions of rows that are not stored: queries before kvq_attend,
 * and, with KVQ_ROPE_INVERSE, its output rows, whose rotated dims carry the
 * cached rows' positions (turned back by the query's, they carry those relative
 * to it).
 *   x          [n_tokens, heads, dim] fp32 or bf16 (dtype), strides in
 *              elements, unit inner stride; a stride of 0 repeats a row.
 *   rot_start, rot_dim   the rotated dims of a row: an even number, at most
 *              1024, within dim (at most 65536); the others are copied.
 *   flags      pairs are neighbours, (start + 2i, start + 2i + 1), or, with
 *              KVQ_ROPE_HALF, (start + i, start + rot_dim / 2 + i);
 *              (u, v) -> (u c - v s, v c + u s), or with KVQ_ROPE_INVERSE
 *              (u c + v s, v c - u s), the transpose (also the gradient).
 *              The transpose undoes the turn where the table's amplitude is 1.
 *              What a table of amplitude A turned is undone with one of 1 / A;
 *              with its own table it comes back times A * A, as do the rotated
 *              dims of outputs over rows that were stored with amplitude A.
 *              fp32, each product and sum rounded, as kvq_store does it.
 *   cos_sin    [cos_sin_rows, rot_dim] fp32, 8-B aligned: cosines, then sines.
 *   pos        [n_tokens] int32: row of cos_sin of every head of a token.
 *   out        dtype; x itself with x's strides (then only the rotated dims
 *              are read and written), or rows that overlap neither x's nor
 *              each other.  Sets of rows that share an address range are
 *              accepted where equal strides keep them beside each other.
 * A pos outside [0, cos_sin_rows) sets KVQ_DEVERR_POS and leaves the token's
 * rows of out as they are.  Rows, parts and halves that begin on 16 (halves of
 * bf16: 8) bytes are faster.  out overlaps neither cos_sin nor pos. */
kvq_status kvq_rope(const void *x, kvq_dtype dtype, int64_t n_tokens, int64_t heads, int64_t dim,
                    int64_t x_token_stride, int64_t x_head_stride, int64_t rot_start, int64_t rot_dim, unsigned flags,
                    const float *cos_sin, int64_t cos_sin_rows, const int32_t *pos, void *out,
                    int64_t out_token_stride, int64_t out_head_stride, int32_t *err, struct CUstream_st *stream);

/* Which cached tokens stay when a sequence is cut to `keep`: the first `first`
 * and the last `last` of it anyway, and of those between the ones of most
 * weight (kvq_attend_mass); of equal weights the first ones.  A sequence of
 * at most `keep` tokens stays whole.
 *   mass       [mass_rows, mass_row_stride] fp32, the first mass_width of a
 *              row used: a weight for each token.  Zeros of both signs are
 *              equal, a NaN is above everything.
 *   rows       [n_seq] int32: row of mass of sequence i (NULL: row i).
 *   kv_len     [n_seq] int32: tokens of a sequence, at most mass_width.
 *   keep       >= first + last, at least 1.
 *   kept       [n_seq, kept_stride] int32: the tokens that stay, ascending,
 *              then -1 up to `keep`.
 *   count      [n_seq] int32: how many stay.
 * A bad kv_len (KVQ_DEVERR_LEN) or row (KVQ_DEVERR_STATE) makes the sequence
 * an empty one. */
kvq_status kvq_evict_select(const float *mass, int64_t mass_rows, int64_t mass_width, int64_t mass_row_stride,
                            const int32_t *rows, const int32_t *kv_len, int64_t n_seq, int64_t keep, int64_t first,
                            int64_t last, int32_t *kept, int64_t kept_stride, int32_t *count, int32_t *err,
                            struct CUstream_st *stream);

/* Moves the rows that stay to pages of their own: token kept[i][k] of sequence
 * i, codes and scales as they are, becomes token k of the pages in row i of
 * new_table, and its weight mass_out[i][k].  An entry of -1 moves nothing.
 *   page_table, req   as in kvq_attend.
 *   new_table  [n_seq, new_stride] int32: pages of this pool, as many as hold
 *              `keep` tokens (new_width).  A page in it that holds rows of the
 *              old tables too is fine only where its rows stay where they are
 *              (the first pages of a sequence whose first tokens all stay):
 *              otherwise rows may be overwritten before they are read.  No
 *              page is in two places of it that tokens move to.
 *   mass, rows as in kvq_evict_select; mass and mass_out NULL: no weights.
 *   mass_out   [n_seq, mass_out_stride] fp32, apart from mass.
 * An entry outside the table or the weights sets KVQ_DEVERR_SLOT, a page
 * outside the pool, old or new, KVQ_DEVERR_PAGE, a bad req or row
 * KVQ_DEVERR_STATE: the token does not move, and its place stays as it is.
 * The rows keep the rotation of the positions that they had.  From then on the
 * caller has two lengths of a sequence: `count` and what is stored behind it,
 * for the calls over pages, and the one without the cut, for positions
 * (kvq_tree_mask, kvq_rope, kvq_store). */
kvq_status kvq_evict_move(kvq_layout layout, int page_bits, uint8_t *pool, int64_t pool_pages,
                          const int32_t *page_table, int64_t table_rows, int64_t table_width, int64_t table_stride,
                          const int32_t *req, const int32_t *new_table, int64_t new_width, int64_t new_stride,
                          const int32_t *kept, int64_t n_seq, int64_t keep, int64_t kept_stride, const float *mass,
                          int64_t mass_rows, int64_t mass_width, int64_t mass_row_stride, const int32_t *rows,
                          float *mass_out, int64_t mass_out_stride, int32_t *err, struct CUstream_st *stream);

/* Human-readable name of a status. */
const char *kvq_status_string(kvq_status status);

#ifdef __cplusplus
}
#endif
#endif /* KVQ_H */
