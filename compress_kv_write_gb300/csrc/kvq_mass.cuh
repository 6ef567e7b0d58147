// kvq_mass.cuh -- arguments shared by the attention-mass kernels and their C
// entry point.
#pragma once

#include "kvq_attend.cuh"

namespace kvq {

struct MassArgs {
    const uint16_t *q;  // bf16
    int64_t q_tok, q_head;
    int64_t n_seq;
    int q_len, heads;
    const uint8_t *pool;
    int64_t pool_limit;  // pages
    int page_bits;
    const int32_t *table;
    int64_t table_rows, table_stride;
    int64_t max_len;  // tokens that a row of the table, and of the weights, has
    const int32_t *req;
    const int32_t *kv_len;
    const uint64_t *mask;  // tree: mask_words a query token; or NULL
    int mask_words;
    const float *lse;
    // A weight is 2^(S c + n) with c = scale log2(e) and n = -log2(e) lse, whose roundings to fp32 would be up to 2^-24 (|S c|
    // + |n|) of the exponent.  S c is about -n wherever a weight counts, so a row's weights are taken times 2^((n - fl(n)) - n
    // c_off), c_off being the relative error of fl(c): what is left is relative to S c + n.  What the tensor cores drop of S
    // is kept small (kvq_mass_kernel.cuh) but not made up for: how much it is depends on the row.  (Its mean over N(0, 1) rows added
    // here left rows whose products sum exactly off by 1.6 10^-4 at a score of 1,000.)
    float c, c_off, scale;
    float *mass;
    int64_t mass_stride;
    const float *prev;
    int64_t prev_stride;
    const int32_t *rows;
    int64_t n_rows;
    float decay;
    float *part;  // workspace: a tile's sums, where a sequence has several tiles
    int64_t part_stride;
    int32_t *err;
    uint32_t wait_tries;
    int row_tiles;  // set at the launch: tiles of query rows a sequence
};

// Query rows a tile holds, by the rows of a sequence (kvq_mass_kernel.cuh has the times).
constexpr int mass_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }
constexpr int64_t mass_tiles(int64_t rows) { return (rows + mass_rows(rows) - 1) / mass_rows(rows); }
constexpr int64_t mass_part_stride(int64_t max_len) { return (max_len + 3) & ~int64_t(3); }

kvq_status launch_mass_v41(const MassArgs &a, cudaStream_t s);
kvq_status launch_mass_fp4(const MassArgs &a, cudaStream_t s);

}  // namespace kvq
