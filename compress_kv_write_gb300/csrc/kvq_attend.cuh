// kvq_attend.cuh -- arguments shared by the attention kernels and their C
// entry points.
#pragma once

#include "kvq_launch.cuh"

namespace kvq {

struct AttendArgs {
    const uint16_t *q;  // bf16
    int64_t q_tok, q_head;
    int64_t n_seq;   // sequences (paged) or query tokens (slots)
    int q_len;       // query tokens a sequence; 1 with slots
    int heads;
    const uint8_t *pool;
    int64_t pool_limit;  // pages (paged) or slots
    int page_bits;
    const int32_t *table;  // paged
    int64_t table_rows, table_stride;
    int64_t max_len;  // table_width pages, or n_sel
    const int32_t *req;
    const int32_t *kv_len;
    const void *slots;  // slots
    int64_t slots_stride;
    float scale;
    void *out;
    int64_t out_tok, out_head;
    float *lse;
    uint8_t *ws;
    int32_t *err;
};

}  // namespace kvq
