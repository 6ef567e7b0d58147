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
    bool slots64, out_bf16;
    uint32_t wait_tries;  // how often a wait inside the kernel tries before the call gives up
    // set at the launch
    int row_tiles;  // tiles of query rows a sequence
    int2 *join;     // workspace, one a CTA: the tile it began and another CTA went on with (or -1), that tile's last CTA
    float *part;    // workspace, two a CTA: a tile it went on with, a tile it began; kPartRow floats a query row
};

// A partial result of a query row: 512 sums, the running maximum (log2), the
// weights' sum, padding to 16 bytes.
constexpr int kPartRow = kD + 4;
constexpr int kMaxAttendCtas = 160;

// Query rows a tile holds, by the rows of a sequence: the fewest that hold them, up to 64 (kvq_attend_kernel.cuh has
// both sides' times).
constexpr int attend_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// (m + log2 sum) ln 2.  The sum's power of two is added to m, since the two may cancel (rows of large powers of two).
__device__ __forceinline__ float attend_lse(float m, float sum) {
    const int e = int(__float_as_uint(sum) >> 23) - 127;
    if (e < -126 || e > 127) return (m + log2f(sum)) * 0.6931471805599453f;  // zero, infinite, NaN
    return ((m + float(e)) + log2f(__uint_as_float((__float_as_uint(sum) & 0x7FFFFFu) | 0x3F800000u))) * 0.6931471805599453f;
}

kvq_status launch_attend_v41(const AttendArgs &a, bool slots, cudaStream_t s);
kvq_status launch_attend_fp4(const AttendArgs &a, bool slots, cudaStream_t s);

}  // namespace kvq
