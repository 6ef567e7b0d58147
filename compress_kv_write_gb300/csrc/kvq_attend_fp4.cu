// kvq_attend_fp4.cu -- the attention kernels over V41_FP4 rows.
#include "kvq_attend_kernel.cuh"

namespace kvq {
kvq_status launch_attend_fp4(const AttendArgs &a, bool slots, cudaStream_t s) {
    return slots ? launch_attend_layout<Layout::FP4, true>(a, s) : launch_attend_layout<Layout::FP4, false>(a, s);
}
}  // namespace kvq
