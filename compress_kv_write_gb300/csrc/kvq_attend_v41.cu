// kvq_attend_v41.cu -- the attention kernels over V41 rows.
#include "kvq_attend_kernel.cuh"

namespace kvq {
kvq_status launch_attend_v41(const AttendArgs &a, bool slots, cudaStream_t s) {
    return slots ? launch_attend_layout<Layout::V41, true>(a, s) : launch_attend_layout<Layout::V41, false>(a, s);
}
}  // namespace kvq
