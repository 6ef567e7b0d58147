// kvq_tree_v41.cu -- the attention kernels of a tree of drafted tokens over V41 rows.
#include "kvq_attend_kernel.cuh"

namespace kvq {
kvq_status launch_attend_tree_v41(const AttendArgs &a, cudaStream_t s) { return launch_attend_layout<Layout::V41, kByTree>(a, s); }
}  // namespace kvq
