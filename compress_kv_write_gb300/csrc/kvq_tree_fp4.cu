// kvq_tree_fp4.cu -- the attention kernels of a tree of drafted tokens over V41_FP4 rows.
#include "kvq_attend_kernel.cuh"

namespace kvq {
kvq_status launch_attend_tree_fp4(const AttendArgs &a, cudaStream_t s) { return launch_attend_layout<Layout::FP4, kByTree>(a, s); }
}  // namespace kvq
