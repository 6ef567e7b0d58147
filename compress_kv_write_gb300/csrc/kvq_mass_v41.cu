// kvq_mass_v41.cu -- the attention-mass kernels over V41 rows.
#include "kvq_mass_kernel.cuh"

namespace kvq {
kvq_status launch_mass_v41(const MassArgs &a, cudaStream_t s) { return launch_mass_layout<Layout::V41>(a, s); }
}  // namespace kvq
