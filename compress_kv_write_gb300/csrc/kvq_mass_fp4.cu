// kvq_mass_fp4.cu -- the attention-mass kernels over V41_FP4 rows.
#include "kvq_mass_kernel.cuh"

namespace kvq {
kvq_status launch_mass_fp4(const MassArgs &a, cudaStream_t s) { return launch_mass_layout<Layout::FP4>(a, s); }
}  // namespace kvq
