// The norms' gradient for fp32 rows.
#include "norm_ring.cuh"

namespace moe {

template int launch_norm_ring<float>(const BackArgs&, int, int, bool, int, int, cudaStream_t);

}  // namespace moe
