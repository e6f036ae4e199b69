// The norms' gradient for fp32 rows of 16-byte words.
#include "norm_ring.cuh"

namespace moe {

template int launch_norm_ring<float>(const BackArgs&, int, int, int, int, cudaStream_t);

}  // namespace moe
