// The norms' gradient for fp16 rows.
#include "norm_ring.cuh"

namespace moe {

template int launch_norm_ring<__half>(const BackArgs&, int, int, bool, int, int, cudaStream_t);

}  // namespace moe
