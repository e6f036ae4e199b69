// The norms' gradient for bf16 rows.
#include "norm_ring.cuh"

namespace moe {

template int launch_norm_ring<__nv_bfloat16>(const BackArgs&, int, int, bool, int, int, cudaStream_t);

}  // namespace moe
