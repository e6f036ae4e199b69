// The norms' gradient for bf16 rows of 16-byte words.
#include "norm_ring.cuh"

namespace moe {

template int launch_norm_ring<__nv_bfloat16>(const BackArgs&, int, int, int, int, cudaStream_t);

}  // namespace moe
