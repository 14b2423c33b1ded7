// w4_matvec_f16.cu -- products of a few rows with 4-bit weights, float16 activations.
#include "w4_matvec.cuh"

namespace om {
cudaError_t launch_w4_matvec_f16(const W4Problem &p, cudaStream_t s) { return run_w4_matvec<__half>(p, s); }
}  // namespace om
