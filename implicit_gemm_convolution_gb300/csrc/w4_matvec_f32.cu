// w4_matvec_f32.cu -- products of a few rows with 4-bit weights, 32-bit activations.
#include "w4_matvec.cuh"

namespace om {
cudaError_t launch_w4_matvec_f32(const W4Problem &p, cudaStream_t s) { return run_w4_matvec<float>(p, s); }
}  // namespace om
