// kv_shared_e4m3.cu -- attention to shared prefixes, 8-bit floats.
#include "kv_shared.cuh"

namespace om {
cudaError_t launch_kv_shared_e4m3(const SharedProblem &p, cudaStream_t s) { return run_kv_shared<OM_E4M3, false>(p, s); }
}  // namespace om
