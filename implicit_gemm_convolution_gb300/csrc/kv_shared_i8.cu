// kv_shared_i8.cu -- attention to shared prefixes, whole numbers.
#include "kv_shared.cuh"

namespace om {
cudaError_t launch_kv_shared_i8(const SharedProblem &p, cudaStream_t s) { return run_kv_shared<OM_I8, false>(p, s); }
}  // namespace om
