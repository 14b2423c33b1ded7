// kv_shared_pages_e4m3.cu -- attention to shared prefixes, 8-bit floats, in pages smaller than a tile.
#include "kv_shared.cuh"

namespace om {
cudaError_t launch_kv_shared_pages_e4m3(const SharedProblem &p, cudaStream_t s) { return run_kv_shared<OM_E4M3, true>(p, s); }
}  // namespace om
