// kv_attention_part_f32.cu -- attention over the paged 8-bit cache, 32-bit queries, as a part of a larger softmax.
#include "kv_attention.cuh"

namespace om {
cudaError_t launch_kv_attention_part_f32(const KvAttentionProblem &p, cudaStream_t s) { return run_kv_attention<float, kPartForm>(p, s); }
}  // namespace om
