// kv_attention_sinks_f32.cu -- attention over the paged 8-bit cache, 32-bit queries, first tokens that stay visible.
#include "kv_attention.cuh"

namespace om {
cudaError_t launch_kv_attention_sinks_f32(const KvAttentionProblem &p, cudaStream_t s) { return run_kv_attention<float, kSinksForm>(p, s); }
}  // namespace om
