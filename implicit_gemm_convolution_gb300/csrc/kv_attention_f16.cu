// kv_attention_f16.cu -- attention over the paged 8-bit cache, float16 queries.
#include "kv_attention.cuh"

namespace om {
cudaError_t launch_kv_attention_f16(const KvAttentionProblem &p, cudaStream_t s) { return run_kv_attention<__half>(p, s); }
}  // namespace om
