// kv_attention_bf16.cu -- attention over the paged 8-bit cache, bfloat16 queries.
#include "kv_attention.cuh"

namespace om {
cudaError_t launch_kv_attention_bf16(const KvAttentionProblem &p, cudaStream_t s) { return run_kv_attention<__nv_bfloat16, kPlainForm>(p, s); }
}  // namespace om
