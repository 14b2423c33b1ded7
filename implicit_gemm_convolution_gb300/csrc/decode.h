// decode.h -- problems of the decoding operators (4-bit matrix-vector product,
// paged 8-bit cache: append, attention, read back), validated by
// decode_api.cu and run by w4_matvec.cuh, kv_cache.cu and kv_attention.cuh. Not
// installed; not part of the public ABI.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "om.h"

namespace om {

// Launches a kernel that may be started while the stream's kernel before it still runs: it has to
// call wait_for_earlier() before its first access to memory.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What a launcher has found out or set up, for each device: a kernel's attributes and occupancy belong to one. Host threads that
// meet here write the same value.
class PerDevice {
    std::atomic<int> kept_[64] = {};

public:
    // The current device's place, 0 at first; NULL for a device behind the last place.
    std::atomic<int> *here() {
        int dev = 0;
        return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? &kept_[dev] : nullptr;
    }
};

// y[i][j] = sum_p x[i][p] * (u[j][p] - z[j][p / group]) * s[j][p / group].
struct W4Problem {
    int64_t m, n, k, group;
    const void *x;
    int64_t ldx;  // elements
    int x_dtype;  // also y's
    const uint8_t *u;
    int64_t ldu;  // bytes
    const void *s;
    int64_t lds;  // elements
    int s_dtype;
    const uint8_t *z;  // NULL: every zero point is 8
    int64_t ldz;
    void *y;
    int64_t ldy;
};
cudaError_t launch_w4_matvec_f32(const W4Problem &p, cudaStream_t s);
cudaError_t launch_w4_matvec_f16(const W4Problem &p, cudaStream_t s);
cudaError_t launch_w4_matvec_bf16(const W4Problem &p, cudaStream_t s);

// A token-major, head-strided operand: element (t, h, d) at t*ts + h*hs + d.
struct Heads {
    const void *p;
    int64_t ts, hs;
};

struct KvAppendProblem {
    om_kv_cache c;
    int64_t seqs, tokens, max_new, q_heads;
    Heads q, k, v, q_out;
    int dtype;
    const float *table;  // [rows][rot / 2][2]: cos, sin
    int64_t rows, rot;
    int interleaved;
    const int32_t *block_table;
    int64_t width;
    const int32_t *ctx, *cu;
};
cudaError_t launch_kv_append(const KvAppendProblem &p, cudaStream_t s);

struct KvReadProblem {
    om_kv_cache c;
    int64_t seqs, tokens;
    const int32_t *block_table;
    int64_t width;
    const int32_t *start, *cu;
    void *k_out, *v_out;  // [tokens][heads][dim]
    int dtype;
};
cudaError_t launch_kv_read(const KvReadProblem &p, cudaStream_t s);

struct KvAttentionProblem {
    om_kv_cache c;
    int64_t seqs, tokens, max_new, q_heads;
    Heads q, out;
    int dtype;
    float *lse;  // [tokens][q_heads] or NULL
    const int32_t *block_table;
    int64_t width;
    const int32_t *ctx, *cu;
    float scale;
    int64_t window;  // 0: none
    void *workspace;
};
// Query rows that a block holds at once (query tokens times heads of a group,
// in eights), and the workspace of a call: a page of arrival counters, then
// two partial results (rows x (dim + 2) floats) for each of kKvMaxBlocks blocks.
constexpr int64_t kKvMaxBlocks = 608;
constexpr size_t kKvCounterBytes = 4096;
inline int64_t kv_block_rows(int64_t group, int64_t max_new) {
    // more rows than a block holds take further blocks
    const int64_t rows = max_new > (int64_t(1) << 20) || group > (int64_t(1) << 20) ? int64_t(1) << 20 : group * max_new;
    return rows <= 8 ? 8 : 16;
}
inline size_t kv_workspace_bytes(int64_t group, int64_t dim, int64_t max_new) {
    return kKvCounterBytes + static_cast<size_t>(2 * kKvMaxBlocks * kv_block_rows(group, max_new) * (dim + 2) * 4);
}
cudaError_t launch_kv_attention_f32(const KvAttentionProblem &p, cudaStream_t s);
cudaError_t launch_kv_attention_f16(const KvAttentionProblem &p, cudaStream_t s);
cudaError_t launch_kv_attention_bf16(const KvAttentionProblem &p, cudaStream_t s);

cudaError_t launch_rope_table(int64_t rows, int64_t rot, double base, int scaling, double factor,
                              double original, double beta_fast, double beta_slow, float *table,
                              cudaStream_t s);

}  // namespace om
