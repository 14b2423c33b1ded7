// kv_attention.cu -- attention over the paged 8-bit cache.

#include <type_traits>

#include "decode_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kWarps = 4;

// One block per (token, query head); warp w takes the visible positions w, w + 4, ...,
// its lanes the head dimension, one pass with the running maximum and sum;
// the warps' results are joined at the end.
template <typename T, int KV, int DIM>
__global__ void __launch_bounds__(kWarps * 32) kv_attention_simple_kernel(const __grid_constant__ KvAttentionProblem p) {
    constexpr int kPer = DIM / 32;
    __shared__ float part[kWarps][DIM + 2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x / p.q_heads, hq = blockIdx.x % p.q_heads;
    const int64_t h = hq / (p.q_heads / p.c.heads), page = p.c.page;
    const int64_t b = block_sequence_of(p.cu, p.seqs, t);
    int64_t pos = -1;
    if (b < p.seqs && t >= p.cu[b]) {
        int64_t t0, t1;
        token_range(p.cu, b, p.tokens, &t0, &t1);
        pos = p.ctx[b] - t1 + t;
    }
    int64_t hi = pos + 1 < p.width * page ? pos + 1 : p.width * page;
    const int64_t lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    float q[kPer], acc[kPer], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
        q[e] = to_float(static_cast<const T *>(p.q.p)[t * p.q.ts + hq * p.q.hs + lane * kPer + e]);
        acc[e] = 0.0f;
    }
    for (int64_t i = lo + warp; i < hi; i += kWarps) {
        const int64_t id = p.block_table[b * p.width + i / page];
        if (id < 0 || id >= p.c.pages) continue;
        const int64_t row = ((id * p.c.heads + h) * page + i % page) * DIM + lane * kPer;
        const uint8_t *kr = static_cast<const uint8_t *>(p.c.k) + row, *vr = static_cast<const uint8_t *>(p.c.v) + row;
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < kPer; ++e) dot = __fmaf_rn(q[e], decode<KV>(kr[e]), dot);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, o));
        const float sc = dot * p.c.k_scale[id * p.c.heads + h] * p.scale;
        const float vs = p.c.v_scale[id * p.c.heads + h];
        const float m = fmaxf(top, sc), ref = m == -INFINITY ? 0.0f : m;
        const float old = expf(top - ref), e1 = sc != sc ? sc : expf(sc - ref);
        top = m;
        sum = sum * old + e1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = __fmaf_rn(e1, decode<KV>(vr[e]) * vs, acc[e] * old);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) part[warp][lane * kPer + e] = acc[e];
    if (lane == 0) {
        part[warp][DIM] = top;
        part[warp][DIM + 1] = sum;
    }
    __syncthreads();
    float m = -INFINITY, l = 0.0f;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, part[w][DIM]);
    const float ref = m == -INFINITY ? 0.0f : m;
    for (int w = 0; w < kWarps; ++w) l += part[w][DIM + 1] * expf(part[w][DIM] - ref);
    for (int d = threadIdx.x; d < DIM; d += kWarps * 32) {
        float o = 0.0f;
        for (int w = 0; w < kWarps; ++w) o += part[w][d] * expf(part[w][DIM] - ref);
        static_cast<T *>(const_cast<void *>(p.out.p))[t * p.out.ts + hq * p.out.hs + d] = from_float<T>(l == 0.0f ? 0.0f : o / l);
    }
    if (p.lse && threadIdx.x == 0) p.lse[t * p.q_heads + hq] = l == 0.0f ? -INFINITY : ref + logf(l);
}

template <typename T, int KV>
cudaError_t run(const KvAttentionProblem &p, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.tokens * p.q_heads);
    if (p.c.dim == 64)
        kv_attention_simple_kernel<T, KV, 64><<<grid, kWarps * 32, 0, s>>>(p);
    else if (p.c.dim == 128)
        kv_attention_simple_kernel<T, KV, 128><<<grid, kWarps * 32, 0, s>>>(p);
    else
        kv_attention_simple_kernel<T, KV, 256><<<grid, kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_codes(const KvAttentionProblem &p, cudaStream_t s) {
    return p.c.dtype == OM_I8 ? run<T, OM_I8>(p, s) : run<T, OM_E4M3>(p, s);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionProblem &p, cudaStream_t s) {
    if (p.dtype == OM_F32) return run_codes<float>(p, s);
    if (p.dtype == OM_F16) return run_codes<__half>(p, s);
    return run_codes<__nv_bfloat16>(p, s);
}

}  // namespace om
