// block_norm.cu -- the norms before and after a block of a decoder layer, with the block's gate and
// residual scale in between: x = residual + scale act(gate) N_post(y), h = N(x), one pass over a row.
//
// Mathematics. N of a row v: v / sqrt(mean(v^2) + eps) weight (rms), or with v - mean(v) in v's place and + bias
// (layer; the mean first, then the squares of what is left, so that a large mean costs no bits). All of it in 32 bits;
// h is taken from x before x is rounded to its type: two roundings in a row would show in 16-bit outputs.
//
// Split. A row stays in the registers of its threads between the reductions (a warp, or a block of up to 1024 threads
// with up to 32 elements each), so every operand is read once. Few rows take as many threads as leave each eight
// elements: what counts is the latency of the loads and reductions. Many rows take 32 elements a thread
// (all loads of a row in flight together, several blocks an SM overlap their reductions).
//
// Bound: HBM for many rows, latency for few.

#include <type_traits>

#include "decode_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kVector = 8;  // elements of a thread's load

struct NormArgs {
    NormProblem p;
    int row_warps;  // warps of a row
};

// Where element e of a thread's vector v lies in its row: with ALIGNED eight neighbours in a vector, else every
// thread-count-th element (neighbouring lanes take neighbouring elements, at any alignment).
template <bool ALIGNED>
__device__ __forceinline__ int place(int v, int e, int thread, int threads) {
    return ALIGNED ? (v * threads + thread) * kVector + e : (v * kVector + e) * threads + thread;
}

// A vector as it is read, two 16-bit elements a word; 0 behind the width.
template <typename T>
struct Held {
    static constexpr int kWords = kVector * sizeof(T) / 4;
    uint32_t w[kWords];
};

template <typename T, bool ALIGNED>
__device__ __forceinline__ Held<T> load_vector(const T *row, int v, int width, int thread, int threads) {
    Held<T> h;
    if constexpr (ALIGNED) {
        const int i = place<true>(v, 0, thread, threads);
#pragma unroll
        for (int q = 0; q < Held<T>::kWords; q += 4) {
            const uint4 x = i < width ? *reinterpret_cast<const uint4 *>(row + i + q * 4 / sizeof(T)) : make_uint4(0, 0, 0, 0);
            h.w[q] = x.x; h.w[q + 1] = x.y; h.w[q + 2] = x.z; h.w[q + 3] = x.w;
        }
    } else {
        T x[kVector];
#pragma unroll
        for (int e = 0; e < kVector; ++e) {
            const int i = place<false>(v, e, thread, threads);
            x[e] = i < width ? row[i] : from_float<T>(0.0f);
        }
        memcpy(h.w, x, sizeof(x));
    }
    return h;
}

template <typename T>
__device__ __forceinline__ void expand(const Held<T> &h, float *x) {
    T e[kVector];
    memcpy(e, h.w, sizeof(e));
#pragma unroll
    for (int i = 0; i < kVector; ++i) x[i] = to_float(e[i]);
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_vector(T *row, int v, int width, int thread, int threads, const float *x) {
    T e[kVector];
#pragma unroll
    for (int i = 0; i < kVector; ++i) e[i] = from_float<T>(x[i]);
    if constexpr (ALIGNED) {
        const int i = place<true>(v, 0, thread, threads);
        Held<T> h;
        memcpy(h.w, e, sizeof(e));
        if (i < width) {
#pragma unroll
            for (int q = 0; q < Held<T>::kWords; q += 4)
                *reinterpret_cast<uint4 *>(row + i + q * 4 / sizeof(T)) = make_uint4(h.w[q], h.w[q + 1], h.w[q + 2], h.w[q + 3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVector; ++j) {
            const int i = place<false>(v, j, thread, threads);
            if (i < width) row[i] = e[j];
        }
    }
}

// A vector of weights, of the activations' type or 32 bits.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_weights(const void *w, bool wide, int v, int width, int thread, int threads, float *x) {
    if (std::is_same_v<T, float> || wide)
        expand(load_vector<float, ALIGNED>(static_cast<const float *>(w), v, width, thread, threads), x);
    else
        expand(load_vector<T, ALIGNED>(static_cast<const T *>(w), v, width, thread, threads), x);
}

// The sum over a row's threads, in one order whatever the timing. held: of this use alone.
__device__ __forceinline__ float row_sum(float x, int row_warps, float *held) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (row_warps == 1) return x;
    if ((threadIdx.x & 31) == 0) held[threadIdx.x / 32] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < row_warps ? held[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// x <- N(x). Elements behind the width are 0 and stay out of the sums.
template <typename T, bool ALIGNED, int V>
__device__ __forceinline__ void normalise(float (&x)[V][kVector], const NormProblem &p, const void *weight, const void *bias, int thread, int threads,
                                          int row_warps, float (*held)[32]) {
    const float count = static_cast<float>(p.width);
    const int width = static_cast<int>(p.width);
    const bool wide = p.weight_dtype == OM_F32;
    if (p.layer) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) sum = __fadd_rn(sum, x[v][e]);
        const float mean = __fdiv_rn(row_sum(sum, row_warps, held[0]), count);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = place<ALIGNED>(v, e, thread, threads) < width ? __fsub_rn(x[v][e], mean) : 0.0f;
    }
    float squares = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < kVector; ++e) squares = __fmaf_rn(x[v][e], x[v][e], squares);
    const float inv = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(row_sum(squares, row_warps, held[1]), count), p.eps)));
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[kVector];
        if (weight) load_weights<T, ALIGNED>(weight, wide, v, width, thread, threads, w);
#pragma unroll
        for (int e = 0; e < kVector; ++e) {
            x[v][e] = __fmul_rn(x[v][e], inv);
            if (weight) x[v][e] = __fmul_rn(x[v][e], w[e]);
        }
        if (bias) {
            load_weights<T, ALIGNED>(bias, wide, v, width, thread, threads, w);
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fadd_rn(x[v][e], w[e]);
        }
    }
}

__device__ __forceinline__ float gate_factor(float g, int activation) {
    if (activation == OM_GATE_NONE) return g;
    const float t = __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-g)));
    if (activation == OM_GATE_SIGMOID) return t;
    return t == 0.0f ? 0.0f : __fmul_rn(g, t);  // g t at the low end, minus infinity included, is its limit
}

template <typename T, typename R, int V, int THREADS, bool ALIGNED>
__global__ void __launch_bounds__(THREADS) block_norm_kernel(const __grid_constant__ NormArgs a) {
    const NormProblem &p = a.p;
    __shared__ float held[4][32];  // the warps' parts of each sum
    const int threads = a.row_warps * 32, thread = a.row_warps == 1 ? threadIdx.x & 31 : threadIdx.x, width = static_cast<int>(p.width);
    const int64_t row = a.row_warps == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    wait_for_earlier();
    if (row >= p.tokens) return;  // a warp that has a row of its own, never a part of a block that shares one
    Held<T> y[V], g[V];
    Held<R> r[V];
    // all of the row's operands are on their way together, where the registers hold them: 1024 threads of 32 elements have room for x alone
    constexpr bool kTogether = V * THREADS <= 2048;
    auto residual = [&](int v) { return load_vector<R, ALIGNED>(static_cast<const R *>(p.residual) + row * p.ldr, v, width, thread, threads); };
    auto gate = [&](int v) { return load_vector<T, ALIGNED>(static_cast<const T *>(p.gate) + row * p.ldg, v, width, thread, threads); };
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = load_vector<T, ALIGNED>(static_cast<const T *>(p.y) + row * p.ldy, v, width, thread, threads);
    if (kTogether && p.residual) {
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = residual(v);
    }
    if (kTogether && p.gate) {
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = gate(v);
    }
    float x[V][kVector];
#pragma unroll
    for (int v = 0; v < V; ++v) expand(y[v], x[v]);
    if (p.post) normalise<T, ALIGNED, V>(x, p, p.post_weight, p.post_bias, thread, threads, a.row_warps, held);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[kVector];
        if (p.gate) {
            expand(kTogether ? g[v] : gate(v), f);
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fmul_rn(x[v][e], gate_factor(f[e], p.activation));
        }
        if (p.residual) expand(kTogether ? r[v] : residual(v), f);
#pragma unroll
        for (int e = 0; e < kVector; ++e) x[v][e] = p.residual ? __fmaf_rn(p.scale, x[v][e], f[e]) : __fmul_rn(p.scale, x[v][e]);
    }
    if (p.sum) {
#pragma unroll
        for (int v = 0; v < V; ++v) store_vector<R, ALIGNED>(static_cast<R *>(p.sum) + row * p.lds, v, width, thread, threads, x[v]);
    }
    if (!p.out) return;
    normalise<T, ALIGNED, V>(x, p, p.weight, p.bias, thread, threads, a.row_warps, held + 2);
#pragma unroll
    for (int v = 0; v < V; ++v) store_vector<T, ALIGNED>(static_cast<T *>(p.out) + row * p.ldo, v, width, thread, threads, x[v]);
}

template <typename T, typename R, int V, int THREADS>
cudaError_t by_alignment(const NormArgs &a, bool aligned, cudaStream_t s) {
    const int rows = a.row_warps == 1 ? 4 : 1;  // of a block
    const dim3 grid(static_cast<unsigned>((a.p.tokens + rows - 1) / rows)), block(32 * a.row_warps * rows);
    return launch_behind(aligned ? block_norm_kernel<T, R, V, THREADS, true> : block_norm_kernel<T, R, V, THREADS, false>, grid, block, 0, s, a);
}

template <typename T, typename R>
cudaError_t by_width(const NormProblem &p, cudaStream_t s) {
    auto ok = [](const void *x, int64_t ld, int64_t bytes) { return !x || (reinterpret_cast<uintptr_t>(x) % 16 == 0 && ld * bytes % 16 == 0); };
    const int64_t tb = sizeof(T), rb = sizeof(R);
    const bool aligned = p.width % kVector == 0 && ok(p.y, p.ldy, tb) && ok(p.residual, p.ldr, rb) && ok(p.gate, p.ldg, tb) && ok(p.sum, p.lds, rb) &&
                         ok(p.out, p.ldo, tb) && ok(p.weight, 0, tb) && ok(p.bias, 0, tb) && ok(p.post_weight, 0, tb) && ok(p.post_bias, 0, tb);
    const int64_t vectors = (p.width + kVector - 1) / kVector;
    auto warps = [&](int v) { return static_cast<int>((vectors + 32 * v - 1) / (32 * v)); };
    if (warps(1) <= 32 && p.tokens <= 2 * num_sms()) return by_alignment<T, R, 1, 1024>(NormArgs{p, warps(1)}, aligned, s);
    if (warps(4) <= 16) return by_alignment<T, R, 4, 512>(NormArgs{p, warps(4)}, aligned, s);
    return by_alignment<T, R, 4, 1024>(NormArgs{p, warps(4)}, aligned, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormProblem &p, cudaStream_t s) {
    if (p.dtype == OM_F32) return by_width<float, float>(p, s);
    if (p.dtype == OM_F16) return p.stream_dtype == OM_F32 ? by_width<__half, float>(p, s) : by_width<__half, __half>(p, s);
    return p.stream_dtype == OM_F32 ? by_width<__nv_bfloat16, float>(p, s) : by_width<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace om
