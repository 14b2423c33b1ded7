// block_norm.cu -- the norms before and after a block of a decoder layer, with the block's gate and
// residual scale in between: x = residual + scale act(gate) N_post(y), h = N(x), one pass over a row.
//
// Mathematics. N of a row v: v / sqrt(mean(v^2) + eps) weight (rms), or with v - mean(v) in v's place and + bias (layer). All of it in 32 bits;
// h is taken from x before x is rounded to its type: two roundings in a row would show in 16-bit outputs.
// A layer's mean comes first, rounded to 32 bits; d = v - mean is exact where the mean is large beside the spread, and what the mean is off by is
// in every d alike, so the mean of d is taken out too: (d - mean(d)) / sqrt(mean(d^2) - mean(d)^2 + eps), whose sums go together. Without it
// a row of mean 4096 and spread 1 was 3e-4 off and a row of one value 4096.3 came out as 0.4; with it 1e-6 and 0 (16000 x 8192 with
// both norms 374 -> 383 us).
//
// Split. A row stays in the registers of its threads between the reductions (a warp, or a block of up to 1024 threads
// with up to 32 elements each), so every operand is read once. Few rows take as many threads as leave each eight
// elements: what counts is the latency of the loads and reductions. Many rows take up to 32 elements a thread; residual and gate wait in shared
// memory (asynchronous copies, each thread's own), so that 80 registers do and three blocks of 256 threads an SM hide each other's reductions.
//
// Alignment. Vectors of eight elements start at 16-byte boundaries. Rows that do not (odd widths) are taken from the boundary before
// them, the same one for all operands as they lie in rows of the same width; their first and last vectors go element by element.
// Operands whose rows lie differently to the boundaries go element by element throughout.
//
// Bound and measured (GB300; 6 786 GB/s is the measured copy bandwidth). HBM for many rows: 16000 x 8192, bfloat16 with a 32-bit stream, a gate of
// each token and both norms 311 us (5 890 GB/s, 87 %), without gate and first norm 232 us (100 %), all of it bfloat16 156 us (99 %). Residual and
// gate in registers from the start (124 of them, two blocks an SM) took 447 us of the first; pieces of 32 bytes a lane instead of 16 for 32-bit streams
// 381 us (each copy took half of a sector). Latency for few: one token 2.8 us in a row of calls in a graph; 192 rows of 8177, layer norm, float16, 8.7 us.

#include <type_traits>

#include "decode_device.cuh"
#include "om_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kVector = 8;  // elements of a thread's load

struct NormArgs {
    NormProblem p;
    int row_warps;        // warps of a row
    int offset, advance;  // elements between a 16-byte boundary and the first row, and from row to row (modulo 8)
    bool stage_gate;      // the gate waits in shared memory too
    bool one_gate;        // the gate is one row for all tokens, read as weights are
};

// Where element e of a thread's vector v lies in its row. Vectors are pieces of PIECE neighbours, neighbouring lanes' pieces side by side: what 16
// bytes of the widest operand hold, so that no copy takes half of a 32-byte sector. kApart: single elements instead.
enum Lie : int { kApart, kEven, kShifted };  // how operands lie to 16-byte boundaries: each differently, on them, all as far off them
template <int PIECE, int LIE>
struct Place {
    int thread, threads, width, shift;  // shift: elements of the first piece that are before the row
    __device__ __forceinline__ int at(int v, int e) const {
        if (LIE == kApart) return (v * kVector + e) * threads + thread;
        return ((v * (kVector / PIECE) + e / PIECE) * threads + thread) * PIECE + e % PIECE - (LIE == kShifted ? shift : 0);
    }
    __device__ __forceinline__ bool inside(int v, int e) const { return static_cast<unsigned>(at(v, e)) < static_cast<unsigned>(width); }
    // the whole piece lies in the row
    __device__ __forceinline__ bool whole(int v, int q) const { return inside(v, q * PIECE) && (LIE == kEven || inside(v, q * PIECE + PIECE - 1)); }
};

// A vector as it is read, two 16-bit elements a word; 0 outside the row.
template <typename T>
struct Held {
    static constexpr int kWords = kVector * sizeof(T) / 4;
    uint32_t w[kWords];
};

// A piece's words between memory and registers: 8 bytes, 16, or 32 (weights of 32 bits) at once.
template <int WORDS>
__device__ __forceinline__ void get_words(const void *from, uint32_t *w, bool there = true) {
    if constexpr (WORDS == 2) {
        const uint2 x = there ? *static_cast<const uint2 *>(from) : make_uint2(0, 0);
        w[0] = x.x; w[1] = x.y;
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) {
            const uint4 x = there ? static_cast<const uint4 *>(from)[i / 4] : make_uint4(0, 0, 0, 0);
            w[i] = x.x; w[i + 1] = x.y; w[i + 2] = x.z; w[i + 3] = x.w;
        }
    }
}
template <int WORDS>
__device__ __forceinline__ void put_words(void *to, const uint32_t *w) {
    if constexpr (WORDS == 2) {
        *static_cast<uint2 *>(to) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int i = 0; i < WORDS; i += 4) static_cast<uint4 *>(to)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
}

template <typename T, int PIECE, int LIE>
__device__ __forceinline__ void load_elements(const T *row, int v, int q, const Place<PIECE, LIE> &l, uint32_t *w) {
    T x[PIECE];
#pragma unroll
    for (int e = 0; e < PIECE; ++e) x[e] = l.inside(v, q * PIECE + e) ? row[l.at(v, q * PIECE + e)] : from_float<T>(0.0f);
    memcpy(w, x, sizeof(x));
}

template <typename T, int PIECE, int LIE>
__device__ __forceinline__ Held<T> load_vector(const T *row, int v, const Place<PIECE, LIE> &l) {
    constexpr int kWords = PIECE * sizeof(T) / 4;
    Held<T> h;
#pragma unroll
    for (int q = 0; q < kVector / PIECE; ++q) {
        uint32_t *const w = h.w + q * kWords;
        if (LIE == kEven || (LIE == kShifted && l.whole(v, q)))
            get_words<kWords>(row + l.at(v, q * PIECE), w, l.whole(v, q));
        else
            load_elements(row, v, q, l, w);
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

template <typename T, int PIECE, int LIE>
__device__ __forceinline__ void store_vector(T *row, int v, const Place<PIECE, LIE> &l, const float *x) {
    constexpr int kWords = PIECE * sizeof(T) / 4;
    T e[kVector];
#pragma unroll
    for (int i = 0; i < kVector; ++i) e[i] = from_float<T>(x[i]);
#pragma unroll
    for (int q = 0; q < kVector / PIECE; ++q) {
        if (LIE != kApart && l.whole(v, q)) {
            uint32_t w[kWords];
            memcpy(w, e + q * PIECE, sizeof(w));
            put_words<kWords>(row + l.at(v, q * PIECE), w);
        } else if (LIE != kEven) {
#pragma unroll
            for (int i = q * PIECE; i < (q + 1) * PIECE; ++i)
                if (l.inside(v, i)) row[l.at(v, i)] = e[i];
        }
    }
}

// A vector on its way to the thread's own place in shared memory, a piece of each thread side by side.
template <typename T, int PIECE, int LIE>
__device__ __forceinline__ void stage_vector(const T *row, int v, const Place<PIECE, LIE> &l, uint8_t *stage) {
    constexpr int kBytes = PIECE * sizeof(T);
#pragma unroll
    for (int q = 0; q < kVector / PIECE; ++q) {
        uint8_t *const to = stage + ((v * (kVector / PIECE) + q) * l.threads + l.thread) * kBytes;
        if (LIE == kEven || l.whole(v, q)) {
            const bool there = l.whole(v, q);
            const T *const from = there ? row + l.at(v, q * PIECE) : row;
            if constexpr (kBytes == 16)
                cp_async_16(smem_u32(to), from, there ? 16 : 0);
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(there ? 8 : 0) : "memory");
        } else {
            uint32_t w[kBytes / 4];
            load_elements(row, v, q, l, w);
            put_words<kBytes / 4>(to, w);
        }
    }
}
template <typename T, int PIECE, int LIE>
__device__ __forceinline__ Held<T> staged_vector(int v, const Place<PIECE, LIE> &l, const uint8_t *stage) {
    constexpr int kBytes = PIECE * sizeof(T);
    Held<T> h;
#pragma unroll
    for (int q = 0; q < kVector / PIECE; ++q) get_words<kBytes / 4>(stage + ((v * (kVector / PIECE) + q) * l.threads + l.thread) * kBytes, h.w + q * kBytes / 4);
    return h;
}

// A vector of weights, of the activations' type or 32 bits; rows that start off a boundary read them element by element.
template <typename T, int PIECE, int LIE>
__device__ __forceinline__ Held<T> load_weight(const T *w, int v, const Place<PIECE, LIE> &l) {
    if (LIE != kShifted || l.shift == 0) return load_vector(w, v, l);
    Held<T> h;
#pragma unroll
    for (int q = 0; q < kVector / PIECE; ++q) load_elements(w, v, q, l, h.w + q * static_cast<int>(PIECE * sizeof(T) / 4));
    return h;
}
template <typename T, int PIECE, int LIE>
__device__ __forceinline__ void load_weights(const void *w, bool wide, int v, const Place<PIECE, LIE> &l, float *x) {
    if (std::is_same_v<T, float> || wide)
        expand(load_weight(static_cast<const float *>(w), v, l), x);
    else
        expand(load_weight(static_cast<const T *>(w), v, l), x);
}

// The sums of N values over a row's threads, in one order whatever the timing. held: of this use alone.
template <int N>
__device__ __forceinline__ void row_sum(float (&x)[N], int row_warps, float (*held)[32]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __fadd_rn(x[i], __shfl_xor_sync(0xffffffffu, x[i], o));
    if (row_warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) held[i][threadIdx.x / 32] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = (threadIdx.x & 31) < row_warps ? held[i][threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __fadd_rn(x[i], __shfl_xor_sync(0xffffffffu, x[i], o));
}

// x <- N(x). Elements outside the row are 0 and stay out of the sums.
template <typename T, int V, int PIECE, int LIE>
__device__ __forceinline__ void normalise(float (&x)[V][kVector], const NormProblem &p, const void *weight, const void *bias, const Place<PIECE, LIE> &l, int row_warps,
                                          float (*held)[32]) {
    const float count = static_cast<float>(l.width);
    const bool wide = p.weight_dtype == OM_F32;
    auto inverse = [&](float variance) { return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(variance, p.eps))); };
    float inv;
    if (p.layer) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) sum[0] = __fadd_rn(sum[0], x[v][e]);
        row_sum(sum, row_warps, held);
        const float mean = __fdiv_rn(sum[0], count);
        float left[2] = {0.0f, 0.0f};  // what the differences add up to, and their squares
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) {
                x[v][e] = l.inside(v, e) ? __fsub_rn(x[v][e], mean) : 0.0f;
                left[0] = __fadd_rn(left[0], x[v][e]);
                left[1] = __fmaf_rn(x[v][e], x[v][e], left[1]);
            }
        row_sum(left, row_warps, held + 1);
        const float rest = __fdiv_rn(left[0], count), variance = __fmaf_rn(-rest, rest, __fdiv_rn(left[1], count));
        inv = inverse(variance < 0.0f ? 0.0f : variance);  // NaN stays
        const float shift = __fmul_rn(-rest, inv);  // (x - rest) inv = x inv + shift
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fmaf_rn(x[v][e], inv, shift);
        if (!weight)  // which are 0 outside the row
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < kVector; ++e) x[v][e] = l.inside(v, e) ? x[v][e] : 0.0f;
    } else {
        float squares[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) squares[0] = __fmaf_rn(x[v][e], x[v][e], squares[0]);
        row_sum(squares, row_warps, held);
        inv = inverse(__fdiv_rn(squares[0], count));
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fmul_rn(x[v][e], inv);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float w[kVector];
        if (weight) {
            load_weights<T>(weight, wide, v, l, w);
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fmul_rn(x[v][e], w[e]);
        }
        if (bias) {
            load_weights<T>(bias, wide, v, l, w);
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fadd_rn(x[v][e], w[e]);
        }
    }
}

// 1 / (1 + e^-g) within 2^-21: e^-g = 2^h (1 + l ln 2) with h + l = -g log2(e), the product's rounding in l; both approximate instructions are
// within 2^-22. Factors of gates below -87, which leave the range of 32 bits, are 0.
__device__ __forceinline__ float gate_factor(float g, int activation) {
    if (activation == OM_GATE_NONE) return g;
    const float c = g > 88.0f ? 88.0f : (g < -87.0f ? -87.0f : g);  // NaN stays
    constexpr float kHigh = 1.44269502f, kLow = 1.92596303e-8f;     // log2(e)
    const float h = __fmul_rn(-c, kHigh), l = __fmaf_rn(-c, kLow, __fmaf_rn(-c, kHigh, -h));
    float e, t;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(h));
    e = __fmaf_rn(e, __fmul_rn(l, 0.693147182f), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(__fadd_rn(1.0f, e)));
    if (g < -87.0f) return 0.0f;
    return activation == OM_GATE_SIGMOID ? t : __fmul_rn(g, t);
}

template <typename T, typename R, int V, int THREADS, int LIE>
__global__ void __launch_bounds__(THREADS, LIE == kApart ? 1 : (THREADS == 256 ? 3 : 1024 / THREADS)) block_norm_kernel(const __grid_constant__ NormArgs a) {
    const NormProblem &p = a.p;
    constexpr bool kStaged = LIE != kApart && V == 4;  // residual and gate wait in shared memory
    constexpr int kPiece = 16 / sizeof(R);
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ float held[6][32];  // the warps' parts of each sum
    const int64_t row = a.row_warps == 1 ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
    const Place<kPiece, LIE> l{a.row_warps == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x), a.row_warps * 32, static_cast<int>(p.width),
                               LIE == kShifted ? (a.offset + static_cast<int>(row & 7) * a.advance) & 7 : 0};
    const int own = l.threads * V * kVector;  // elements of a row's place
    uint8_t *const r_stage = stage + (a.row_warps == 1 ? threadIdx.x / 32 * own * (sizeof(R) + sizeof(T)) : 0);
    uint8_t *const g_stage = r_stage + (p.residual ? own * sizeof(R) : 0);
    wait_for_earlier();
    if (row >= p.tokens) return;  // a warp that has a row of its own, never a part of a block that shares one
    const T *const y_row = static_cast<const T *>(p.y) + row * p.ldy, *const g_row = static_cast<const T *>(p.gate) + row * p.ldg;
    const R *const r_row = static_cast<const R *>(p.residual) + row * p.ldr;
    Held<T> y[V], g[kStaged ? 1 : V];
    Held<R> r[kStaged ? 1 : V];
    // all of the row's operands are on their way together
#pragma unroll
    for (int v = 0; v < V; ++v) y[v] = load_vector(y_row, v, l);
    if constexpr (kStaged) {
        if (p.residual) {
#pragma unroll
            for (int v = 0; v < V; ++v) stage_vector(r_row, v, l, r_stage);
        }
        if (a.stage_gate) {
#pragma unroll
            for (int v = 0; v < V; ++v) stage_vector(g_row, v, l, g_stage);
        }
    } else {
        if (p.residual) {
#pragma unroll
            for (int v = 0; v < V; ++v) r[v] = load_vector(r_row, v, l);
        }
        if (p.gate) {
#pragma unroll
            for (int v = 0; v < V; ++v) g[v] = a.one_gate ? load_weight(g_row, v, l) : load_vector(g_row, v, l);
        }
    }
    float x[V][kVector];
#pragma unroll
    for (int v = 0; v < V; ++v) expand(y[v], x[v]);
    if (p.post) normalise<T>(x, p, p.post_weight, p.post_bias, l, a.row_warps, held);
    if constexpr (kStaged) cp_async_wait_all();  // a thread's own copies
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float f[kVector];
        if (p.gate) {
            if constexpr (kStaged)
                expand(a.stage_gate ? staged_vector<T>(v, l, g_stage) : (a.one_gate ? load_weight(g_row, v, l) : load_vector(g_row, v, l)), f);
            else
                expand(g[v], f);
#pragma unroll
            for (int e = 0; e < kVector; ++e) x[v][e] = __fmul_rn(x[v][e], gate_factor(f[e], p.activation));
        }
        if (p.residual) {
            if constexpr (kStaged)
                expand(staged_vector<R>(v, l, r_stage), f);
            else
                expand(r[v], f);
        }
#pragma unroll
        for (int e = 0; e < kVector; ++e) x[v][e] = p.residual ? __fmaf_rn(p.scale, x[v][e], f[e]) : __fmul_rn(p.scale, x[v][e]);
    }
    if (p.sum) {
#pragma unroll
        for (int v = 0; v < V; ++v) store_vector(static_cast<R *>(p.sum) + row * p.lds, v, l, x[v]);
    }
    if (!p.out) return;
    normalise<T>(x, p, p.weight, p.bias, l, a.row_warps, held + 3);
#pragma unroll
    for (int v = 0; v < V; ++v) store_vector(static_cast<T *>(p.out) + row * p.ldo, v, l, x[v]);
}

constexpr int kMostStage = 200 * 1024;

template <typename T, typename R, int V, int THREADS, int LIE>
cudaError_t launch(NormArgs a, cudaStream_t s) {
    const int rows = a.row_warps == 1 ? 4 : 1;  // of a block
    const dim3 grid(static_cast<unsigned>((a.p.tokens + rows - 1) / rows)), block(32 * a.row_warps * rows);
    int stage = 0;
    if (LIE != kApart && V == 4) {
        const int elements = static_cast<int>(block.x) * V * kVector, r = elements * static_cast<int>(sizeof(R)), g = elements * static_cast<int>(sizeof(T));
        a.stage_gate = a.p.gate && !a.one_gate && r + g <= kMostStage;
        // a block of several rows has a place for both of them in each
        stage = rows > 1 ? r + g : (a.p.residual ? r : 0) + (a.stage_gate ? g : 0);
        static PerDevice ready;
        std::atomic<int> *const kept = ready.here();
        if (!kept || kept->load(std::memory_order_relaxed) == 0) {
            const cudaError_t e = cudaFuncSetAttribute(block_norm_kernel<T, R, V, THREADS, LIE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostStage);
            if (e != cudaSuccess) return e;
            if (kept) kept->store(1, std::memory_order_relaxed);
        }
    }
    return launch_behind(block_norm_kernel<T, R, V, THREADS, LIE>, grid, block, stage, s, a);
}

template <typename T, typename R, int LIE>
cudaError_t by_width(const NormProblem &p, int offset, int advance, cudaStream_t s) {
    // a row that starts off a boundary can take a vector more
    const int64_t vectors = (p.width + kVector - 1) / kVector + (LIE == kShifted);
    auto warps = [&](int v) { return static_cast<int>((vectors + 32 * v - 1) / (32 * v)); };
    auto args = [&](int v) { return NormArgs{p, warps(v), offset, advance, false, p.tokens > 1 && p.ldg == 0}; };
    // eight elements a thread where all rows are in flight at once (153 rows of 4096: 3.1 us, with 32 elements 4.8; 192 of 8177, which are not: 8.3 with 32, 9.7 with eight)
    if ((warps(1) <= 32 && p.tokens * warps(1) <= 36 * num_sms()) || warps(1) == 1) return launch<T, R, 1, 1024, LIE>(args(1), s);
    if (warps(2) == 1) return launch<T, R, 2, 512, LIE>(args(2), s);
    if (warps(4) <= 8) return launch<T, R, 4, 256, LIE>(args(4), s);
    if (warps(4) <= 16) return launch<T, R, 4, 512, LIE>(args(4), s);
    if (warps(4) <= 32) return launch<T, R, 4, 1024, LIE>(args(4), s);
    return launch<T, R, 4, 1024, kApart>(NormArgs{p, static_cast<int>((p.width + 1023) / 1024), 0, 0, false, false}, s);  // the widest rows off their boundaries
}

template <typename T, typename R>
cudaError_t by_alignment(const NormProblem &p, cudaStream_t s) {
    // elements from a 16-byte boundary to the operands' first rows and from row to row; vectors where all of them agree
    const int offset = static_cast<int>(reinterpret_cast<uintptr_t>(p.y) / sizeof(T) % kVector), advance = p.tokens > 1 ? static_cast<int>(p.ldy % kVector) : 0;
    auto alike = [&](const void *x, int64_t ld, int64_t bytes) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(x);
        return !x || (static_cast<int>(at / bytes % kVector) == offset && (p.tokens == 1 || static_cast<int>(ld % kVector) == advance));
    };
    auto aligned = [&](const void *x) { return reinterpret_cast<uintptr_t>(x) % 16 == 0; };
    // weights, and a gate of one row, are read by vectors where a row starts on a boundary
    const bool vectors = alike(p.residual, p.ldr, sizeof(R)) && (p.tokens > 1 && p.ldg == 0 ? aligned(p.gate) : alike(p.gate, p.ldg, sizeof(T))) && alike(p.sum, p.lds, sizeof(R)) && alike(p.out, p.ldo, sizeof(T)) &&
                         aligned(p.weight) && aligned(p.bias) && aligned(p.post_weight) && aligned(p.post_bias);
    if (!vectors) return by_width<T, R, kApart>(p, 0, 0, s);
    if (offset == 0 && advance == 0 && p.width % kVector == 0) return by_width<T, R, kEven>(p, 0, 0, s);
    return by_width<T, R, kShifted>(p, offset, advance, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormProblem &p, cudaStream_t s) {
    if (p.dtype == OM_F32) return by_alignment<float, float>(p, s);
    if (p.dtype == OM_F16) return p.stream_dtype == OM_F32 ? by_alignment<__half, float>(p, s) : by_alignment<__half, __half>(p, s);
    return p.stream_dtype == OM_F32 ? by_alignment<__nv_bfloat16, float>(p, s) : by_alignment<__nv_bfloat16, __nv_bfloat16>(p, s);
}

}  // namespace om
