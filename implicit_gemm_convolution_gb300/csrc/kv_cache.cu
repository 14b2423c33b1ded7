// kv_cache.cu -- the paged 8-bit cache: appending rotated keys and values,
// reading tokens back as values, and the rotation table.
//
// A page holds `page` tokens of every head, [head][token][dim] codes, and one
// 32-bit scale per head for its keys and one for its values; a value is
// code * scale. Every step of the append is one separately rounded binary32
// operation (the library is built without contraction), so codes, scales and
// rotated queries have one bit pattern each, whatever the launch.
//
// Bound and measured (GB300; 6 790 GB/s is the measured copy bandwidth): HBM. Prompts of 12031 tokens in all, 32 query
// and 8 key heads of 128, 32-bit: 93 us for 525 MB (5 600 GB/s, 83 %). Reading 76166 tokens of 8 heads of 128 back as
// bfloat16: 79 us, 5 930 GB/s (87 %); with 16-byte loads whose lanes stored 32 or 64 bytes each it took 108 us. One
// token for each of 192 sequences: 15 us, the latency of the lookups, the page's old codes and its barrier.

#include <type_traits>

#include "decode_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kThreads = 128;

// Eight elements of one head's row: unit u of the rotated part holds the four
// pairs 4u .. 4u+3, later units eight consecutive elements behind it. *second
// is the offset of elements 4..7.
__device__ __forceinline__ int unit_offset(int u, int rot, bool interleaved, int *second) {
    if (8 * u < rot && !interleaved) {
        *second = rot / 2 + 4 * u;
        return 4 * u;
    }
    *second = 8 * u + 4;
    return 8 * u;
}

// The table's cos and sin of unit u's four pairs at position pos; NaN for positions the table does not hold.
__device__ __forceinline__ void load_turn(float *cs, const float *table, int64_t rows, int rot, int64_t pos, int u) {
    if (pos >= 0 && pos < rows) {
        const float4 *t = reinterpret_cast<const float4 *>(table + pos * rot + 8 * u);
        const float4 lo = __ldg(t), hi = __ldg(t + 1);
        cs[0] = lo.x; cs[1] = lo.y; cs[2] = lo.z; cs[3] = lo.w;
        cs[4] = hi.x; cs[5] = hi.y; cs[6] = hi.z; cs[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = __int_as_float(0x7FC00000);
    }
}

__device__ __forceinline__ void turn_pair(float &a, float &b, float c, float s) {
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Turns the four pairs of a unit: (a, b) -> (a c - b s, b c + a s), every product and sum rounded.
__device__ __forceinline__ void turn(float *v, const float *cs, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_pair(v[2 * i], v[2 * i + 1], cs[2 * i], cs[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) turn_pair(v[i], v[4 + i], cs[2 * i], cs[2 * i + 1]);
    }
}

struct AppendArgs {
    KvAppendProblem p;
    int64_t slots;         // pages a sequence's new tokens can touch
    int64_t cache_blocks;  // blocks that write the cache; the others rotate queries
    int tokens;            // that such a block takes
};

// One block per (page the new tokens touch, head, keys or values): the page's
// largest new magnitude first, then its scale, its old codes under the new scale and
// its new codes. No two blocks write the same page and head, so there is
// nothing to order between them. A thread keeps its first four units in registers in between.
template <typename T, int KV, bool ALIGNED>
__device__ void append_page(const AppendArgs &a, int64_t block) {
    constexpr int kKept = 4;
    const KvAppendProblem &p = a.p;
    const int kind = static_cast<int>(block & 1);
    const int64_t heads = p.c.heads, page = p.c.page;
    const int dim = static_cast<int>(p.c.dim), per_row = dim / 8, row_log = 31 - __clz(per_row);
    const int64_t h = (block >> 1) % heads, slot = (block >> 1) / heads;
    const int64_t b = slot / a.slots, j = slot % a.slots;
    int64_t t0, t1;
    token_range(p.cu, b, p.tokens, &t0, &t1);
    const int64_t ctx = p.ctx[b], start = ctx - (t1 - t0);
    if (t1 == t0 || ctx <= 0) return;
    const int64_t pidx = (start > 0 ? start / page : 0) + j, p_lo = pidx * page;
    if (p_lo >= ctx || pidx >= p.width) return;
    const int64_t id = p.block_table[b * p.width + pidx];
    const int64_t lo = start > p_lo ? start : p_lo, hi = ctx < p_lo + page ? ctx : p_lo + page;
    const int had = static_cast<int>(lo - p_lo);
    const int units = static_cast<int>(hi - lo) * per_row;

    const Heads &src = kind ? p.v : p.k;
    const int rot = kind ? 0 : static_cast<int>(p.rot);
    const bool inter = p.interleaved != 0;
    const T *rows = static_cast<const T *>(src.p) + (t0 + lo - start) * src.ts + h * src.hs;
    auto load = [&](int i, float *v) {  // unit i, rotated
        const int t = i >> row_log, u = i & (per_row - 1);
        int second;
        const int first = unit_offset(u, rot, inter, &second);
        load4<T, ALIGNED>(rows + t * src.ts + first, v);
        load4<T, ALIGNED>(rows + t * src.ts + second, v + 4);
        if (8 * u < rot) {
            float cs[8];
            load_turn(cs, p.table, p.rows, rot, lo + t, u);
            turn(v, cs, inter);
        }
    };
    // magnitudes compare as their bits: a NaN is above infinity, which is
    // above every finite value
    unsigned top = 0;
    float kept[kKept][8];
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < units) load(i, kept[k]);
    }
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (static_cast<int>(threadIdx.x) + k * kThreads < units)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(kept[k][e]) & 0x7fffffffu);
#pragma unroll 1
    for (int i = threadIdx.x + kKept * kThreads; i < units; i += kThreads) {
        float v[8];
        load(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    if (id < 0 || id >= p.c.pages) return;  // by the whole block
    float *scale = (kind ? p.c.v_scale : p.c.k_scale) + id * heads + h;
    uint8_t *codes = static_cast<uint8_t *>(kind ? p.c.v : p.c.k) + (id * heads + h) * page * dim;
    const float old = had > 0 ? fabsf(*scale) : 0.0f;
    // old codes, in case the scale grows: their load's latency is beside the scale's
    uint4 *const old_codes = reinterpret_cast<uint4 *>(codes);
    const int old_words = had * dim / 16;
    uint4 ahead[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (static_cast<int>(threadIdx.x) + k * kThreads < old_words) ahead[k] = old_codes[threadIdx.x + k * kThreads];

    __shared__ unsigned warp_top[kThreads / 32];
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, warp_top[w]);

    // A page with a value that is not finite gets the scale NaN and codes 0:
    // every read of it shows.
    const float want = __fmul_rn(__uint_as_float(top), KV == OM_I8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    const bool finite = top < 0x7f800000u && __float_as_uint(old) < 0x7f800000u;
    const float grown = finite ? fmaxf(old, want) : __int_as_float(0x7FC00000);
    if (threadIdx.x == 0) *scale = grown;  // every thread has read the old one: the barrier above

    if (had > 0 && (grown != old || !finite)) {
        const float ratio = finite ? __fdiv_rn(old, grown) : 0.0f;  // grown > old >= 0
        auto rescale = [&](int i, uint4 w4) {
            uint32_t *w = &w4.x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float v[4];
                decode4<KV>(w[q], v);
                w[q] = finite ? encode4<KV>(__fmul_rn(v[0], ratio), __fmul_rn(v[1], ratio), __fmul_rn(v[2], ratio), __fmul_rn(v[3], ratio)) : 0;
            }
            old_codes[i] = w4;
        };
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (static_cast<int>(threadIdx.x) + k * kThreads < old_words) rescale(threadIdx.x + k * kThreads, ahead[k]);
#pragma unroll 1
        for (int i = threadIdx.x + 2 * kThreads; i < old_words; i += kThreads) rescale(i, old_codes[i]);
    }
    auto store = [&](int i, const float *v) {
        const int t = i >> row_log;
        int second;
        const int first = unit_offset(i & (per_row - 1), rot, inter, &second);
        uint32_t w[2] = {0, 0};
        if (finite && grown > 0.0f) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                w[e] = encode4<KV>(__fdiv_rn(v[4 * e], grown), __fdiv_rn(v[4 * e + 1], grown), __fdiv_rn(v[4 * e + 2], grown), __fdiv_rn(v[4 * e + 3], grown));
        }
        uint8_t *dst = codes + (had + t) * dim;
        *reinterpret_cast<uint32_t *>(dst + first) = w[0];
        *reinterpret_cast<uint32_t *>(dst + second) = w[1];
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i < units) store(i, kept[k]);
    }
#pragma unroll 1
    for (int i = threadIdx.x + kKept * kThreads; i < units; i += kThreads) {
        float v[8];
        load(i, v);
        store(i, v);
    }
}

// The sequence of each of a block's `count` tokens t, t + 1, ..., and their offset in it (-1: none), in
// shared memory; every thread of the block takes part.
constexpr int kMostTokens = 32;
struct Places {
    int seq[kMostTokens];
    int64_t at[kMostTokens];
};
__device__ __forceinline__ void find_tokens(Places *places, const int32_t *cu, int64_t seqs, int64_t tokens, int64_t t, int count) {
    for (int i = threadIdx.x; i < count; i += blockDim.x) {
        places->seq[i] = 0;
        places->at[i] = -1;
    }
    __syncthreads();
    // a sequence that overlaps the block's tokens writes its own
    for (int64_t b = threadIdx.x; b < seqs; b += blockDim.x) {
        int64_t lo, hi;
        token_range(cu, b, tokens, &lo, &hi);
        for (int64_t i = max(lo, t); i < min(hi, t + count); ++i) {
            places->seq[i - t] = static_cast<int>(b);
            places->at[i - t] = i - lo;
        }
    }
    __syncthreads();
}

// Some tokens' queries; four units of a thread in flight.
template <typename T, bool ALIGNED>
__device__ void rotate_queries(const AppendArgs &a, int64_t block) {
    const KvAppendProblem &p = a.p;
    const int dim = static_cast<int>(p.c.dim), rot = static_cast<int>(p.rot), per_row = dim / 8;
    const int64_t t = block * a.tokens;
    const int count = static_cast<int>(min(static_cast<int64_t>(a.tokens), p.tokens - t));
    __shared__ Places places;
    find_tokens(&places, p.cu, p.seqs, p.tokens, t, count);
    const bool inter = p.interleaved != 0;
    // a token that no sequence owns has no position: its queries become NaN
    if (threadIdx.x < count) {
        const int64_t at = places.at[threadIdx.x], b = places.seq[threadIdx.x];
        int64_t lo, hi;
        token_range(p.cu, b, p.tokens, &lo, &hi);
        places.at[threadIdx.x] = at < 0 ? -1 : static_cast<int64_t>(p.ctx[b]) - (hi - lo) + at;
    }
    __syncthreads();
    const int units = static_cast<int>(p.q_heads) * per_row, row_log = 31 - __clz(per_row);
    constexpr int kAhead = 4;
#pragma unroll 1
    for (int tok = 0; tok < count; ++tok) {
        const T *const src = static_cast<const T *>(p.q.p) + (t + tok) * p.q.ts;
        T *const dst = static_cast<T *>(const_cast<void *>(p.q_out.p)) + (t + tok) * p.q_out.ts;
        const int64_t pos = places.at[tok];
#pragma unroll 1
        for (int base = threadIdx.x; base < units; base += kAhead * kThreads) {
            float v[kAhead][8];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = base + k * kThreads, u = i & (per_row - 1);
                if (i >= units) break;
                int second;
                const int first = unit_offset(u, rot, inter, &second);
                const T *const row = src + (i >> row_log) * p.q.hs;
                load4<T, ALIGNED>(row + first, v[k]);
                load4<T, ALIGNED>(row + second, v[k] + 4);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = base + k * kThreads, u = i & (per_row - 1);
                if (i >= units) break;
                int second;
                const int first = unit_offset(u, rot, inter, &second);
                if (8 * u < rot) {
                    float cs[8];
                    load_turn(cs, p.table, p.rows, rot, pos, u);
                    turn(v[k], cs, inter);
                }
                T *const row = dst + (i >> row_log) * p.q_out.hs;
                store4<T, ALIGNED>(row + first, v[k]);
                store4<T, ALIGNED>(row + second, v[k] + 4);
            }
        }
    }
}

template <typename T, int KV, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    wait_for_earlier();
    const int64_t block = blockIdx.x;
    if (block < a.cache_blocks)
        append_page<T, KV, ALIGNED>(a, block);
    else
        rotate_queries<T, ALIGNED>(a, block - a.cache_blocks);
}

struct ReadArgs {
    KvReadProblem p;
    int tokens;  // of a block
    int slice;   // 16-byte pieces of codes of a round, a power of two
};

// Some tokens, in rounds of up to 32 KB of codes: all of a round's copies into shared memory are in flight together
// (neighbouring tokens of one head after the other, as they lie in the cache); then neighbouring lanes
// store neighbouring 16 bytes of values.
constexpr int kReadThreads = 256, kMostSlice = 2048;
template <typename T, int KV>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const __grid_constant__ ReadArgs a) {
    const KvReadProblem &p = a.p;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * a.tokens, page = p.c.page;
    const int heads = static_cast<int>(p.c.heads), dim = static_cast<int>(p.c.dim);
    const int count = static_cast<int>(min(static_cast<int64_t>(a.tokens), p.tokens - t));
    extern __shared__ __align__(16) uint8_t held[];
    __shared__ Places places;
    __shared__ int ids[kMostTokens], rows[kMostTokens];
    __shared__ float scales[kMostSlice / 4];  // of the rows of a round
    wait_for_earlier();
    find_tokens(&places, p.cu, p.seqs, p.tokens, t, count);
    if (threadIdx.x < kMostTokens) {
        int64_t id = -1, pos = -1;
        if (threadIdx.x < count) {
            const int64_t at = places.at[threadIdx.x], b = places.seq[threadIdx.x];
            if (at >= 0) {
                pos = p.start[b] + at;
                if (pos >= 0 && pos / page < p.width) id = p.block_table[b * p.width + pos / page];
                if (id >= p.c.pages || id < 0) id = -1;
            }
        }
        ids[threadIdx.x] = static_cast<int>(id);
        rows[threadIdx.x] = id < 0 ? 0 : static_cast<int>(pos % page);
    }
    __syncthreads();
    // piece i: of (keys or values, head, token, place in the row); powers of two but for the heads
    const int row_log = 31 - __clz(dim / 16), head_log = row_log + 31 - __clz(a.tokens), pieces = 2 * heads << head_log;
    for (int first = 0; first < pieces; first += a.slice) {
        const int many = min(a.slice, pieces - first);
        for (int i = threadIdx.x; i < many; i += kReadThreads) {
            const int q = first + i, kh = q >> head_log, tok = (q >> row_log) & (a.tokens - 1), h = kh >= heads ? kh - heads : kh;
            const int64_t at = static_cast<int64_t>(ids[tok]) * heads + h;
            if (ids[tok] >= 0) {
                const uint8_t *const src = static_cast<const uint8_t *>(kh >= heads ? p.c.v : p.c.k) + (at * page + rows[tok]) * dim + (q & ((1 << row_log) - 1)) * 16;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(held)) + i * 16), "l"(src) : "memory");
            } else {
                reinterpret_cast<uint4 *>(held)[i] = make_uint4(0, 0, 0, 0);
            }
            // a position the cache does not hold reads as NaN
            if ((q & ((1 << row_log) - 1)) == 0) scales[i >> row_log] = ids[tok] >= 0 ? (kh >= heads ? p.c.v_scale : p.c.k_scale)[at] : __int_as_float(0x7FC00000);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        constexpr int kCodes = 16 / sizeof(T), kPer = 16 / kCodes;  // values of a store; stores of a piece
#pragma unroll 4
        for (int i = threadIdx.x; i < many * kPer; i += kReadThreads) {
            const int q = first + i / kPer, kh = q >> head_log, tok = (q >> row_log) & (a.tokens - 1), h = kh >= heads ? kh - heads : kh;
            if (tok >= count) continue;
            uint32_t w[kCodes / 4];
            memcpy(w, held + i * kCodes, kCodes);
            const float scale = scales[(i / kPer) >> row_log];
            float v[kCodes];
#pragma unroll
            for (int j = 0; j < kCodes / 4; ++j) decode4<KV>(w[j], v + 4 * j);
            T e[kCodes];
#pragma unroll
            for (int j = 0; j < kCodes; ++j) e[j] = from_float<T>(__fmul_rn(v[j], scale));
            uint4 o;
            memcpy(&o, e, 16);
            T *out = static_cast<T *>(kh >= heads ? p.v_out : p.k_out) + ((t + tok) * heads + h) * dim + (q & ((1 << row_log) - 1)) * 16 + i % kPer * kCodes;
            __stcs(reinterpret_cast<uint4 *>(out), o);
        }
        __syncthreads();
    }
}

// Row r of the table: cos and sin of r * frequency, evaluated in 64 bits and rounded
// once. Frequency i is base^(-2i/rot), then scaled for contexts longer than
// `original`: linear divides all by factor; ntk raises the base to
// base * factor^(rot / (rot - 2)); yarn divides those that turn fewer than beta_slow
// times in `original` positions, keeps those that turn more than beta_fast
// times, blends linearly between (in the pair index) and multiplies cos and sin by
// 0.1 ln(factor) + 1.
__global__ void __launch_bounds__(kThreads)
    rope_table_kernel(int64_t rows, int64_t rot, double base, int scaling, double factor,
                      double original, double beta_fast, double beta_slow, float *table) {
    const int64_t half = rot / 2, i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= rows * half) return;
    const int64_t r = i / half, e = i % half;
    double b = base, amp = 1.0;
    if (scaling == OM_ROPE_NTK && rot > 2) b = base * pow(factor, static_cast<double>(rot) / (rot - 2));
    double f = pow(b, -2.0 * e / rot);
    if (scaling == OM_ROPE_LINEAR) f /= factor;
    if (scaling == OM_ROPE_YARN) {
        constexpr double kTwoPi = 6.283185307179586476925;
        // the pair index that turns beta times in `original` positions
        const double lnb = log(base);
        double lo = floor(rot * log(original / (beta_fast * kTwoPi)) / (2.0 * lnb));
        double hi = ceil(rot * log(original / (beta_slow * kTwoPi)) / (2.0 * lnb));
        lo = fmax(lo, 0.0);
        hi = fmin(hi, rot - 1.0);
        if (lo == hi) hi += 0.001;
        const double ramp = fmin(fmax((e - lo) / (hi - lo), 0.0), 1.0);
        f = f / factor * ramp + f * (1.0 - ramp);
        if (factor > 1.0) amp = 0.1 * log(factor) + 1.0;
    }
    double s, c;
    sincos(r * f, &s, &c);
    table[2 * i] = static_cast<float>(c * amp);
    table[2 * i + 1] = static_cast<float>(s * amp);
}

template <typename T, int KV>
cudaError_t append_typed(const AppendArgs &a, bool aligned, int64_t blocks, cudaStream_t s) {
    return launch_behind(aligned ? kv_append_kernel<T, KV, true> : kv_append_kernel<T, KV, false>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, a);
}

template <typename T>
cudaError_t append_codes(const AppendArgs &a, bool aligned, int64_t blocks, cudaStream_t s) {
    return a.p.c.dtype == OM_I8 ? append_typed<T, OM_I8>(a, aligned, blocks, s)
                                : append_typed<T, OM_E4M3>(a, aligned, blocks, s);
}

template <typename T>
cudaError_t read_codes(const ReadArgs &a, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((a.p.tokens + a.tokens - 1) / a.tokens);
    return launch_behind(a.p.c.dtype == OM_I8 ? kv_read_kernel<T, OM_I8> : kv_read_kernel<T, OM_E4M3>, dim3(grid), dim3(kReadThreads), a.slice * 16, s, a);
}

// Tokens of a block: as many as leave every SM several blocks.
int tokens_of_block(int64_t tokens, int most) {
    int n = 1;
    while (n < most && tokens >= int64_t(n) * 2 * 8 * num_sms()) n *= 2;
    return n;
}

// Groups of four elements start on their own size's boundary in every row.
bool heads_aligned(const Heads &x, int64_t heads, int bytes) {
    return reinterpret_cast<uintptr_t>(x.p) % (4 * bytes) == 0 && x.ts % 4 == 0 && (heads == 1 || x.hs % 4 == 0);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendProblem &p, cudaStream_t s) {
    AppendArgs a{p, 0, 0, tokens_of_block(p.tokens, 8)};
    const int64_t most = p.max_new < p.tokens ? p.max_new : p.tokens;
    a.slots = (most + p.c.page - 2) / p.c.page + 1;
    a.cache_blocks = p.seqs * a.slots * p.c.heads * 2;
    const int64_t blocks = a.cache_blocks + (p.q_heads > 0 ? (p.tokens + a.tokens - 1) / a.tokens : 0);
    const int bytes = p.dtype == OM_F32 ? 4 : 2;
    const bool aligned = heads_aligned(p.k, p.c.heads, bytes) && heads_aligned(p.v, p.c.heads, bytes) &&
                         (p.q_heads == 0 || (heads_aligned(p.q, p.q_heads, bytes) && heads_aligned(p.q_out, p.q_heads, bytes)));
    if (p.dtype == OM_F32) return append_codes<float>(a, aligned, blocks, s);
    if (p.dtype == OM_F16) return append_codes<__half>(a, aligned, blocks, s);
    return append_codes<__nv_bfloat16>(a, aligned, blocks, s);
}

cudaError_t launch_kv_read(const KvReadProblem &p, cudaStream_t s) {
    ReadArgs a{p, tokens_of_block(p.tokens, kMostTokens), 1};
    const int64_t row = p.c.dim / 16, pieces = 2 * p.c.heads * row * a.tokens;
    while (a.slice < kMostSlice && (a.slice < pieces || a.slice < row)) a.slice *= 2;
    if (p.dtype == OM_F32) return read_codes<float>(a, s);
    if (p.dtype == OM_F16) return read_codes<__half>(a, s);
    return read_codes<__nv_bfloat16>(a, s);
}

cudaError_t launch_rope_table(int64_t rows, int64_t rot, double base, int scaling, double factor,
                              double original, double beta_fast, double beta_slow, float *table,
                              cudaStream_t s) {
    const int64_t blocks = (rows * (rot / 2) + kThreads - 1) / kThreads;
    rope_table_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(rows, rot, base, scaling, factor, original,
                                                                        beta_fast, beta_slow, table);
    return cudaGetLastError();
}

}  // namespace om
