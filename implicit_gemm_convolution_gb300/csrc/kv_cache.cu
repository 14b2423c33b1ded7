// kv_cache.cu -- the paged 8-bit cache: appending rotated keys and values,
// reading tokens back as values, and the rotation table.
//
// A page holds `page` tokens of every head, [head][token][dim] codes, and one
// 32-bit scale per head for its keys and one for its values; a value is
// code * scale. Every step of the append is one separately rounded binary32
// operation (the library is built without contraction), so codes, scales and
// rotated queries have one bit pattern each, whatever the launch.

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

// Rotates the four pairs of unit u by the table row of position pos:
// (a, b) -> (a c - b s, b c + a s), every product and sum rounded. Positions
// the table does not hold give NaN.
__device__ __forceinline__ void rotate_unit(float *v, const float *table, int64_t rows, int rot,
                                            bool interleaved, int64_t pos, int u) {
    if (8 * u >= rot) return;
    float cs[8];
    if (pos >= 0 && pos < rows) {
        const float4 *t = reinterpret_cast<const float4 *>(table + pos * rot + 8 * u);
        const float4 lo = __ldg(t), hi = __ldg(t + 1);
        cs[0] = lo.x; cs[1] = lo.y; cs[2] = lo.z; cs[3] = lo.w;
        cs[4] = hi.x; cs[5] = hi.y; cs[6] = hi.z; cs[7] = hi.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) cs[i] = __int_as_float(0x7FC00000);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float &a = interleaved ? v[2 * i] : v[i];
        float &b = interleaved ? v[2 * i + 1] : v[4 + i];
        const float c = cs[2 * i], s = cs[2 * i + 1], x = a, y = b;
        a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
        b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    }
}

struct AppendArgs {
    KvAppendProblem p;
    int64_t slots;         // pages a sequence's new tokens can touch
    int64_t cache_blocks;  // blocks that write the cache; the others rotate queries, one token each
};

template <typename T, bool ALIGNED>
__device__ __forceinline__ void load_unit(const T *row, int first, int second, float *v) {
    load4<T, ALIGNED>(row + first, v);
    load4<T, ALIGNED>(row + second, v + 4);
}

// One block per (page the new tokens touch, head, keys or values): the page's
// largest new magnitude first, then its scale, its old codes under the new scale and
// its new codes. No two blocks write the same page and head, so there is
// nothing to order between them.
template <typename T, int KV, bool ALIGNED>
__device__ void append_page(const AppendArgs &a, int64_t block) {
    const KvAppendProblem &p = a.p;
    const int kind = static_cast<int>(block & 1);
    const int64_t heads = p.c.heads, page = p.c.page;
    const int dim = static_cast<int>(p.c.dim);
    const int64_t h = (block >> 1) % heads, slot = (block >> 1) / heads;
    const int64_t b = slot / a.slots, j = slot % a.slots;
    int64_t t0, t1;
    token_range(p.cu, b, p.tokens, &t0, &t1);
    const int64_t ctx = p.ctx[b], start = ctx - (t1 - t0);
    if (t1 == t0 || ctx <= 0) return;
    const int64_t pidx = (start > 0 ? start / page : 0) + j, p_lo = pidx * page;
    if (p_lo >= ctx || pidx >= p.width) return;
    const int64_t id = p.block_table[b * p.width + pidx];
    if (id < 0 || id >= p.c.pages) return;
    const int64_t lo = start > p_lo ? start : p_lo, hi = ctx < p_lo + page ? ctx : p_lo + page;
    const int had = static_cast<int>(lo - p_lo);
    const int units = static_cast<int>(hi - lo) * (dim / 8);

    const Heads &src = kind ? p.v : p.k;
    const int rot = kind ? 0 : static_cast<int>(p.rot);
    const bool inter = p.interleaved != 0;
    const T *rows = static_cast<const T *>(src.p) + (t0 + lo - start) * src.ts + h * src.hs;
    float *scale = (kind ? p.c.v_scale : p.c.k_scale) + id * heads + h;
    uint8_t *codes = static_cast<uint8_t *>(kind ? p.c.v : p.c.k) + (id * heads + h) * page * dim;

    __shared__ unsigned warp_top[kThreads / 32];
    // magnitudes compare as their bits: a NaN is above infinity, which is
    // above every finite value
    unsigned top = 0;
    for (int i = threadIdx.x; i < units; i += kThreads) {
        const int t = i / (dim / 8), u = i % (dim / 8);
        int second;
        const int first = unit_offset(u, rot, inter, &second);
        float v[8];
        load_unit<T, ALIGNED>(rows + t * src.ts, first, second, v);
        rotate_unit(v, p.table, p.rows, rot, inter, lo + t, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x / 32] = top;
    const float old = had > 0 ? fabsf(*scale) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = max(top, warp_top[w]);

    // A page with a value that is not finite gets the scale NaN and codes 0:
    // every read of it shows.
    const bool finite_new = top < 0x7f800000u;
    const float want = __fmul_rn(__uint_as_float(top), KV == OM_I8 ? 1.0f / 127.0f : 1.0f / 448.0f);
    const bool finite = finite_new && __float_as_uint(old) < 0x7f800000u;
    const float grown = finite ? fmaxf(old, want) : __int_as_float(0x7FC00000);
    if (threadIdx.x == 0) *scale = grown;

    if (had > 0 && (grown != old || !finite)) {
        const float ratio = finite ? __fdiv_rn(old, grown) : 0.0f;  // grown > old >= 0
        uint4 *c = reinterpret_cast<uint4 *>(codes);
        for (int i = threadIdx.x; i < had * dim / 16; i += kThreads) {
            uint4 w4 = c[i];
            uint32_t *w = &w4.x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t r = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    r |= encode<KV>(finite ? __fmul_rn(decode<KV>(w[q] >> (8 * e)), ratio) : 0.0f) << (8 * e);
                w[q] = r;
            }
            c[i] = w4;
        }
    }
    for (int i = threadIdx.x; i < units; i += kThreads) {
        const int t = i / (dim / 8), u = i % (dim / 8);
        int second;
        const int first = unit_offset(u, rot, inter, &second);
        float v[8];
        load_unit<T, ALIGNED>(rows + t * src.ts, first, second, v);
        rotate_unit(v, p.table, p.rows, rot, inter, lo + t, u);
        uint32_t w[2] = {0, 0};
        if (finite && grown > 0.0f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e / 4] |= encode<KV>(__fdiv_rn(v[e], grown)) << (8 * (e % 4));
        }
        uint8_t *dst = codes + (had + t) * dim;
        *reinterpret_cast<uint32_t *>(dst + first) = w[0];
        *reinterpret_cast<uint32_t *>(dst + second) = w[1];
    }
}

// One block per token rotates its queries.
template <typename T, bool ALIGNED>
__device__ void rotate_queries(const AppendArgs &a, int64_t t) {
    const KvAppendProblem &p = a.p;
    const int dim = static_cast<int>(p.c.dim), rot = static_cast<int>(p.rot);
    const int64_t b = block_sequence_of(p.cu, p.seqs, t);
    // a token that no sequence owns has no position: its queries become NaN
    const int64_t pos = b < p.seqs && t >= p.cu[b]
                            ? static_cast<int64_t>(p.ctx[b]) - (p.cu[b + 1] < p.tokens ? p.cu[b + 1] : p.tokens) + t
                            : -1;
    const T *src = static_cast<const T *>(p.q.p) + t * p.q.ts;
    T *dst = static_cast<T *>(const_cast<void *>(p.q_out.p)) + t * p.q_out.ts;
    const int units = static_cast<int>(p.q_heads) * (dim / 8);
    for (int i = threadIdx.x; i < units; i += kThreads) {
        const int h = i / (dim / 8), u = i % (dim / 8);
        int second;
        const int first = unit_offset(u, rot, p.interleaved != 0, &second);
        float v[8];
        load_unit<T, ALIGNED>(src + h * p.q.hs, first, second, v);
        rotate_unit(v, p.table, p.rows, rot, p.interleaved != 0, pos, u);
        store4<T, ALIGNED>(dst + h * p.q_out.hs + first, v);
        store4<T, ALIGNED>(dst + h * p.q_out.hs + second, v + 4);
    }
}

template <typename T, int KV, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    const int64_t block = blockIdx.x;
    if (block < a.cache_blocks)
        append_page<T, KV, ALIGNED>(a, block);
    else
        rotate_queries<T, ALIGNED>(a, block - a.cache_blocks);
}

// One block per token: 16 codes of one head's keys or values per thread.
template <typename T, int KV>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ KvReadProblem p) {
    const int64_t t = blockIdx.x;
    const int64_t b = block_sequence_of(p.cu, p.seqs, t);
    const int64_t heads = p.c.heads, page = p.c.page;
    const int dim = static_cast<int>(p.c.dim);
    int64_t id = -1, pos = -1;
    if (b < p.seqs && t >= p.cu[b]) {
        pos = static_cast<int64_t>(p.start[b]) + t - p.cu[b];
        if (pos >= 0 && pos / page < p.width) id = p.block_table[b * p.width + pos / page];
        if (id >= p.c.pages) id = -1;
    }
    const int per_head = dim / 16, units = static_cast<int>(heads) * per_head;
    for (int i = threadIdx.x; i < 2 * units; i += kThreads) {
        const int kind = i >= units, r = kind ? i - units : i;
        const int64_t h = r / per_head;
        const int d = r % per_head * 16;
        T *out = static_cast<T *>(kind ? p.v_out : p.k_out) + (t * heads + h) * dim + d;
        float scale = __int_as_float(0x7FC00000);  // a position the cache does not hold reads as NaN
        uint4 w4 = make_uint4(0, 0, 0, 0);
        if (id >= 0) {
            scale = (kind ? p.c.v_scale : p.c.k_scale)[id * heads + h];
            w4 = *reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kind ? p.c.v : p.c.k) +
                                                  ((id * heads + h) * page + pos % page) * dim + d);
        }
        const uint32_t *w = &w4.x;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(decode<KV>(w[q] >> (8 * e)), scale);
            store4<T, true>(out + 4 * q, v);
        }
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
    if (aligned)
        kv_append_kernel<T, KV, true><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
    else
        kv_append_kernel<T, KV, false><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t append_codes(const AppendArgs &a, bool aligned, int64_t blocks, cudaStream_t s) {
    return a.p.c.dtype == OM_I8 ? append_typed<T, OM_I8>(a, aligned, blocks, s)
                                : append_typed<T, OM_E4M3>(a, aligned, blocks, s);
}

template <typename T>
cudaError_t read_codes(const KvReadProblem &p, cudaStream_t s) {
    if (p.c.dtype == OM_I8)
        kv_read_kernel<T, OM_I8><<<static_cast<unsigned>(p.tokens), kThreads, 0, s>>>(p);
    else
        kv_read_kernel<T, OM_E4M3><<<static_cast<unsigned>(p.tokens), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

// Groups of four elements start on their own size's boundary in every row.
bool heads_aligned(const Heads &x, int64_t heads, int bytes) {
    return reinterpret_cast<uintptr_t>(x.p) % (4 * bytes) == 0 && x.ts % 4 == 0 && (heads == 1 || x.hs % 4 == 0);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendProblem &p, cudaStream_t s) {
    AppendArgs a{p, 0, 0};
    const int64_t most = p.max_new < p.tokens ? p.max_new : p.tokens;
    a.slots = (most + p.c.page - 2) / p.c.page + 1;
    a.cache_blocks = p.seqs * a.slots * p.c.heads * 2;
    const int64_t blocks = a.cache_blocks + (p.q_heads > 0 ? p.tokens : 0);
    const int bytes = p.dtype == OM_F32 ? 4 : 2;
    const bool aligned = heads_aligned(p.k, p.c.heads, bytes) && heads_aligned(p.v, p.c.heads, bytes) &&
                         (p.q_heads == 0 || (heads_aligned(p.q, p.q_heads, bytes) && heads_aligned(p.q_out, p.q_heads, bytes)));
    if (p.dtype == OM_F32) return append_codes<float>(a, aligned, blocks, s);
    if (p.dtype == OM_F16) return append_codes<__half>(a, aligned, blocks, s);
    return append_codes<__nv_bfloat16>(a, aligned, blocks, s);
}

cudaError_t launch_kv_read(const KvReadProblem &p, cudaStream_t s) {
    if (p.dtype == OM_F32) return read_codes<float>(p, s);
    if (p.dtype == OM_F16) return read_codes<__half>(p, s);
    return read_codes<__nv_bfloat16>(p, s);
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
