// kv_attention.cuh -- attention over the paged 8-bit cache, few query rows at a time; one
// translation unit for each type of activations (kv_attention_*.cu).
//
// Mathematics. With keys k_t = c_t a (codes c_t, a the page's scale) and values
// v_t = e_t s:  out = sum_t 2^(x_t - m) s e_t / sum_t 2^(x_t - m),  x_t = (q . c_t) a scale log2(e),
// one pass over the positions with a running m. Codes are exact in 16-bit floats,
// so both products run on the tensor cores with 32-bit sums; the query row is
// scaled by a power of two to fill the 16-bit range and, for 32-bit queries, held in
// two parts of 11 bits, as are the weights 2^(x - m) (one part, 11 bits, for
// 16-bit queries: their outputs are rounded to at most 11 bits anyway). Value scales go
// into the weights, relative to the largest value scale met so far, so that they
// stay in 16-bit range.
//
// Layout. The products are taken transposed, S^T = C Q^T and O^T = E^T P^T: codes
// are the 16-row operand and the query rows (query tokens times the heads that
// share a key head) the 8-column one, so a block holds 8, 16 or 32 of them and one
// query head wastes no more than 7 columns. Each byte of the cache is
// used by exactly one lane: the sums run over head dimensions (for S) and positions (for O), whose
// order is free, so a lane takes 16 consecutive bytes of a row as four
// k-steps (keys) or eight row pairs (values). A lane's copies therefore go through a ring in
// shared memory that only the lane itself reads, with no barrier and no
// bank conflict; S^T turns into P^T's operand by one 8 x 8 transpose per 8 positions.
#pragma once

#include <cfloat>
#include <type_traits>

#include "decode_device.cuh"
#include "om_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 16;              // positions of a warp's step
constexpr int kUnit = kTile * kWarps;  // positions of a unit of work
constexpr int kMinUnits = 4;           // a block takes at least so many units
constexpr float kLog2e = 1.4426950408889634f;
// Weights carry a factor of 2^6 and may exceed the running maximum's by 2^8 before it is
// raised: below 2^14, inside 16-bit range, with the small ones above its subnormals.
constexpr float kBias = 6.0f, kSlack = 8.0f;

template <int DIM>
struct Shape {
    static constexpr int kKeyChunks = DIM / 64;              // 16-byte pieces of a key row, per lane
    static constexpr int kValueBytes = DIM >= 128 ? 16 : 8;  // of a value row's piece
    static constexpr int kValueChunks = DIM / 8 / kValueBytes;
    static constexpr int kSteps = DIM / 16;                  // k-steps of S, row tiles of O
    static constexpr int kTileBytes = 2 * kTile * DIM;
    static constexpr int kStages = DIM == 64 ? 6 : (DIM == 128 ? 4 : 3);
    static constexpr int kRing = kStages * kTileBytes;       // of one warp
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
__device__ __forceinline__ float2 unpack_half(uint32_t x) {
    __half2 h;
    memcpy(&h, &x, 4);
    return __half22float2(h);
}

// Codes as 16-bit floats. A whole number c becomes 1024 + (c + 128) by placing its byte
// (sign bit flipped) under the exponent byte 0x64, then loses 1152: both steps exact.
template <int KV>
__device__ __forceinline__ uint32_t prepare_codes(uint32_t w) {
    return KV == OM_I8 ? w ^ 0x80808080u : w;
}
template <int KV, int HIGH>
__device__ __forceinline__ uint32_t widen(uint32_t w) {  // bytes 0, 1 (or 2, 3) of w
    if constexpr (KV == OM_I8) {
        const uint32_t u = __byte_perm(w, 0x64646464u, HIGH ? 0x4342 : 0x4140);
        __half2 h, c = __half2half2(__ushort_as_half(0x6480));
        memcpy(&h, &u, 4);
        h = __hsub2(h, c);
        uint32_t r;
        memcpy(&r, &h, 4);
        return r;
    } else {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(HIGH ? w >> 16 : w & 0xffffu), __NV_E4M3);
        return static_cast<uint32_t>(h.x) | static_cast<uint32_t>(h.y) << 16;
    }
}

struct Args {
    KvAttentionProblem p;
    int pairs;  // outputs are aligned for stores of two
};

// What a block does for one sequence.
struct Sequence {
    int64_t b, t0;         // first token of the batch
    int64_t ctx, limit;    // tokens, and positions the table reaches
    int queries;
    int row_blocks;
    int64_t first_unit, units;
};

template <int ROWS>
__device__ __forceinline__ Sequence sequence_of(const KvAttentionProblem &p, int64_t b, int group) {
    Sequence s;
    int64_t t1;
    token_range(p.cu, b, p.tokens, &s.t0, &t1);
    s.b = b;
    s.ctx = p.ctx[b];
    s.queries = static_cast<int>(t1 - s.t0);
    s.row_blocks = static_cast<int>((static_cast<int64_t>(s.queries) * group + ROWS - 1) / ROWS);
    s.limit = p.width * p.c.page;
    const int64_t hi = s.ctx < s.limit ? s.ctx : s.limit;
    int64_t lo = 0;
    if (p.window > 0) lo = s.ctx - s.queries - p.window + 1;
    if (lo < 0) lo = 0;
    s.first_unit = lo / kUnit;
    s.units = (hi + kUnit - 1) / kUnit - s.first_unit;
    if (s.units < 1) s.units = 1;  // rows that see nothing are written too
    return s;
}

// Joins two partial results of the same columns: (m, l, O) with O of 2^(x - m) weights.
template <int N>
__device__ __forceinline__ float weight_of(float m, float top) {
    return m == -INFINITY ? 0.0f : ex2(m - top);
}

template <typename T>
__device__ __forceinline__ void store_pair(T *dst, float a, float b, bool pairs) {
    if (!pairs) {
        dst[0] = from_float<T>(a);
        dst[1] = from_float<T>(b);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(dst) = make_float2(a, b);
    } else {
        T e[2] = {from_float<T>(a), from_float<T>(b)};
        uint32_t w;
        memcpy(&w, e, 4);
        *reinterpret_cast<uint32_t *>(dst) = w;
    }
}

template <typename T, int KV, int DIM, int NT>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const __grid_constant__ Args a) {
    using S = Shape<DIM>;
    constexpr int kRows = 8 * NT;
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    // query fragments stay in registers where they fit beside the sums
    constexpr bool kQShared = NT * kParts * S::kSteps > 16;
    constexpr int kFrag = S::kSteps * NT;  // float4 of O per lane
    const KvAttentionProblem &p = a.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, c = lane % 4;
    const int group = static_cast<int>(p.q_heads / p.c.heads);
    const int page = static_cast<int>(p.c.page), heads = static_cast<int>(p.c.heads);

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float row_factor[kRows];
    __shared__ long long scan[kWarps];
    __shared__ int is_last;
    uint8_t *const ring = smem + warp * S::kRing;
    const uint32_t ring_at = smem_u32(ring);
    uint2 *const q_shared = reinterpret_cast<uint2 *>(smem + kWarps * S::kRing);  // [part][step][nt][lane]

    // ---- this block's share of the units of all items (sequence, key head, row block)
    long long total = 0;
    for (int64_t b = threadIdx.x; b < p.seqs; b += kThreads) {
        const Sequence s = sequence_of<kRows>(p, b, group);
        total += static_cast<long long>(heads) * s.row_blocks * s.units;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += scan[w];
    const bool split = p.workspace != nullptr;
    long long per = (total + gridDim.x - 1) / gridDim.x;
    if (per < kMinUnits) per = kMinUnits;
    const long long u0 = blockIdx.x * per, u1 = u0 + per < total ? u0 + per : total;
    if (u0 >= total) return;

    // the sequence that unit u0 belongs to, and the units before it
    int64_t b = 0;
    long long before = 0;
    for (int64_t base = 0;; base += kThreads) {
        const int64_t mine = base + threadIdx.x;
        long long n = 0;
        if (mine < p.seqs) {
            const Sequence s = sequence_of<kRows>(p, mine, group);
            n = static_cast<long long>(heads) * s.row_blocks * s.units;
        }
        long long up = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += x;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = up;
        __syncthreads();
        long long chunk = 0, lower = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) lower += scan[w];
            chunk += scan[w];
        }
        up += lower;  // units up to and with this thread's sequence, in the chunk
        if (before + chunk > u0) {
            __shared__ long long found[2];
            if (before + up > u0 && before + up - n <= u0) {
                found[0] = mine;
                found[1] = before + up - n;
            }
            __syncthreads();
            b = found[0];
            before = found[1];
            break;
        }
        before += chunk;
    }

    Sequence seq = sequence_of<kRows>(p, b, group);
    long long u = u0;
    while (u < u1) {
        while (u >= before + static_cast<long long>(heads) * seq.row_blocks * seq.units) {
            before += static_cast<long long>(heads) * seq.row_blocks * seq.units;
            seq = sequence_of<kRows>(p, ++b, group);
        }
        const long long item = (u - before) / seq.units;
        const long long item_start = before + item * seq.units, item_end = item_start + seq.units;
        const int h = static_cast<int>(item / seq.row_blocks), rb = static_cast<int>(item % seq.row_blocks);
        long long stop = item_end < u1 ? item_end : u1;
        if (!split) {  // whole items, by the block that has their first unit
            if (u > item_start) {
                u = stop;
                continue;
            }
            stop = item_end;
        }
        const int64_t pos0 = (seq.first_unit + (u - item_start)) * kUnit;
        const int n_tiles = static_cast<int>(stop - u);  // of each warp

        // ---- rows of this block: their positions and what they see
        const int row0 = rb * kRows;
        const int rows = min(kRows, seq.queries * group - row0);
        const int64_t start = seq.ctx - seq.queries;  // position of the first query
        const int64_t p_first = start + row0 / group, p_last = start + (row0 + rows - 1) / group;
        const int64_t hi = p_last + 1 < seq.limit ? p_last + 1 : seq.limit;
        const int64_t lo = p.window > 0 && p_first - p.window + 1 > 0 ? p_first - p.window + 1 : 0;
        const int64_t lo_last = p.window > 0 && p_last - p.window + 1 > 0 ? p_last - p.window + 1 : 0;
        int64_t w0 = pos0 + static_cast<int64_t>(warp) * n_tiles * kTile;
        int64_t w1 = w0 + static_cast<int64_t>(n_tiles) * kTile;
        if (w0 < lo) w0 = lo / kTile * kTile;
        if (w1 > hi) w1 = hi;
        const int tiles = w1 > w0 ? static_cast<int>((w1 - w0 + kTile - 1) / kTile) : 0;

        // ---- pages: lane i holds page pb + i (cur) and pb + 32 + i (next), with their scales
        const int32_t *const row_table = p.block_table + seq.b * p.width;
        int64_t pb = w0 / page;
        auto load_id = [&](int64_t j) -> int {
            int id = -1;
            if (j < p.width && j * page < hi) id = row_table[j];
            return id < p.c.pages && id >= 0 ? id : -1;
        };
        int id0 = -1, id1 = -1;
        float ka0 = 0.0f, va0 = 0.0f, ka1 = 0.0f, va1 = 0.0f;
        if (tiles > 0) {
            id0 = load_id(pb + lane);
            id1 = load_id(pb + 32 + lane);
        }
        const int first_row = static_cast<int>(w0 % page);  // of the first tile, in its page
        const int64_t head_bytes = static_cast<int64_t>(page) * DIM;
        auto fetch = [&](int tile) {
            if (tile < tiles) {
                const int row = first_row + tile * kTile, off = row / page - static_cast<int>(pb - w0 / page);
                const int id = __shfl_sync(0xffffffffu, off < 32 ? id0 : id1, off & 31);
                const int64_t at = (static_cast<int64_t>(id < 0 ? 0 : id) * heads + h) * head_bytes + (id < 0 ? 0 : row % page) * DIM;
                const uint8_t *ks = static_cast<const uint8_t *>(p.c.k) + at + g * DIM + c * 16;
                const uint8_t *vs = static_cast<const uint8_t *>(p.c.v) + at + 2 * c * DIM + g * S::kValueBytes;
                const uint32_t dst = ring_at + tile % S::kStages * S::kTileBytes;
                const int key_bytes = id < 0 ? 0 : 16;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < S::kKeyChunks; ++i)
                        cp16(dst + (r * S::kKeyChunks + i) * 512 + lane * 16, ks + r * 8 * DIM + i * 64, key_bytes);
                // values behind the last visible position are taken as zero: a weight of
                // zero would not hide a NaN among them
                const int left = id < 0 ? 0 : static_cast<int>(min(hi - w0 - static_cast<int64_t>(tile) * kTile, static_cast<int64_t>(kTile)));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = 2 * c + (r & 1) + (r & 2) * 4;
#pragma unroll
                    for (int i = 0; i < S::kValueChunks; ++i) {
                        const uint32_t d = dst + kTile * DIM + (r * S::kValueChunks + i) * 32 * S::kValueBytes + lane * S::kValueBytes;
                        const uint8_t *s = vs + ((r & 1) + (r & 2) * 4) * DIM + i * 128;
                        if constexpr (S::kValueBytes == 16)
                            cp16(d, s, t < left ? 16 : 0);
                        else
                            cp8(d, s, t < left ? 8 : 0);
                    }
                }
            }
            cp_commit();
        };
        __syncthreads();  // the ring's other uses (the joins) are over
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) fetch(i);
        auto load_scales = [&](int id, float *ka, float *va) {
            *ka = id < 0 ? 0.0f : p.c.k_scale[static_cast<int64_t>(id) * heads + h];
            *va = id < 0 ? 0.0f : p.c.v_scale[static_cast<int64_t>(id) * heads + h];
        };
        load_scales(id0, &ka0, &va0);
        int next_scaled = 0;

        // ---- query fragments: column n = row of the block, k-step s of lane c: elements d .. d+3
        uint32_t qf[kQShared ? 1 : kParts][kQShared ? 1 : S::kSteps][kQShared ? 1 : NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (kQShared && nt % kWarps != warp) continue;
            const int r = row0 + nt * 8 + g;
            const bool live = nt * 8 + g < rows;
            const T *src = static_cast<const T *>(p.q.p) + (live ? (seq.t0 + r / group) * p.q.ts + (static_cast<int64_t>(h) * group + r % group) * p.q.hs : 0);
            unsigned top = 0;
#pragma unroll
            for (int i = 0; i < S::kKeyChunks; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (live) top = max(top, __float_as_uint(to_float(src[i * 64 + c * 16 + e])) & 0x7fffffffu);
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row's largest element to [2^13, 2^14)
            int e = static_cast<int>(top >> 23) - 127;
            e = e < -100 ? -100 : e;
            const float up = __uint_as_float(static_cast<unsigned>(13 - e + 127) << 23);
            const float down = __uint_as_float(static_cast<unsigned>(e - 13 + 127) << 23);
            if (c == 0 && (kQShared || warp == 0)) row_factor[nt * 8 + g] = __fmul_rn(down, __fmul_rn(p.scale, kLog2e));
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = live ? __fmul_rn(to_float(src[s / 4 * 64 + c * 16 + s % 4 * 4 + j]), up) : 0.0f;
                uint32_t w[2] = {pack_half(v[0], v[1]), pack_half(v[2], v[3])};
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    if constexpr (kQShared) {
                        q_shared[((part * S::kSteps + s) * NT + nt) * 32 + lane] = make_uint2(w[0], w[1]);
                    } else {
                        qf[part][s][nt][0] = w[0];
                        qf[part][s][nt][1] = w[1];
                    }
                    const float2 x = unpack_half(w[0]), y = unpack_half(w[1]);
                    w[0] = pack_half(v[0] - x.x, v[1] - x.y);
                    w[1] = pack_half(v[2] - y.x, v[3] - y.y);
                }
            }
        }
        __syncthreads();
        float factor[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) factor[nt][j] = row_factor[nt * 8 + 2 * c + j];

        // ---- one pass over the warp's positions
        float o[S::kSteps][NT][4], m[NT][2], l[NT][2], vmax = FLT_MIN;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[s][nt][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = -INFINITY;
                l[nt][j] = 0.0f;
            }
        }
        for (int tile = 0; tile < tiles; ++tile) {
            fetch(tile + S::kStages - 1);
            cp_wait<S::kStages - 1>();
            const int off = (first_row + tile * kTile) / page - static_cast<int>(pb - w0 / page);
            const int id = __shfl_sync(0xffffffffu, id0, off);
            const float ka = __shfl_sync(0xffffffffu, ka0, off), va = __shfl_sync(0xffffffffu, va0, off);
            if (off >= 16 && !next_scaled) {  // the ids have arrived long ago
                load_scales(id1, &ka1, &va1);
                next_scaled = 1;
            }
            const uint32_t src = ring_at + tile % S::kStages * S::kTileBytes;

            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[nt][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < S::kKeyChunks; ++i) {
                const uint4 ra = lds16(src + i * 512 + lane * 16);
                const uint4 rc = lds16(src + (S::kKeyChunks + i) * 512 + lane * 16);
                const uint32_t x[4] = {ra.x, ra.y, ra.z, ra.w}, y[4] = {rc.x, rc.y, rc.z, rc.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t xa = prepare_codes<KV>(x[w]), ya = prepare_codes<KV>(y[w]);
                    const uint32_t frag[4] = {widen<KV, 0>(xa), widen<KV, 0>(ya), widen<KV, 1>(xa), widen<KV, 1>(ya)};
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (kQShared) {
                                const uint2 q = q_shared[((part * S::kSteps + i * 4 + w) * NT + nt) * 32 + lane];
                                mma(s[nt], frag, q.x, q.y);
                            } else {
                                mma(s[nt], frag, qf[part][i * 4 + w][nt][0], qf[part][i * 4 + w][nt][1]);
                            }
                        }
                }
            }
            // x = (q . c) a scale log2(e); what a row does not see becomes -infinity
            const int64_t t0 = w0 + static_cast<int64_t>(tile) * kTile;
            const bool inside = id >= 0 && t0 >= lo_last && t0 + kTile - 1 <= p_first && t0 + kTile <= hi;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[nt][j] = __fmul_rn(s[nt][j], __fmul_rn(ka, factor[nt][j & 1]));
            if (!inside) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t t = t0 + g + (j & 2) * 4;
                        const int64_t pos = start + (row0 + nt * 8 + 2 * c + (j & 1)) / group;
                        if (id < 0 || t > pos || t >= hi || (p.window > 0 && t <= pos - p.window)) s[nt][j] = -INFINITY;
                    }
            }
            // the maximum is raised only when a weight would pass the slack
            bool high = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) high |= s[nt][j] > m[nt][j & 1] + kSlack;
            const bool scaled = fabsf(va) <= FLT_MAX;  // an infinite scale counts as NaN
            if (__any_sync(0xffffffffu, high) || (scaled && fabsf(va) > vmax)) {
                const float vnew = scaled ? fmaxf(vmax, fabsf(va)) : vmax, vr = __fdividef(vmax, vnew);
                vmax = vnew;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = fmaxf(s[nt][j], s[nt][j + 2]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float top = fmaxf(m[nt][j], x);
                        const float r = m[nt][j] == -INFINITY ? 0.0f : ex2(m[nt][j] - top);
                        m[nt][j] = top;
                        l[nt][j] = __fmul_rn(l[nt][j], r);
                        const float ro = __fmul_rn(r, vr);
#pragma unroll
                        for (int st = 0; st < S::kSteps; ++st) {
                            o[st][nt][j] = __fmul_rn(o[st][nt][j], ro);
                            o[st][nt][j + 2] = __fmul_rn(o[st][nt][j + 2], ro);
                        }
                    }
            }
            const float vr = scaled ? __fdividef(va, vmax) : __int_as_float(0x7FC00000);
            uint32_t pf[kParts][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float ref = m[nt][j & 1] == -INFINITY ? 0.0f : m[nt][j & 1];
                    const float e = ex2(__fadd_rn(__fsub_rn(s[nt][j], ref), kBias));
                    l[nt][j & 1] = __fadd_rn(l[nt][j & 1], e);
                    w[j] = e == 0.0f ? 0.0f : __fmul_rn(e, vr);  // a hidden position, whatever its scale
                }
                uint32_t x[2] = {pack_half(w[0], w[1]), pack_half(w[2], w[3])};
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    pf[part][nt][0] = transpose8(x[0]);
                    pf[part][nt][1] = transpose8(x[1]);
                    const float2 y = unpack_half(x[0]), z = unpack_half(x[1]);
                    x[0] = pack_half(w[0] - y.x, w[1] - y.y);
                    x[1] = pack_half(w[2] - z.x, w[3] - z.y);
                }
            }
            const uint32_t vsrc = src + kTile * DIM;
#pragma unroll
            for (int i = 0; i < S::kValueChunks; ++i) {
                constexpr int kWords = S::kValueBytes / 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t at = vsrc + (r * S::kValueChunks + i) * 32 * S::kValueBytes + lane * S::kValueBytes;
                    if constexpr (kWords == 4) {
                        const uint4 x = lds16(at);
                        v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
                    } else {
                        const uint2 x = lds8(at);
                        v[r][0] = x.x; v[r][1] = x.y;
                    }
                }
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    const uint32_t r0 = prepare_codes<KV>(v[0][w]), r1 = prepare_codes<KV>(v[1][w]);
                    const uint32_t r8 = prepare_codes<KV>(v[2][w]), r9 = prepare_codes<KV>(v[3][w]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {  // bytes 0, 1, then 2, 3: one row tile each
                        const uint32_t x = __byte_perm(r0, r1, half ? 0x7362 : 0x5140);
                        const uint32_t y = __byte_perm(r8, r9, half ? 0x7362 : 0x5140);
                        const uint32_t frag[4] = {widen<KV, 0>(x), widen<KV, 1>(x), widen<KV, 0>(y), widen<KV, 1>(y)};
                        const int st = i * 2 * kWords + 2 * w + half;
#pragma unroll
                        for (int part = 0; part < kParts; ++part)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma(o[st][nt], frag, pf[part][nt][0], pf[part][nt][1]);
                    }
                }
            }
            // the next tile's page may be the first of the next 32
            if ((first_row + (tile + 1) * kTile) / page - static_cast<int>(pb - w0 / page) >= 32) {
                if (!next_scaled) load_scales(id1, &ka1, &va1);
                next_scaled = 0;
                pb += 32;
                id0 = id1;
                ka0 = ka1;
                va0 = va1;
                id1 = load_id(pb + 32 + lane);
            }
        }
        cp_wait<0>();

        // ---- sums over the lanes that share a column; value scales back into the sums
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[nt][j] = __fadd_rn(l[nt][j], __shfl_xor_sync(0xffffffffu, l[nt][j], x));
#pragma unroll
                for (int st = 0; st < S::kSteps; ++st) {
                    o[st][nt][j] = __fmul_rn(o[st][nt][j], vmax);
                    o[st][nt][j + 2] = __fmul_rn(o[st][nt][j + 2], vmax);
                }
            }

        // ---- join the warps: 2, 3 into 0, 1, then 1 into 0, in the fragments' own layout
        float *const join = reinterpret_cast<float *>(smem);
        constexpr int kJoin = kFrag * 128 + 4 * NT * 32;  // floats of one warp's state
        static_assert(2 * kJoin * 4 <= kWarps * S::kRing, "the join fits in the ring");
#pragma unroll
        for (int step = 2; step >= 1; step >>= 1) {
            __syncthreads();
            if (warp >= step && warp < 2 * step) {
                float *dst = join + (warp - step) * kJoin;
#pragma unroll
                for (int st = 0; st < S::kSteps; ++st)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        reinterpret_cast<float4 *>(dst)[(st * NT + nt) * 32 + lane] = make_float4(o[st][nt][0], o[st][nt][1], o[st][nt][2], o[st][nt][3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    reinterpret_cast<float4 *>(dst)[(kFrag + nt) * 32 + lane] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
            }
            __syncthreads();
            if (warp < step) {
                const float4 *from = reinterpret_cast<const float4 *>(join + warp * kJoin);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float4 x = from[(kFrag + nt) * 32 + lane];
                    const float om[2] = {x.x, x.y}, ol[2] = {x.z, x.w};
                    float wa[2], wb[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float top = fmaxf(m[nt][j], om[j]);
                        wa[j] = m[nt][j] == -INFINITY ? 0.0f : ex2(m[nt][j] - top);
                        wb[j] = om[j] == -INFINITY ? 0.0f : ex2(om[j] - top);
                        m[nt][j] = top;
                        l[nt][j] = __fmaf_rn(l[nt][j], wa[j], __fmul_rn(ol[j], wb[j]));
                    }
#pragma unroll
                    for (int st = 0; st < S::kSteps; ++st) {
                        const float4 y = from[(st * NT + nt) * 32 + lane];
                        o[st][nt][0] = __fmaf_rn(o[st][nt][0], wa[0], __fmul_rn(y.x, wb[0]));
                        o[st][nt][1] = __fmaf_rn(o[st][nt][1], wa[1], __fmul_rn(y.y, wb[1]));
                        o[st][nt][2] = __fmaf_rn(o[st][nt][2], wa[0], __fmul_rn(y.z, wb[0]));
                        o[st][nt][3] = __fmaf_rn(o[st][nt][3], wa[1], __fmul_rn(y.w, wb[1]));
                    }
                }
            }
        }

        // d of (step st, lane group g, row 0 or 8 of the tile): consecutive in a lane
        auto dim_of = [&](int st) {
            return DIM >= 128 ? st / 8 * 128 + g * 16 + st % 8 * 2 : g * 8 + st * 2;
        };
        auto write_row = [&](int col, int st, float x, float y) {  // outputs d, d + 1 of a row
            const int r = row0 + col;
            T *dst = static_cast<T *>(const_cast<void *>(p.out.p)) + (seq.t0 + r / group) * p.out.ts +
                     (static_cast<int64_t>(h) * group + r % group) * p.out.hs + dim_of(st);
            store_pair<T>(dst, x, y, a.pairs);
        };
        auto write_lse = [&](int col, float top, float sum) {
            const int r = row0 + col;
            if (p.lse)
                p.lse[(seq.t0 + r / group) * p.q_heads + static_cast<int64_t>(h) * group + r % group] =
                    sum == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(top - kBias, log2f(sum)), 0.6931471805599453f);
        };

        const bool whole = u == item_start && stop == item_end;
        if (whole) {
            if (warp == 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int col = nt * 8 + 2 * c + j;
                        if (col >= rows) continue;
                        const float inv = l[nt][j] == 0.0f ? 0.0f : __fdiv_rn(1.0f, l[nt][j]);
#pragma unroll
                        for (int st = 0; st < S::kSteps; ++st)
                            write_row(col, st, __fmul_rn(o[st][nt][j], inv), __fmul_rn(o[st][nt][j + 2], inv));
                        if (g == 0) write_lse(col, m[nt][j], l[nt][j]);
                    }
            }
        } else {
            // ---- a part of an item: stored; the block that arrives last joins the parts in
            // their order. Part j of blocks first .. last is in slot 2j, or 2j + 1 where the
            // item starts inside block j's share.
            unsigned *const counters = static_cast<unsigned *>(p.workspace);
            float *const slots = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + kKvCounterBytes);
            constexpr int64_t kSlot = static_cast<int64_t>(kRows) * (DIM + 2);
            const int first = static_cast<int>(item_start / per), last = static_cast<int>((item_end - 1) / per);
            if (warp == 0) {
                float *dst = slots + (2 * static_cast<int64_t>(blockIdx.x) + (u > u0)) * kSlot;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int st = 0; st < S::kSteps; ++st)
                        reinterpret_cast<float4 *>(dst)[(st * NT + nt) * 32 + lane] = make_float4(o[st][nt][0], o[st][nt][1], o[st][nt][2], o[st][nt][3]);
                    if (g == 0) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            dst[kRows * DIM + nt * 8 + 2 * c + j] = m[nt][j];
                            dst[kRows * DIM + kRows + nt * 8 + 2 * c + j] = l[nt][j];
                        }
                    }
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const int here = static_cast<int>(atomicAdd(counters + first, 1u)) == last - first;
                    if (here) counters[first] = 0;  // for the next call
                    is_last = here;
                }
            }
            __syncthreads();
            if (is_last) {
                __threadfence();
                auto slot_of = [&](int j) { return slots + (2 * static_cast<int64_t>(j) + (j == first && item_start > j * per)) * kSlot; };
                for (int f = threadIdx.x; f < kFrag * 32; f += kThreads) {  // f % 32 == lane
                    const int st = f / 32 / NT, nt = f / 32 % NT, col = nt * 8 + 2 * c;
                    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
                    for (int j = first; j <= last; ++j) {
                        const float *from = slot_of(j) + kRows * DIM;
                        top[0] = fmaxf(top[0], __ldcg(from + col));
                        top[1] = fmaxf(top[1], __ldcg(from + col + 1));
                    }
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int j = first; j <= last; ++j) {
                        const float *from = slot_of(j);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(from) + f);
                        const float ma = __ldcg(from + kRows * DIM + col), mb = __ldcg(from + kRows * DIM + col + 1);
                        const float la = __ldcg(from + kRows * DIM + kRows + col), lb = __ldcg(from + kRows * DIM + kRows + col + 1);
                        const float wa = ma == -INFINITY ? 0.0f : ex2(ma - top[0]), wb = mb == -INFINITY ? 0.0f : ex2(mb - top[1]);
                        sum[0] = __fmaf_rn(la, wa, sum[0]);
                        sum[1] = __fmaf_rn(lb, wb, sum[1]);
                        acc.x = __fmaf_rn(y.x, wa, acc.x);
                        acc.y = __fmaf_rn(y.y, wb, acc.y);
                        acc.z = __fmaf_rn(y.z, wa, acc.z);
                        acc.w = __fmaf_rn(y.w, wb, acc.w);
                    }
                    const float ia = sum[0] == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum[0]), ib = sum[1] == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum[1]);
                    if (col < rows) {
                        write_row(col, st, __fmul_rn(acc.x, ia), __fmul_rn(acc.z, ia));
                        if (st == 0 && g == 0) write_lse(col, top[0], sum[0]);
                    }
                    if (col + 1 < rows) {
                        write_row(col + 1, st, __fmul_rn(acc.y, ib), __fmul_rn(acc.w, ib));
                        if (st == 0 && g == 0) write_lse(col + 1, top[1], sum[1]);
                    }
                }
            }
        }
        u = stop;
    }
}

template <typename T, int KV, int DIM, int NT>
cudaError_t launch(const Args &a, cudaStream_t s) {
    using S = Shape<DIM>;
    constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    constexpr bool kQShared = NT * kParts * S::kSteps > 16;
    constexpr int kSmem = kWarps * S::kRing + (kQShared ? kParts * S::kSteps * NT * 32 * 8 : 0);
    static int blocks_per_sm = 0;
    if (blocks_per_sm == 0) {
        cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<T, KV, DIM, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv_attention_kernel<T, KV, DIM, NT>, kThreads, kSmem);
        if (e != cudaSuccess) return e;
        blocks_per_sm = n < 1 ? 1 : n;
    }
    const KvAttentionProblem &p = a.p;
    // no more blocks than the table's units could ask for
    const int64_t rows = p.tokens * (p.q_heads / p.c.heads);
    const __int128 units = static_cast<__int128>((p.width * p.c.page + kUnit - 1) / kUnit) * p.c.heads * (rows / (8 * NT) + p.seqs);
    int64_t grid = static_cast<int64_t>(num_sms()) * blocks_per_sm;
    if (grid > kKvMaxBlocks) grid = kKvMaxBlocks;
    if (units < grid * kMinUnits) grid = static_cast<int64_t>((units + kMinUnits - 1) / kMinUnits);
    if (grid < 1) grid = 1;
    kv_attention_kernel<T, KV, DIM, NT><<<static_cast<unsigned>(grid), kThreads, kSmem, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int KV, int DIM>
cudaError_t by_rows(const Args &a, cudaStream_t s) {
    const int64_t rows = kv_block_rows(a.p.q_heads / a.p.c.heads, DIM, a.p.max_new);
    if (rows == 8) return launch<T, KV, DIM, 1>(a, s);
    if constexpr (DIM <= 128) {
        if (rows == 32) return launch<T, KV, DIM, 4>(a, s);
    }
    return launch<T, KV, DIM, 2>(a, s);
}

template <typename T, int KV>
cudaError_t by_dim(const Args &a, cudaStream_t s) {
    if (a.p.c.dim == 64) return by_rows<T, KV, 64>(a, s);
    if (a.p.c.dim == 128) return by_rows<T, KV, 128>(a, s);
    return by_rows<T, KV, 256>(a, s);
}

template <typename T>
cudaError_t by_codes(const Args &a, cudaStream_t s) {
    return a.p.c.dtype == OM_I8 ? by_dim<T, OM_I8>(a, s) : by_dim<T, OM_E4M3>(a, s);
}

template <typename T>
cudaError_t run_kv_attention(const KvAttentionProblem &p, cudaStream_t s) {
    const bool pairs = reinterpret_cast<uintptr_t>(p.out.p) % (2 * sizeof(T)) == 0 && p.out.ts % 2 == 0 && p.out.hs % 2 == 0;
    return by_codes<T>(Args{p, pairs}, s);
}

}  // namespace
}  // namespace om
