// kv_attention.cuh -- attention over the paged 8-bit cache, few query rows at a time; one
// translation unit for each type of activations (kv_attention_*.cu).
//
// Mathematics. With keys k_t = c_t a (codes c_t, a the page's scale) and values
// v_t = e_t s:  out = sum_t 2^(x_t - m) s e_t / sum_t 2^(x_t - m),  x_t = (q . c_t) a scale log2(e),
// one pass over the positions with a running m. Codes are exact in 16-bit floats,
// so both products run on the tensor cores with 32-bit sums; the query row is
// scaled by a power of two to fill the 16-bit range and, for 32-bit queries, held in
// two parts of 11 bits. The weights are two parts of 11 bits too, for every type: with one part, 16-bit outputs
// were off by more than their own rounding.
//
// Range. What goes to the tensor cores for a position is w = 2^(x - m) s / u with a unit u of the row's sums, a power of two
// that is set anew when the largest |w| of a tile (16 positions of a page) leaves [2^-1, 2^15]. So a weight is off by no more than 2^-22 of
// itself or 2^-24 of its tile's largest, however far the tile's scores and scale are from other tiles' (relative to the
// largest scale met, pages with smaller ones lost their bits).
//
// Layout. The products are taken transposed, S^T = C Q^T and O^T = E^T P^T: codes
// are the 16-row operand and the query rows (query tokens times the heads that
// share a key head) the 8-column one, so a block holds 8 or 16 of them and one
// query head wastes no more than 7 columns. The sums run over head dimensions (for S) and positions (for
// O), whose order is free, so a lane takes 16 consecutive bytes of a row as four k-steps (keys) or
// eight row pairs (values): no byte is moved within a register row. A warp copies its own
// 16 positions of a page, keys and values, each as they lie in memory (whole lines: pieces of
// half a line read at three quarters of the rate), into a ring that no other warp reads, rows turned by an
// exclusive-or so that both ways of reading them are free of bank conflicts. S^T turns into P^T's operand by
// one 8 x 8 transpose per 8 positions.
//
// Split. The work of all (sequence, key head, row block) items, in units of 64 positions, is cut into equal
// shares of the blocks that fit at once, found on the device from the lengths; an item that a cut crosses is joined by
// the block that finishes its last part. More and shorter shares (four times as many) ran no faster.
//
// Roundings beside those parts: exponentials and reciprocals are the approximate instructions (2^-22), and 16-bit calls leave
// their sums of values to the tensor cores, which cut them off (2^-23 of the sum, twice a tile). Relative error of 131071 values of one
// sign: 1e-5 split over the GPU, 2e-4 by one block (half a unit of float16: 4.9e-4).
//
// Bound and measured (GB300; 6 790 GB/s is the measured copy bandwidth). HBM, 2 dim bytes a position and key head:
// 64 sequences of up to 16384 tokens, 8 key heads of 128, 8 query heads each, bfloat16, whole numbers: 248 us,
// 6 510 GB/s, 96 %. One sequence of 131071 tokens, float16, 8-bit floats, pages of 16: 60 us, 4 500 GB/s; with two
// blocks an SM about 4 us until the first product, 45 us in the loop, 9 us for the joins. One of 331 tokens: 7.8 us, latency. 25
// rows of 32-bit queries over a window of 4096: 73 us, 31 %: latency, at two warps a scheduler (255 registers), with
// the tensor pipe 34 % and the ALU 34 % busy; rows are in two blocks that each copy and widen the codes.
#pragma once

#include <cfloat>
#include <climits>
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
constexpr int kWholeUnits = 12;        // items of no more units are not split: joining parts takes longer than that many units
constexpr float kLog2e = 1.4426950408889634f;
// A tile's largest weight is 2^8 as its unit is set, and may go to 2^15 and 2^-1 with the same one: inside 16-bit
// range, its second part above the subnormals. The maximum may lag behind while exponentials are below 2^40.
constexpr float kBias = 8.0f, kMost = 32768.0f, kLeast = 0.5f, kMostExp = 1099511627776.0f;
constexpr float kNone = -FLT_MAX;  // the maximum of no scores
// Units from 2^-126 to 2^126, and no smaller than a value scale by 2^100; a smaller one may not raise sums above 2^100.
constexpr float kLeastUnit = FLT_MIN, kLeastOfScale = 7.8886090522101181e-31f;
constexpr unsigned kMostUnit = 253u << 23;
// A value scale in units, finite: a weight of 0 stays 0.
__device__ __forceinline__ float in_units(float value, float per_unit) { return fminf(fmaxf(__fmul_rn(value, per_unit), -FLT_MAX), FLT_MAX); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }
__device__ __forceinline__ float reciprocal(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }

template <int DIM>
struct Shape {
    static constexpr int kKeyChunks = DIM / 64;              // 16-byte pieces of a key row, per lane
    static constexpr int kValueBytes = DIM >= 128 ? 16 : 8;  // of a value row's piece
    static constexpr int kValueChunks = DIM / 8 / kValueBytes;
    static constexpr int kSteps = DIM / 16;                  // k-steps of S, row tiles of O
    static constexpr int kTileBytes = 2 * kTile * DIM;
    static constexpr int kCopies = kTile * DIM / 512;        // 16-byte copies of a lane, for keys and for values
    static constexpr int kCopyRows = 512 / DIM;              // rows that one of them covers for a warp
    // Where piece p (16 bytes) of row r < 8 lies in a tile (rows r + 8: 8 rows further). Rows of 128 bytes and
    // more: pieces by an exclusive-or whose low bit is the row's and whose third bit parts even rows from
    // odd ones; rows of 64 bytes: neighbouring pairs of rows and of pieces change places.
    __device__ static __forceinline__ int place(int r, int p) {
        if constexpr (DIM == 64) return (r ^ ((r >> 1) & 1)) * 64 + (p ^ ((r >> 1) & 2)) * 16;
        return r * DIM + (p ^ (r & 7) ^ ((r & 1) << 2)) * 16;
    }
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x to a unit in the last place, and 0 for a sum of nothing. Sums lie far inside the range. (Three rounded
// divisions in a row took 0.4 us of one short sequence's 6.9 us.)
__device__ __forceinline__ float inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return x == 0.0f ? 0.0f : y;
}

// A part's sum of weights, taken relative to the maximum of all parts. Without a maximum a part saw nothing (its sum is 0) or
// scores that are all NaN (its sum is NaN, and stays).
__device__ __forceinline__ float joined(float sum, float top, float best) { return top == -INFINITY ? sum : __fmul_rn(sum, ex2(top - best)); }

__device__ __forceinline__ void mma(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
        uint32_t r;
        if constexpr (HIGH)
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
        else
            asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
        return r;
    }
}

struct Args {
    KvAttentionProblem p;
    bool out_fours, q_fours;  // outputs and queries are aligned for stores and loads of four
};

// What a block does for one sequence. Units and positions are below 2^31.
struct Sequence {
    int b, t0;  // t0: its first token in the batch
    int queries, row_blocks;
    int first_unit, units;
    int64_t start;  // position of the first query
    int limit;      // positions before it are in the cache
};

template <int ROWS>
__device__ __forceinline__ Sequence sequence_of(const KvAttentionProblem &p, int64_t b, int group) {
    Sequence s;
    int64_t t0, t1;
    token_range(p.cu, b, p.tokens, &t0, &t1);
    const int64_t ctx = p.ctx[b], reach = p.width * p.c.page;
    s.b = static_cast<int>(b);
    s.t0 = static_cast<int>(t0);
    s.queries = static_cast<int>(t1 - t0);
    s.row_blocks = (s.queries * group + ROWS - 1) / ROWS;
    s.start = ctx - s.queries;
    s.limit = static_cast<int>(max(min(ctx, reach), static_cast<int64_t>(0)));
    const int lo = p.window > 0 ? static_cast<int>(max(s.start - p.window + 1, static_cast<int64_t>(0))) : 0;
    s.first_unit = lo / kUnit;
    s.units = max((s.limit + kUnit - 1) / kUnit - s.first_unit, 1);  // rows that see nothing are written too
    return s;
}

// What the output of a finished item needs: its units and its rows.
struct Part {
    int begin, end;
    int t0, h, row0, rows;
};

// Finished rows, [row][DIM + 4] floats in shared memory, to the outputs; every thread of the block.
template <typename T, int DIM>
__device__ __forceinline__ void write_rows(const Args &a, const Part &part, int group, const float *stage) {
    constexpr int kQuads = DIM / 4;
#pragma unroll 1
    for (int i = threadIdx.x; i < part.rows * kQuads; i += kThreads) {
        const int col = i / kQuads, d = i % kQuads * 4, r = part.row0 + col;
        T *dst = static_cast<T *>(const_cast<void *>(a.p.out.p)) + (part.t0 + r / group) * a.p.out.ts +
                 (static_cast<int64_t>(part.h) * group + r % group) * a.p.out.hs + d;
        const float4 f = *reinterpret_cast<const float4 *>(stage + col * (DIM + 4) + d);
        const float v[4] = {f.x, f.y, f.z, f.w};
        if (a.out_fours)
            store4<T, true>(dst, v);
        else
            store4<T, false>(dst, v);
    }
}

__device__ __forceinline__ void write_lse(const KvAttentionProblem &p, const Part &part, int group, int col, float top, float sum) {
    const int r = part.row0 + col;
    if (p.lse && col < part.rows)
        p.lse[(part.t0 + r / group) * p.q_heads + static_cast<int64_t>(part.h) * group + r % group] =
            sum == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(top - kBias, log2f(sum)), 0.6931471805599453f);
}

template <typename T, int DIM, int NT>
struct Config {
    using S = Shape<DIM>;
    // 11-bit parts of queries: a 16-bit query is one part as it is
    static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
    // query fragments stay in registers where they fit beside the sums
    static constexpr bool kQShared = NT * kParts * S::kSteps > 16;
    static constexpr int kQBytes = kParts * S::kSteps * NT * 256;
    static constexpr int kStages = DIM == 64 ? 6 : (DIM == 256 ? 2 : 3);
    static constexpr int kJoin = S::kSteps * NT * 128 + NT * 128;  // floats of one warp's state
    // the next segment's copies start before the join of the warps, which then has memory of its own
    static constexpr bool kEarly = NT * DIM <= 256;
    static constexpr int kRing = kStages * S::kTileBytes;  // of one warp
    static constexpr int kSmem = kWarps * kRing + kQBytes + (kEarly ? 2 * kJoin * 4 : 0);
    static constexpr int64_t kSlot = 8 * NT * (DIM + 2);
    // a weight for each part and row, then the finished rows, fit in the ring
    static constexpr int kMostParts = (kWarps * kRing / 4 - 8 * NT * (DIM + 4) - 4) / (8 * NT);
    static constexpr int kMaxBlocks = kMostParts < kKvMaxBlocks ? kMostParts : kKvMaxBlocks;
    static_assert(8 * NT * (DIM + 4) <= 2 * kJoin, "finished rows fit where the warps are joined");
    static_assert(kEarly || 2 * kJoin * 4 <= kWarps * kRing, "the join fits in the ring");
    static_assert(2 * kThreads * 4 <= kQBytes, "the sums of the parts' join fit where the queries were");
};

// BLOCKS: of an SM, at least. Three where the registers allow it (heads of up to 128, 8 rows of 16 bits), two elsewhere. With two, 256
// sequences of 500 tokens, 8 key heads, take 66 us instead of 57, 64 of up to 8000 tokens with heads of 64 101 instead of 89; one of
// 131071 tokens, whose parts are more with three, the same (float16 59.5 and 59.9 us, bfloat16 59.4 and 57.9).
template <typename T, int KV, int DIM, int NT, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) kv_attention_kernel(const __grid_constant__ Args a) {
    using S = Shape<DIM>;
    using C = Config<T, DIM, NT>;
    constexpr int kRows = 8 * NT;
    constexpr int kParts = C::kParts;
    constexpr bool kQShared = C::kQShared;
    constexpr int kFrag = S::kSteps * NT;  // float4 of O per lane
    const KvAttentionProblem &p = a.p;
    unsigned *const counters = static_cast<unsigned *>(p.workspace);
    float *const slots = reinterpret_cast<float *>(static_cast<uint8_t *>(p.workspace) + kKvCounterBytes);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, c = lane % 4;
    const int group = static_cast<int>(p.q_heads / p.c.heads);
    const int page = static_cast<int>(p.c.page), page_log = 31 - __clz(page), heads = static_cast<int>(p.c.heads);

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float row_factor[kRows];
    __shared__ int2 row_seen[kRows];  // a row sees the positions in (x, y]
    __shared__ int scan[kWarps], scan_longest[kWarps], found_before;
    __shared__ unsigned scan_doubt[kWarps];
    __shared__ Sequence found;
    __shared__ Part pending[2];  // parts of items of this block: its first and its last segment's
    __shared__ int arrived_last[2];
    const uint32_t ring_at = smem_u32(smem + warp * C::kRing);
    uint2 *const q_shared = reinterpret_cast<uint2 *>(smem + kWarps * C::kRing);  // [part][step][nt][lane]
    float *const join = reinterpret_cast<float *>(C::kEarly ? smem + kWarps * C::kRing + C::kQBytes : smem);

    wait_for_earlier();
    // ---- this block's share of the units of all items (sequence, key head, row block)
    const int seqs = static_cast<int>(p.seqs);
    int64_t mine = 0;
    int longest = 0;
    bool falls = false;
#pragma unroll 1
    for (int i = threadIdx.x; i < seqs; i += kThreads) {
        const Sequence s = sequence_of<kRows>(p, i, group);
        mine += heads * s.row_blocks * s.units;
        longest = max(longest, s.units);
        falls |= p.cu[i] > p.cu[i + 1];
    }
    int total = __reduce_add_sync(0xffffffffu, static_cast<int>(mine));
    longest = __reduce_max_sync(0xffffffffu, longest);
    // Offsets that never decrease share the tokens out, and the host has bounded their units. Others can count a
    // token for many sequences: nothing is done where their units might pass 32 bits.
    const unsigned doubt = __reduce_or_sync(0xffffffffu, (falls ? 1u : 0u) | (mine > (INT_MAX - kKvMaxBlocks) / kThreads ? 2u : 0u));
    if (lane == 0) {
        scan_doubt[warp] = doubt;
        scan[warp] = total;
        scan_longest[warp] = longest;
    }
    __syncthreads();
    total = longest = 0;
    unsigned doubts = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        total += scan[w];
        longest = max(longest, scan_longest[w]);
        doubts |= scan_doubt[w];
    }
    if (doubts == 3) return;
    const bool split = p.workspace != nullptr && longest > kWholeUnits;
    const int per = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kMinUnits);
    if (static_cast<int64_t>(blockIdx.x) * per >= total) return;
    const int u0 = blockIdx.x * per, u1 = min(u0 + per, total);

    // the sequence that unit u0 belongs to, and the units before it
    int before = 0;
#pragma unroll 1
    for (int base = 0;; base += kThreads) {
        Sequence s;
        int n = 0;
        if (base + static_cast<int>(threadIdx.x) < seqs) {
            s = sequence_of<kRows>(p, base + threadIdx.x, group);
            n = heads * s.row_blocks * s.units;
        }
        int up = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += x;
        }
        __syncthreads();
        if (lane == 31) scan[warp] = up;
        __syncthreads();
        int chunk = 0, lower = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) lower += scan[w];
            chunk += scan[w];
        }
        up += before + lower;  // units up to and with this thread's sequence
        if (up > u0 && up - n <= u0) {
            found = s;
            found_before = up - n;
        }
        before += chunk;
        if (before > u0) break;
    }
    __syncthreads();
    Sequence seq = found;
    before = found_before;

    // ---- the segment at hand: a range of one item's units
    Part part{};
    int u = u0, stop = u0;
    int hi = 0, lo_last = 0, all_see = 0, w0 = 0, w1 = 0, n_parts = 0;
    bool whole = false, at_start = false;
    // pages: lane i holds page pb + i (0) and pb + 32 + i (1), with their scales
    int pb = 0, pages_end = 0, id0 = -1, id1 = -1;
    float ka0 = 0.0f, va0 = 0.0f, ka1 = 0.0f, va1 = 0.0f;
    // the next tile to copy
    int f_pos = 0, f_id = -1;
    uint32_t f_dst = 0;
    const int64_t page_bytes = static_cast<int64_t>(heads) * page * DIM;
    const uint8_t *k_lane = nullptr, *f_k = nullptr;
    const int64_t to_values = static_cast<const uint8_t *>(p.c.v) - static_cast<const uint8_t *>(p.c.k);
    const int copy_row = lane * 16 / DIM;
    const uint32_t copy_to = S::place(copy_row, lane % (DIM / 16));
    bool f_new = true;
    auto load_id = [&](int j) -> int {
        const int id = j < pages_end ? p.block_table[seq.b * p.width + j] : -1;
        return id < p.c.pages ? id : -1;
    };
    auto load_scales = [&](int id, float *ka, float *va) {
        const int64_t at = static_cast<int64_t>(id) * heads + part.h;
        *ka = id < 0 ? 0.0f : p.c.k_scale[at];
        *va = id < 0 ? 0.0f : p.c.v_scale[at];
    };
    auto fetch = [&]() {
        if (f_pos < w1) {
            if (f_new || (f_pos & (page - 1)) == 0) {
                const int off = (f_pos >> page_log) - pb;
                f_id = __shfl_sync(0xffffffffu, off < 32 ? id0 : id1, off & 31);
                f_k = k_lane + (f_id < 0 ? 0 : f_id * page_bytes + (f_pos & (page - 1)) * DIM);
                f_new = false;
            }
            // values behind the last visible position are taken as zero: a weight of zero would
            // not hide a NaN among them
            const int left = f_id < 0 ? 0 : hi - f_pos;
#pragma unroll
            for (int j = 0; j < S::kCopies; ++j) {
                // row j kCopyRows + copy_row: its place differs by constants
                const uint32_t to = f_dst + j * 512 + (copy_to ^ (DIM == 64 ? 0 : (j * S::kCopyRows & 7) * 16));
                const int bytes = copy_row + j * S::kCopyRows < left ? 16 : 0;
                cp16(to, f_k + j * 512, bytes);
                cp16(to + kTile * DIM, f_k + to_values + j * 512, bytes);
            }
            f_k += kTile * DIM;
            f_pos += kTile;
            f_dst = f_dst == ring_at + (C::kStages - 1) * S::kTileBytes ? ring_at : f_dst + S::kTileBytes;
        }
        cp_commit();
    };

    // the next segment's queries: 16 threads a row
    constexpr int kEach = DIM / 16;
    const int q_row = threadIdx.x / 16, q_d = threadIdx.x % 16 * kEach;
    float qv[C::kEarly ? NT : 1][kEach];
    auto load_queries = [&](int nt, float *v) {
        const int r = part.row0 + nt * 8 + q_row;
        if (nt * 8 + q_row < part.rows) {
            const T *src = static_cast<const T *>(p.q.p) + (part.t0 + r / group) * p.q.ts +
                           (static_cast<int64_t>(part.h) * group + r % group) * p.q.hs + q_d;
            if (a.q_fours) {
#pragma unroll
                for (int e = 0; e < kEach; e += 4) load4<T, true>(src + e, v + e);
            } else {
#pragma unroll
                for (int e = 0; e < kEach; e += 4) load4<T, false>(src + e, v + e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kEach; ++e) v[e] = 0.0f;
        }
    };

    // a lane's places in a tile: keys by (row g, pieces c, c + 4, ...), values by (rows 2 c and 2 c + 1,
    // piece g, or half a piece)
    const int key_at = S::place(g, c);
    const unsigned column_bit = 1u << (2 * c);
    const int value_at[2] = {S::place(2 * c, DIM == 64 ? g / 2 : g) + (DIM == 64 ? g % 2 * 8 : 0),
                             S::place(2 * c + 1, DIM == 64 ? g / 2 : g) + (DIM == 64 ? g % 2 * 8 : 0)};

    // Value codes that are NaN, in a tile that not every row sees as a whole: a weight of 0 would not hide them. Rows that see one
    // become NaN in its dimension, and the code becomes 0. o, and the tile's values at vsrc.
    auto hide_nan_codes = [&](float (&o)[S::kSteps][NT][4], uint8_t *vsrc, int pos) {
        auto is_nan = [](uint32_t x) { return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
        uint32_t any = 0;
#pragma unroll
        for (int j = 0; j < S::kCopies; ++j) {
            const uint4 x = *reinterpret_cast<const uint4 *>(vsrc + lane * 16 + j * 512);
            any |= is_nan(x.x) | is_nan(x.y) | is_nan(x.z) | is_nan(x.w);
        }
        if (!__any_sync(0xffffffffu, any != 0)) return;
#pragma unroll 1
        for (int r = 0; r < kTile; ++r) {
            bool sees[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int2 seen = row_seen[nt * 8 + 2 * c + j];
                    sees[nt][j] = pos + r > seen.x && pos + r <= seen.y;
                }
#pragma unroll
            for (int i = 0; i < S::kValueChunks; ++i) {
                // a lane's dimensions: the piece g, or half a piece, as in the product
                constexpr int kWords = S::kValueBytes / 4;
                uint32_t *const at = reinterpret_cast<uint32_t *>(vsrc + S::place(r & 7, DIM == 64 ? g / 2 : g) + (DIM == 64 ? g % 2 * 8 : 0) + r / 8 * 8 * DIM + i * 128);
                uint32_t x[kWords];
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                    x[w] = at[w];
                    const uint32_t bad = is_nan(x[w]);
                    x[w] &= ~((bad >> 7) * 0xffu);
#pragma unroll
                    for (int byte = 0; byte < 4; ++byte)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (sees[nt][j] && (bad >> (8 * byte) & 0x80u)) o[i * 2 * kWords + 2 * w + byte / 2][nt][j + byte % 2 * 2] = __int_as_float(0x7FC00000);
                }
                __syncwarp();  // the four lanes of the piece have read it
                if (c == 0) {
#pragma unroll
                    for (int w = 0; w < kWords; ++w) at[w] = x[w];
                }
            }
        }
        __syncwarp();
    };

    float o[S::kSteps][NT][4], m[NT][2], l[NT][2], per_unit[NT][2];
    bool have = false;
#pragma unroll 1
    for (;;) {
        // ---- the next segment: its rows, its page ids and its first copies, which are on their way
        // during the join and the stores of the last one
        const Part last = part;
        const bool last_whole = whole, last_at_start = at_start;
        bool more = false;
        for (u = stop; u < u1; u = stop) {
            int n;
            while (u >= before + (n = heads * seq.row_blocks * seq.units)) {
                before += n;
                seq = sequence_of<kRows>(p, seq.b + 1, group);
            }
            const int item = (u - before) / seq.units;
            part.begin = before + item * seq.units;
            part.end = part.begin + seq.units;
            stop = min(part.end, u1);
            if (!split) {  // whole items, by the block that has their first unit
                if (u > part.begin) continue;
                stop = part.end;
            }
            part.h = item / seq.row_blocks;
            part.row0 = (item - part.h * seq.row_blocks) * kRows;
            more = true;
            break;
        }
        auto begin_segment = [&]() {
            part.t0 = seq.t0;
            part.rows = min(kRows, seq.queries * group - part.row0);
            whole = u == part.begin && stop == part.end;
            at_start = u == u0;
            const int64_t p_first = seq.start + part.row0 / group, p_last = seq.start + (part.row0 + part.rows - 1) / group;
            hi = static_cast<int>(max(min(p_last + 1, static_cast<int64_t>(seq.limit)), static_cast<int64_t>(0)));
            const int lo = p.window > 0 ? static_cast<int>(max(p_first - p.window + 1, static_cast<int64_t>(0))) : 0;
            lo_last = p.window > 0 ? static_cast<int>(max(p_last - p.window + 1, static_cast<int64_t>(0))) : 0;
            // a tile that starts in [lo_last, all_see] is seen by every row as a whole
            all_see = static_cast<int>(min(p_first, static_cast<int64_t>(hi) - 1)) - (kTile - 1);
            const int pos0 = (seq.first_unit + (u - part.begin)) * kUnit, each = (stop - u) * kTile;
            w0 = pos0 + warp * each;
            w1 = min(w0 + each, hi);
            if (w0 < lo) w0 = lo / kTile * kTile;
            pb = w0 >> page_log;
            pages_end = w0 < w1 ? (hi + page - 1) >> page_log : 0;  // inside the table: hi is
            id0 = load_id(pb + lane);
            id1 = load_id(pb + 32 + lane);
            if constexpr (C::kEarly) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) load_queries(nt, qv[nt]);
            }
            k_lane = static_cast<const uint8_t *>(p.c.k) + static_cast<int64_t>(part.h) * page * DIM + lane * 16;
            f_pos = w0;
            f_new = true;
            f_dst = ring_at;
#pragma unroll 1
            for (int i = 0; i < C::kStages - 1; ++i) fetch();
            load_scales(id0, &ka0, &va0);
        };
        if (C::kEarly && more) begin_segment();

        if (have) {
            // ---- sums over the lanes that share a column. States are joined as weighted means: a mean is no larger than the
            // values, where a sum with its unit could pass the range.
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) l[nt][j] = __fadd_rn(l[nt][j], __shfl_xor_sync(0xffffffffu, l[nt][j], x));
                    const float inv = inverse(l[nt][j]), back = reciprocal(per_unit[nt][j]);
                    if (m[nt][j] == kNone) m[nt][j] = -INFINITY;
#pragma unroll
                    for (int st = 0; st < S::kSteps; ++st) {
                        o[st][nt][j] = __fmul_rn(__fmul_rn(o[st][nt][j], inv), back);
                        o[st][nt][j + 2] = __fmul_rn(__fmul_rn(o[st][nt][j + 2], inv), back);
                    }
                }
            // ---- join the warps: 2, 3 into 0, 1, then 1 into 0, in the fragments' own layout
#pragma unroll 1
            for (int step = 2; step >= 1; step >>= 1) {
                __syncthreads();
                if (warp >= step && warp < 2 * step) {
                    float4 *dst = reinterpret_cast<float4 *>(join + (warp - step) * C::kJoin) + lane;
#pragma unroll
                    for (int st = 0; st < S::kSteps; ++st)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            dst[(st * NT + nt) * 32] = make_float4(o[st][nt][0], o[st][nt][1], o[st][nt][2], o[st][nt][3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) dst[(kFrag + nt) * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
                }
                __syncthreads();
                if (warp < step) {
                    const float4 *from = reinterpret_cast<const float4 *>(join + warp * C::kJoin) + lane;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float4 x = from[(kFrag + nt) * 32];
                        const float om[2] = {x.x, x.y}, ol[2] = {x.z, x.w};
                        float wa[2], wb[2];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float top = fmaxf(m[nt][j], om[j]);
                            wa[j] = joined(l[nt][j], m[nt][j], top);
                            wb[j] = joined(ol[j], om[j], top);
                            m[nt][j] = top;
                            l[nt][j] = __fadd_rn(wa[j], wb[j]);
                            const float inv = inverse(l[nt][j]);
                            wa[j] = __fmul_rn(wa[j], inv);
                            wb[j] = __fmul_rn(wb[j], inv);
                        }
#pragma unroll
                        for (int st = 0; st < S::kSteps; ++st) {
                            const float4 y = from[(st * NT + nt) * 32];
                            o[st][nt][0] = __fmaf_rn(o[st][nt][0], wa[0], __fmul_rn(y.x, wb[0]));
                            o[st][nt][1] = __fmaf_rn(o[st][nt][1], wa[1], __fmul_rn(y.y, wb[1]));
                            o[st][nt][2] = __fmaf_rn(o[st][nt][2], wa[0], __fmul_rn(y.z, wb[0]));
                            o[st][nt][3] = __fmaf_rn(o[st][nt][3], wa[1], __fmul_rn(y.w, wb[1]));
                        }
                    }
                }
            }
            if (last_whole) {
                __syncthreads();
                if (warp == 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int col = nt * 8 + 2 * c + j;
                            // d of (step st, lane group g): consecutive in a lane
                            float *dst = join + col * (DIM + 4) + g * (DIM >= 128 ? 16 : 8);
#pragma unroll
                            for (int st = 0; st < S::kSteps; ++st)
                                *reinterpret_cast<float2 *>(dst + (DIM >= 128 ? st / 8 * 128 + st % 8 * 2 : st * 2)) =
                                    make_float2(o[st][nt][j], o[st][nt][j + 2]);
                            if (g == 0) write_lse(p, last, group, col, m[nt][j], l[nt][j]);
                        }
                }
                __syncthreads();
                write_rows<T, DIM>(a, last, group, join);
            } else if (warp == 0) {
                // a part of an item: kept for the block that joins them. A block has at most
                // two, one that starts with its share (slot 2j) and one that ends with it (2j + 1).
                float *const dst = slots + (2 * static_cast<int64_t>(blockIdx.x) + !last_at_start) * C::kSlot;
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
                if (lane == 0) pending[n_parts] = last;
            }
            n_parts += !last_whole;
        }
        if (!more) break;
        have = true;
        if constexpr (!C::kEarly) {
            __syncthreads();  // the ring is the copies' again
            begin_segment();
        }

        // ---- queries: 16 threads a row scale it by a power of two and lay its parts out as fragments:
        // column n = row of the block, step s of lane c: four elements from 64 (s / 4) + 16 c + 4 (s % 4)
        {
            const int row = q_row;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int r = part.row0 + nt * 8 + row;
                const bool live = nt * 8 + row < part.rows;
                float *const v = qv[C::kEarly ? nt : 0];
                if constexpr (!C::kEarly) load_queries(nt, v);
                unsigned top = 0;
#pragma unroll
                for (int e = 0; e < kEach; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
                // the row's largest element to [2^13, 2^14)
                int e2 = static_cast<int>(top >> 23) - 127;
                e2 = e2 < -100 ? -100 : e2;
                const float up = __uint_as_float(static_cast<unsigned>(13 - e2 + 127) << 23);
                if (threadIdx.x % 16 == 0) {
                    const float down = __uint_as_float(static_cast<unsigned>(e2 - 13 + 127) << 23);
                    row_factor[nt * 8 + row] = __fmul_rn(down, __fmul_rn(p.scale, kLog2e));
                    const int64_t at = seq.start + (live ? r : part.row0) / group;
                    row_seen[nt * 8 + row] = make_int2(p.window > 0 ? static_cast<int>(max(at - p.window, static_cast<int64_t>(-1))) : -1,
                                                       static_cast<int>(max(min(at, static_cast<int64_t>(hi) - 1), static_cast<int64_t>(-1))));
                }
#pragma unroll
                for (int e = 0; e < kEach; e += 4) {
                    const int d = q_d + e, step = d / 64 * 4 + d % 16 / 4, to = row * 4 + d % 64 / 16;
                    float x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = __fmul_rn(v[e + i], up);
#pragma unroll
                    for (int part_i = 0; part_i < kParts; ++part_i) {
                        const uint2 w = make_uint2(pack_half(x[0], x[1]), pack_half(x[2], x[3]));
                        q_shared[((part_i * S::kSteps + step) * NT + nt) * 32 + to] = w;
                        if (part_i + 1 < kParts) {
                            const float2 y = unpack_half(w.x), z = unpack_half(w.y);
                            x[0] -= y.x;
                            x[1] -= y.y;
                            x[2] -= z.x;
                            x[3] -= z.y;
                        }
                    }
                }
            }
        }
        __syncthreads();
        float factor[NT][2];
        uint2 qf[kQShared ? 1 : kParts][kQShared ? 1 : S::kSteps][kQShared ? 1 : NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 f = *reinterpret_cast<const float2 *>(row_factor + nt * 8 + 2 * c);
            factor[nt][0] = f.x;
            factor[nt][1] = f.y;
            if constexpr (!kQShared) {
#pragma unroll
                for (int i = 0; i < kParts; ++i)
#pragma unroll
                    for (int s = 0; s < S::kSteps; ++s) qf[i][s][nt] = q_shared[((i * S::kSteps + s) * NT + nt) * 32 + lane];
            }
        }

        // ---- one pass over the warp's positions
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[s][nt][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nt][j] = kNone;
                l[nt][j] = 0.0f;
                per_unit[nt][j] = 1.0f;
            }
        }
        float kf[NT][2], vf[NT][2], value = 0.0f;  // vf: the page's value scale by the columns' units
        bool next_scaled = false;
        bool page_ok = false, odd_scale = false;
        const uint8_t *const my_ring = smem + warp * C::kRing;
        int src_at = 0;
        bool c_new = true, empty = true;  // empty: no sums yet
#pragma unroll 1
        for (int pos = w0; pos < w1; pos += kTile) {
            cp_wait<C::kStages - 2>();
            __syncwarp();  // the tile is here for every lane, and every lane is done with the last one
            fetch();
            if (c_new || (pos & (page - 1)) == 0) {  // a page's first tile
                c_new = false;
                int off = (pos >> page_log) - pb;
                if (off == 32) {
                    if (!next_scaled) load_scales(id1, &ka1, &va1);
                    next_scaled = false;
                    pb += 32;
                    off = 0;
                    id0 = id1;
                    ka0 = ka1;
                    va0 = va1;
                    id1 = load_id(pb + 32 + lane);
                } else if (off >= 16 && !next_scaled) {  // the ids have arrived long ago
                    load_scales(id1, &ka1, &va1);
                    next_scaled = true;
                }
                page_ok = __shfl_sync(0xffffffffu, id0, off) >= 0;
                const float ka = __shfl_sync(0xffffffffu, ka0, off), va = __shfl_sync(0xffffffffu, va0, off);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) kf[nt][j] = __fmul_rn(ka, factor[nt][j]);
                odd_scale = !(fabsf(va) <= FLT_MAX);  // an infinite scale counts as NaN
                value = va;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) vf[nt][j] = in_units(value, per_unit[nt][j]);
            }

            const uint8_t *const src = my_ring + src_at;
            float s[NT][4], s1[NT][4];  // two chains of products
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[nt][j] = s1[nt][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < S::kKeyChunks; ++i) {
                // piece 4 i + c of rows g and g + 8
                const uint8_t *const at = src + (key_at ^ (i & 1) * 64) + i / 2 * 128;
                const uint4 ra = *reinterpret_cast<const uint4 *>(at);
                const uint4 rc = *reinterpret_cast<const uint4 *>(at + 8 * DIM);
                const uint32_t x[4] = {ra.x, ra.y, ra.z, ra.w}, y[4] = {rc.x, rc.y, rc.z, rc.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t xa = prepare_codes<KV>(x[w]), ya = prepare_codes<KV>(y[w]);
                    const uint32_t frag[4] = {widen<KV, 0>(xa), widen<KV, 0>(ya), widen<KV, 1>(xa), widen<KV, 1>(ya)};
#pragma unroll
                    for (int part_i = 0; part_i < kParts; ++part_i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float *const to = w & 1 ? s1[nt] : s[nt];
                            if constexpr (kQShared) {
                                const uint2 q = q_shared[((part_i * S::kSteps + i * 4 + w) * NT + nt) * 32 + lane];
                                mma(to, frag, q.x, q.y);
                            } else {
                                mma(to, frag, qf[part_i][i * 4 + w][nt].x, qf[part_i][i * 4 + w][nt].y);
                            }
                        }
                }
            }
            // x = (q . c) a scale log2(e); what a row does not see becomes -infinity
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[nt][j] = __fmul_rn(__fadd_rn(s[nt][j], s1[nt][j]), kf[nt][j & 1]);
            unsigned sees_none = 0;  // columns
            if (!(page_ok && pos >= lo_last && pos <= all_see)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int2 seen[2] = {row_seen[nt * 8 + 2 * c], row_seen[nt * 8 + 2 * c + 1]};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = pos + g + (j & 2) * 4;
                        if (!page_ok || t <= seen[j & 1].x || t > seen[j & 1].y) s[nt][j] = -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (!page_ok || pos + kTile - 1 <= seen[j].x || pos > seen[j].y) sees_none |= column_bit << (8 * nt + j);
                }
                if constexpr (KV == OM_E4M3) hide_nan_codes(o, smem + warp * C::kRing + src_at + kTile * DIM, pos);
            }
            float e[NT][4];
            for (bool again = false;; again = true) {
                // a bit for each column whose largest weight is above the low end, and one for what is above the top
                unsigned fit = value == 0.0f || odd_scale ? (1u << kRows) - 1 : sees_none;
                bool high = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float less = m[nt][j] - kBias;
                        e[nt][j] = ex2(__fsub_rn(s[nt][j], less));
                        e[nt][j + 2] = ex2(__fsub_rn(s[nt][j + 2], less));
                        const float top = fmaxf(e[nt][j], e[nt][j + 2]), w = fabsf(__fmul_rn(top, vf[nt][j]));
                        if (w >= kLeast) fit |= column_bit << (8 * nt + j);
                        high |= w > kMost || top > kMostExp;
                    }
                if (high) fit |= 1u << 31;
                if (again || __reduce_or_sync(0xffffffffu, fit) == (1u << kRows) - 1) break;
                // the columns whose largest weight is outside: a new maximum if it is above the old one, and a new unit
                float by[NT][2];  // what the sums are multiplied by
                int up[NT][2];    // the unit goes down by so many powers of two
                bool changed = false, smaller = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float x = fmaxf(s[nt][j], s[nt][j + 2]);
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        const float top = ex2(x - (m[nt][j] - kBias)), w = fabsf(__fmul_rn(top, vf[nt][j]));
                        by[nt][j] = 1.0f;
                        up[nt][j] = 0;
                        if (x > kNone && !(w >= kLeast && w <= kMost && top <= kMostExp)) {
                            if (x > m[nt][j]) {
                                by[nt][j] = ex2(m[nt][j] - x);
                                m[nt][j] = x;
                                l[nt][j] = __fmul_rn(l[nt][j], by[nt][j]);
                            }
                            if (value != 0.0f && !odd_scale) {
                                const float to = fmaxf(__fmul_rn(fmaxf(ex2(x - m[nt][j]), kLeastOfScale), fabsf(value)), kLeastUnit);
                                const unsigned unit = min(__float_as_uint(to) & 0x7f800000u, kMostUnit);
                                up[nt][j] = (static_cast<int>((254u << 23) - unit) - static_cast<int>(__float_as_uint(per_unit[nt][j]))) >> 23;
                                smaller |= up[nt][j] > 0;
                            }
                            changed = true;
                        }
                    }
                const bool sums = !empty && __any_sync(0xffffffffu, changed);
                if (sums && __any_sync(0xffffffffu, smaller)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            unsigned most = 0;  // magnitudes compare as their bits
#pragma unroll
                            for (int st = 0; st < S::kSteps; ++st)
                                most = max(most, max(__float_as_uint(o[st][nt][j]) & 0x7fffffffu, __float_as_uint(o[st][nt][j + 2]) & 0x7fffffffu));
#pragma unroll
                            for (int i = 4; i < 32; i <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, i));
                            most = __float_as_uint(__fmul_rn(__uint_as_float(most), by[nt][j]));
                            up[nt][j] = min(up[nt][j], max(227 - static_cast<int>(most >> 23), 0));
                        }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        per_unit[nt][j] = __uint_as_float(__float_as_uint(per_unit[nt][j]) + (static_cast<unsigned>(up[nt][j]) << 23));
                        vf[nt][j] = in_units(value, per_unit[nt][j]);
                    }
                if (sums) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int st = 0; st < S::kSteps; ++st)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // up to 2^252 either way: in two steps
                                const int k = up[nt][j & 1] / 2;
                                o[st][nt][j] = __fmul_rn(__fmul_rn(o[st][nt][j], __fmul_rn(by[nt][j & 1], power_of_two(k))), power_of_two(up[nt][j & 1] - k));
                            }
                }
            }
            empty = false;
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    l[nt][j & 1] = __fadd_rn(l[nt][j & 1], e[nt][j]);
                    w[j] = __fmul_rn(e[nt][j], vf[nt][j & 1]);
                    if (odd_scale) w[j] = s[nt][j] == -INFINITY ? 0.0f : __int_as_float(0x7FC00000);  // hidden: its scale does not count
                }
                const uint32_t x[2] = {pack_half(w[0], w[1]), pack_half(w[2], w[3])};
                const float2 y = unpack_half(x[0]), z = unpack_half(x[1]);
                pf[0][nt][0] = transpose8(x[0]);
                pf[0][nt][1] = transpose8(x[1]);
                pf[1][nt][0] = transpose8(pack_half(w[0] - y.x, w[1] - y.y));
                pf[1][nt][1] = transpose8(pack_half(w[2] - z.x, w[3] - z.y));
            }
            const uint8_t *const vsrc = src + kTile * DIM;
#pragma unroll
            for (int i = 0; i < S::kValueChunks; ++i) {
                constexpr int kWords = S::kValueBytes / 4;
                uint32_t v[4][kWords];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // rows 2 c, 2 c + 1 and 8 further
                    const uint8_t *const at = vsrc + value_at[r & 1] + r / 2 * 8 * DIM + i * 128;
                    if constexpr (kWords == 4) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(at);
                        v[r][0] = x.x; v[r][1] = x.y; v[r][2] = x.z; v[r][3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(at);
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
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (kParts == 1) {
                                mma(o[st][nt], frag, pf[1][nt][0], pf[1][nt][1]);
                                mma(o[st][nt], frag, pf[0][nt][0], pf[0][nt][1]);
                            } else {
                                // 32-bit outputs: the tensor cores cut their sums off instead of rounding them, which over
                                // thousands of positions adds up; a tile's sum is joined by a rounded addition (relative
                                // error over 60000 positions 2.5e-6 -> below 1e-6)
                                float tile_sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma(tile_sum, frag, pf[1][nt][0], pf[1][nt][1]);
                                mma(tile_sum, frag, pf[0][nt][0], pf[0][nt][1]);
#pragma unroll
                                for (int j = 0; j < 4; ++j) o[st][nt][j] = __fadd_rn(o[st][nt][j], tile_sum[j]);
                            }
                        }
                    }
                }
            }
            src_at = src_at == (C::kStages - 1) * S::kTileBytes ? 0 : src_at + S::kTileBytes;
        }
        cp_wait<0>();
        __syncwarp();  // every lane is done with the last tile: the ring takes the next segment's
    }
    if (n_parts == 0) return;

    // ---- an item's parts are joined, in their order, by the block that arrives last at its counter
    // (that of the item's first block). Nobody waits. The code runs once: it is kept short, its
    // instructions come from memory.
    if (warp == 0) {
        __threadfence();
        __syncwarp();
        if (lane < n_parts) {
            const int first = pending[lane].begin / per, count = (pending[lane].end - 1) / per - first;
            const bool here = static_cast<int>(atomicAdd(counters + first, 1u)) == count;
            if (here) counters[first] = 0;  // for the next call
            arrived_last[lane] = here;
        }
        __threadfence();
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < n_parts; ++i) {
        if (!arrived_last[i]) continue;
        const Part done = pending[i];
        const int first = done.begin / per, n = (done.end - 1) / per - first + 1;
        // part j of the item; the first one starts inside its block's share or with it
        const float *const base = slots + 2 * static_cast<int64_t>(first) * C::kSlot, *const base0 = base + (done.begin > first * per) * C::kSlot;
        auto slot_of = [&](int j) { return j == 0 ? base0 : base + 2 * static_cast<int64_t>(j) * C::kSlot; };
        constexpr int kSets = kThreads / kRows;  // threads of a row
        float *const part_top = reinterpret_cast<float *>(q_shared), *const part_sum = part_top + kThreads;
        float *const weight = reinterpret_cast<float *>(smem);  // [part][row], where the ring was
        const int row = threadIdx.x % kRows, set = threadIdx.x / kRows;
        __syncthreads();
        float best = -INFINITY;
        // the sums of a thread's first parts are loaded beside their maxima
        constexpr int kFirst = 4;
        float first_sum[kFirst];
#pragma unroll
        for (int i = 0; i < kFirst; ++i) {
            const int j = set + i * kSets;
            first_sum[i] = j < n ? __ldcg(slot_of(j) + kRows * DIM + kRows + row) : 0.0f;
        }
#pragma unroll 4
        for (int j = set; j < n; j += kSets) {
            const float mj = __ldcg(slot_of(j) + kRows * DIM + row);
            weight[j * kRows + row] = mj;
            best = fmaxf(best, mj);
        }
        part_top[threadIdx.x] = best;
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kSets; ++s) best = fmaxf(best, part_top[s * kRows + row]);
        float mass = 0.0f;
        auto weigh = [&](int j, float lj) {
            const float mj = weight[j * kRows + row];
            const float w = joined(lj, mj, best);
            mass = __fadd_rn(mass, w);
            weight[j * kRows + row] = w;
        };
#pragma unroll
        for (int i = 0; i < kFirst; ++i)
            if (set + i * kSets < n) weigh(set + i * kSets, first_sum[i]);
#pragma unroll 1
        for (int j = set + kFirst * kSets; j < n; j += kSets) weigh(j, __ldcg(slot_of(j) + kRows * DIM + kRows + row));
        part_sum[threadIdx.x] = mass;
        __syncthreads();
        mass = 0.0f;
#pragma unroll
        for (int s = 0; s < kSets; ++s) mass = __fadd_rn(mass, part_sum[s * kRows + row]);
        if (set == 0) write_lse(p, done, group, row, best, mass);
        const float inv = inverse(mass);
        for (int j = set; j < n; j += kSets) weight[j * kRows + row] = __fmul_rn(weight[j * kRows + row], inv);
        __syncthreads();
        float *const stage = weight + (n * kRows + 3) / 4 * 4;
        const int pairs = (done.rows + 1) / 2;  // of columns that are rows
#pragma unroll 1
        for (int i = threadIdx.x; i < S::kSteps * 8 * pairs; i += kThreads) {
            const int pair = i % pairs, st = i / pairs / 8, gg = i / pairs % 8, col = 2 * pair;
            const int f = (st * NT + pair / 4) * 32 + gg * 4 + pair % 4;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            constexpr int kAhead = 32;  // loads in flight: what the join waits for is their latency
#pragma unroll 1
            for (int j0 = 0; j0 < n; j0 += kAhead) {
                float4 y[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (j0 + j < n) y[j] = __ldcg(reinterpret_cast<const float4 *>(slot_of(j0 + j)) + f);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (j0 + j < n) {
                        const float2 w = *reinterpret_cast<const float2 *>(weight + (j0 + j) * kRows + col);
                        acc.x = __fmaf_rn(y[j].x, w.x, acc.x);
                        acc.y = __fmaf_rn(y[j].y, w.y, acc.y);
                        acc.z = __fmaf_rn(y[j].z, w.x, acc.z);
                        acc.w = __fmaf_rn(y[j].w, w.y, acc.w);
                    }
                }
            }
            float *dst = stage + col * (DIM + 4) + (DIM >= 128 ? st / 8 * 128 + gg * 16 + st % 8 * 2 : gg * 8 + st * 2);
            *reinterpret_cast<float2 *>(dst) = make_float2(acc.x, acc.z);
            *reinterpret_cast<float2 *>(dst + DIM + 4) = make_float2(acc.y, acc.w);
        }
        __syncthreads();
        write_rows<T, DIM>(a, done, group, stage);
    }
}

template <typename T, int KV, int DIM, int NT, int BLOCKS>
cudaError_t launch(const Args &a, cudaStream_t s) {
    constexpr int kSmem = Config<T, DIM, NT>::kSmem;
    static PerDevice blocks;
    std::atomic<int> *const kept = blocks.here();
    int blocks_per_sm = kept ? kept->load(std::memory_order_relaxed) : 0;
    if (blocks_per_sm == 0) {
        cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<T, KV, DIM, NT, BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kv_attention_kernel<T, KV, DIM, NT, BLOCKS>, kThreads, kSmem);
        if (e != cudaSuccess) return e;
        blocks_per_sm = n < 1 ? 1 : n;
        if (kept) kept->store(blocks_per_sm, std::memory_order_relaxed);
    }
    const KvAttentionProblem &p = a.p;
    // no more blocks than the table's units could ask for
    const int64_t rows = p.tokens * (p.q_heads / p.c.heads);
    const __int128 units = static_cast<__int128>((p.width * p.c.page + kUnit - 1) / kUnit) * p.c.heads * (rows / (8 * NT) + p.seqs);
    int64_t grid = static_cast<int64_t>(num_sms()) * blocks_per_sm;
    if (grid > Config<T, DIM, NT>::kMaxBlocks) grid = Config<T, DIM, NT>::kMaxBlocks;
    if (units < grid * kMinUnits) grid = static_cast<int64_t>((units + kMinUnits - 1) / kMinUnits);
    if (grid < 1) grid = 1;
    return launch_behind(kv_attention_kernel<T, KV, DIM, NT, BLOCKS>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), kSmem, s, a);
}

template <typename T, int KV, int DIM>
cudaError_t by_rows(const Args &a, cudaStream_t s) {
    const int64_t rows = kv_block_rows(a.p.q_heads / a.p.c.heads, a.p.max_new);
    if (rows == 8) return launch<T, KV, DIM, 1, DIM <= 128 && sizeof(T) == 2 ? 3 : 2>(a, s);
    return launch<T, KV, DIM, 2, 2>(a, s);
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
    auto fours = [](const Heads &x) { return reinterpret_cast<uintptr_t>(x.p) % (4 * sizeof(T)) == 0 && x.ts % 4 == 0 && x.hs % 4 == 0; };
    return by_codes<T>(Args{p, fours(p.out), fours(p.q)}, s);
}

}  // namespace
}  // namespace om
