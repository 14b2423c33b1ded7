// w4_matvec.cuh -- products of a few rows with 4-bit weights (one translation unit for each type of x):
// y[i][j] = sum_p x[i][p] * (u[j][p] - z[j][p / group]) * s[j][p / group].
//
// Mathematics. The weights are the 16-row operand of the tensor cores' 16 x 8 x 16
// product and the rows of x its 8 columns; sums are 32 bits. A code becomes a 16-bit float by
// placing its four bits under the exponent of a power of two, u / 256 + 1/2 as bfloat16 or u +
// 1024 as float16, and loses the same float of the zero point: both exact. 16-bit x is taken in its own
// type's product; 32-bit x is three bfloat16 parts of 8 bits, one column each, so that products are
// exact to the last bit of x.
//
// Layout. Weights are read as they lie. A lane's 32-bit word of a row, eight codes, gives the
// lane's operands of two 16-deep products, taking code i and i + 4 together (one shift, one
// and-or); the same order is given to x when it is laid out in shared memory. A warp's unit is 16
// rows by 256 codes, copied ahead asynchronously with the group scales and zero points
// it needs. Groups of 4, 8 or 16 warps of a block split the codes of the same 16 rows; their sums
// are joined in shared memory, in the warps' order. x stays in shared memory, for as many
// codes at a time as fit (a slab); sums then wait in shared memory between slabs.
//
// Bound and measured (GB300; 6 790 GB/s is the measured copy bandwidth). No unit of the SM is full: issue slots 50 to 53 %,
// ALU 37 to 40 %, tensor pipe 9 to 17 %. About 11 instructions widen eight codes, in chains that four warps a scheduler
// (registers and shared memory allow no more) do not hide, and no product runs while x is laid out.
// 1 x 11008 x 4096, 32-bit x, groups of 128: 12.7 us, 1 890 GB/s (28 %), 3.6 us of it until x is laid
// out, then 1.4 us for each of up to five rounds of 16 rows; with zero points 13.1 us, and groups of 256 and more 14.9 us (their
// last group's units are copied with clipping), one group a row 16.0 us. 16 x 28669 x 8178, bfloat16, groups of 32 with zero
// points, rows at odd addresses: 77 us, 1 830 GB/s (27 %), 6 us for each of three slabs until x is laid out.
// More rows take the weights again for every 16 (5 of 32 bits): 2048 x 6144 x 4096, bfloat16, 1.40 ms.
// 1 x 1024 x 1024, float16: 3.8 us, latency. Tried and no faster: scales and zeros as a table in shared memory instead of
// between lanes (bank conflicts, 102 against 90 us), units of 128 codes (twice the instructions around them, 148 us),
// x loaded before the first copies (no change), six pieces of x a thread at a time instead of four (79 us).
#pragma once

#include <type_traits>

#include "decode_device.cuh"
#include "om_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 256;      // codes of a unit's rows
constexpr int kRowTile = 16;    // rows of a unit
constexpr int kMaxTiles = 16;   // of a pass: those whose sums wait in shared memory between slabs
constexpr int kMaxSmem = 227 * 1024 - 256;

// GB: 32-code blocks of a group within a unit: 1, 2, or 4 for groups of 128 codes and more.
template <typename T, int NT, int GB, bool ALIGNED>
struct Config {
    static constexpr int kParts = std::is_same_v<T, float> ? 3 : 1;  // columns of a row of x
    static constexpr int kCols = 8 * NT;
    static constexpr int kTokens = kCols / kParts;                 // rows of x a block takes
    static constexpr int kRowPieces = ALIGNED ? 8 : 9;             // 16-byte pieces that hold a unit's row
    static constexpr int kPieces = (kRowTile * kRowPieces + 31) / 32;  // of a lane
    static constexpr int kScaleWords = 8 / GB, kZeroWords = GB == 1 ? 4 : 2;  // that hold a row's scales and zeros
    static constexpr int kScaleAt = kRowTile * kRowPieces * 16, kZeroAt = kScaleAt + kRowTile * kScaleWords * 4;
    static constexpr int kStages = NT == 1 ? 3 : 2;
    static constexpr int kStage = kZeroAt + kRowTile * kZeroWords * 4;
    static_assert(kStage % 128 == 0, "places of words in a stage are whole multiples of 128 bytes apart");
    static constexpr int kRing = kStages * kStage;                 // of one warp
    static constexpr int kJoinWarps = kParts == 3 ? kTokens : NT;  // that join a tile's sums
    static constexpr int kJoins = NT == 1 ? 2 : 1;                 // buffers of the sums of all warps
    static constexpr int kJoin = kJoins * kWarps * NT * 32 * 16;
    static constexpr int kAcc = kMaxTiles * kRowTile * kTokens * 4;
    static constexpr int kFixed = kWarps * kRing + kJoin + kAcc;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// The bytes [base, src + left) of a piece that begins at src, before the operand's first byte.
__device__ __noinline__ void copy_bytes(uint32_t to, const uint8_t *src, const uint8_t *base, int left) {
#pragma unroll 1
    for (int e = static_cast<int>(base - src); e < left; ++e) asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + e), "r"(static_cast<uint32_t>(src[e])) : "memory");
}

// d = a b, or d + a b.
template <bool HALF>
__device__ __forceinline__ void product(float *d, const uint32_t *a, uint32_t b0, uint32_t b1, bool first) {
    const float e[4] = {first ? 0.0f : d[0], first ? 0.0f : d[1], first ? 0.0f : d[2], first ? 0.0f : d[3]};
    if constexpr (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(e[0]), "f"(e[1]), "f"(e[2]), "f"(e[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(e[0]), "f"(e[1]), "f"(e[2]), "f"(e[3]));
}

// Codes i and i + 4 of a word as two 16-bit floats: u + 1024 (float16), u / 256 + 1/2 (bfloat16,
// where x can be so large that its products with u would overflow a sum that its scale makes small).
template <int I>
__device__ __forceinline__ uint32_t widen(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)), "r"(mask), "r"(magic));  // (w & mask) | magic
    return r;
}

template <bool HALF>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    std::conditional_t<HALF, __half2, __nv_bfloat162> x, y;
    memcpy(&x, &a, 4);
    memcpy(&y, &b, 4);
    x = __hsub2(x, y);
    memcpy(&a, &x, 4);
    return a;
}

struct Args {
    W4Problem p;
    int tiles;     // of 16 rows
    int units;     // of 256 codes
    int slab;      // units whose x a block holds at once
    int wide;      // a group's halves of a unit (128 codes), for groups of 128 codes and more
    int split;     // warps that share 16 rows: 4, 8 or 16
    int x_bytes;   // alignment of the rows of x: 16, 4 or 2 bytes
};

// The exponent that scales a row whose largest magnitude has these bits.
__device__ __forceinline__ int exponent(unsigned top) { return min(max(static_cast<int>(top >> 23) - 127, -126), 127); }

// Three bfloat16 parts of a 32-bit float, each the leading 8 bits of what is left (cut off, so that
// nothing overflows); the parts of an infinity are itself and zeros, those of a NaN itself.
__device__ __forceinline__ void split3(float x, uint16_t *part) {
    const uint32_t b = __float_as_uint(x);
    if ((b & 0x7f800000u) == 0x7f800000u) {
        part[0] = (b & 0x007fffffu) ? 0x7fc0 : static_cast<uint16_t>(b >> 16);
        part[1] = part[2] = 0;
        return;
    }
    const float r1 = x - __uint_as_float(b & 0xffff0000u);
    const uint32_t b1 = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(b1);
    part[0] = static_cast<uint16_t>(b >> 16);
    part[1] = static_cast<uint16_t>(b1 >> 16);
    part[2] = static_cast<uint16_t>(__float_as_uint(r2) >> 16);
}

// The first `valid` of eight elements as they lie in memory, zeros behind them.
template <typename T>
__device__ __noinline__ void load_part(const T *src, int valid, uint32_t *raw) {
    uint32_t v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v[e] = 0;
        if (e < valid) {
            if constexpr (sizeof(T) == 4) v[e] = __float_as_uint(src[e]);
            else v[e] = reinterpret_cast<const uint16_t *>(src)[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 4) raw[e] = v[e];
        else if (e % 2 == 0) raw[e / 2] = v[e] | v[e + 1] << 16;
    }
}

template <typename T, int NT, int GB, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 1) w4_matvec_kernel(const __grid_constant__ Args a) {
    using C = Config<T, NT, GB, ALIGNED>;
    constexpr bool kHalf = std::is_same_v<T, __half>, kWhole = std::is_same_v<T, float>;
    constexpr uint32_t kMagic = kHalf ? 0x64006400u : 0x3f003f00u;  // a code of 0, twice
    constexpr float kCode = kHalf ? 1.0f : 1.0f / 256.0f;           // a code's step
    constexpr int kGroups = 8 / GB;                                 // of a unit
    const W4Problem &p = a.p;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, g = lane / 4, c = lane % 4;
    const int n = static_cast<int>(p.n), k = static_cast<int>(p.k);
    const int groups = static_cast<int>((p.k + p.group - 1) / p.group);
    const int64_t row_bytes = (p.k + 1) / 2;
    const int scale_bytes = p.s_dtype == OM_F32 ? 4 : 2;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ unsigned row_top[C::kTokens];
    const uint32_t ring = smem_u32(smem) + warp * C::kRing;
    float4 *const join = reinterpret_cast<float4 *>(smem + kWarps * C::kRing);
    float *const acc_rows = reinterpret_cast<float *>(smem + kWarps * C::kRing + C::kJoin);
    uint8_t *const xs = smem + C::kFixed;  // [column][block][c]: 8 elements, 16 bytes
    const int tokens = min(C::kTokens, static_cast<int>(p.m) - static_cast<int>(blockIdx.y) * C::kTokens);
    const int cols = tokens * C::kParts;
    const int x_stride = a.slab * kUnit * 2 + 64;
    const T *const x = static_cast<const T *>(p.x) + static_cast<int64_t>(blockIdx.y) * C::kTokens * p.ldx;
    T *const y = static_cast<T *>(p.y) + static_cast<int64_t>(blockIdx.y) * C::kTokens * p.ldy;

    // this block's tiles, and this warp's place: team of a tile, part of its codes
    const int t_begin = static_cast<int>(static_cast<int64_t>(a.tiles) * blockIdx.x / gridDim.x);
    const int t_end = static_cast<int>(static_cast<int64_t>(a.tiles) * (blockIdx.x + 1) / gridDim.x);
    const int teams = kWarps / a.split, team = warp / a.split, part = warp - team * a.split;
    auto team_barrier = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(a.split * 32) : "memory"); };
    // the first group of a unit
    auto group_of = [&](int unit) -> int {
        if (GB < 4) return unit * kGroups;
        return a.wide == 1 ? unit * 2 : static_cast<int>(static_cast<unsigned>(unit * 2) / static_cast<unsigned>(a.wide));
    };

    // A row's place in the 16-byte pieces and 4-byte words that are copied: it depends on the row's number
    // in its tile only, 16 rows being a whole number of pieces and words. Offsets within a tile are below
    // 2^31. The operands' first piece and words may begin before the operands.
    const uint8_t *const w_pieces = p.u - (reinterpret_cast<uintptr_t>(p.u) & 15);
    const uint8_t *const s_words = static_cast<const uint8_t *>(p.s) - (reinterpret_cast<uintptr_t>(p.s) & 3);
    const uint8_t *const z_words = p.z - (reinterpret_cast<uintptr_t>(p.z) & 3);
    const int ldu = static_cast<int>(p.ldu), lds = static_cast<int>(p.lds) * scale_bytes, ldz = static_cast<int>(p.ldz);
    const int u_low = static_cast<int>(reinterpret_cast<uintptr_t>(p.u) & 15);
    const int s_low = static_cast<int>(reinterpret_cast<uintptr_t>(p.s) & 3), z_low = static_cast<int>(reinterpret_cast<uintptr_t>(p.z) & 3);
    const int64_t w_step = teams * kRowTile * p.ldu, s_step = teams * kRowTile * p.lds * scale_bytes, z_step = teams * kRowTile * p.ldz;
    int w_at[C::kPieces], w_left[C::kPieces], s_at[kGroups / 2], z_at[C::kZeroWords / 2];
#pragma unroll
    for (int i = 0; i < C::kPieces; ++i) {
        const int q = lane + 32 * i, r = q / C::kRowPieces, off = (q - C::kRowPieces * r) * 16 - (ALIGNED ? 0 : (u_low + r * ldu) & 15);
        w_at[i] = r * ldu + off;
        w_left[i] = static_cast<int>(row_bytes) - off;
    }
#pragma unroll
    for (int i = 0; i < kGroups / 2; ++i) s_at[i] = s_low + (lane + 32 * i) / C::kScaleWords * lds;
#pragma unroll
    for (int i = 0; i < C::kZeroWords / 2; ++i) z_at[i] = z_low + (lane + 32 * i) / C::kZeroWords * ldz;
    // for rows g and g + 8, as they are read
    int skew[2], s_row[2], z_row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        skew[r] = (u_low + (g + 8 * r) * ldu) & 15;
        s_row[r] = (s_low + (g + 8 * r) * lds) & 3;
        z_row[r] = (z_low + (g + 8 * r) * ldz) & 3;
    }

    wait_for_earlier();
    int turn = 0;
    for (int pass = t_begin; pass < t_end; pass += kMaxTiles) {
        const int pass_tiles = min(kMaxTiles, t_end - pass);
        for (int slab = 0; slab < a.units; slab += a.slab) {
            const int slab_units = min(a.slab, a.units - slab);
            const int mine = slab_units > part ? (slab_units - part + a.split - 1) / a.split : 0;  // of a tile

            // ---- the copies of unit after unit: the team's tiles, this warp's units of each
            int f_tile = team, f_i = 0, f_stage = 0;
            const uint8_t *f_w = p.u + static_cast<int64_t>(pass + team) * kRowTile * p.ldu;  // of the tile
            const uint8_t *f_s = s_words + static_cast<int64_t>(pass + team) * kRowTile * p.lds * scale_bytes;
            const uint8_t *f_z = z_words + static_cast<int64_t>(pass + team) * kRowTile * p.ldz;
            auto fetch = [&]() {
                if (f_tile < pass_tiles && mine > 0) {
                    const uint32_t dst = ring + f_stage * C::kStage;
                    const int unit = slab + part + f_i * a.split, byte0 = unit * (kUnit / 2), grp = group_of(unit);
                    const int rows = n - (pass + f_tile) * kRowTile;  // that the matrix has, from the tile's first
                    auto piece_to = [&](int q) {
                        // ALIGNED: the pieces of a row in an order that keeps the reads of one block's words
                        // by all lanes off each other's banks
                        const int r = q / C::kRowPieces;
                        return dst + (ALIGNED ? r * 128 + (((q ^ r) & 7) * 16) : q * 16);
                    };
                    if (rows >= kRowTile + 3 && grp + kGroups <= groups && (grp > 0 || pass + f_tile > 0)) {
                        // Every group is there, and there are rows behind the tile's and groups before it: what is
                        // copied beyond a row's ends lies inside the operands (three rows: two zero points a row, eight
                        // bytes copied). Codes behind k meet zeros of x.
#pragma unroll
                        for (int i = 0; i < C::kPieces; ++i) {
                            const int q = lane + 32 * i;
                            if (ALIGNED || i + 1 < C::kPieces || q < kRowTile * C::kRowPieces) copy16(piece_to(q), f_w + (w_at[i] + byte0), 16);
                        }
#pragma unroll
                        for (int i = 0; i < kGroups / 2; ++i) {
                            const int q = lane + 32 * i;
                            copy4(dst + C::kScaleAt + q * 4, f_s + (((s_at[i] + grp * scale_bytes) & ~3) + q % C::kScaleWords * 4), 4);
                        }
                        if (p.z) {
#pragma unroll
                            for (int i = 0; i < C::kZeroWords / 2; ++i) {
                                const int q = lane + 32 * i;
                                copy4(dst + C::kZeroAt + q * 4, f_z + (((z_at[i] + grp) & ~3) + q % C::kZeroWords * 4), 4);
                            }
                        }
                    } else {
                        const bool head = grp == 0 && pass + f_tile == 0;  // wide groups: the first one goes on in later units
                        auto clipped = [&](uint32_t to, const uint8_t *tile, int at, const uint8_t *base, const uint8_t *aligned, int left, auto size) {
                            constexpr int kSize = decltype(size)::value;
                            left = min(max(left, 0), kSize);
                            const uint8_t *const src = left > 0 ? tile + at : aligned;
                            if (head && left > 0 && src < base) copy_bytes(to, src, base, left);
                            else if constexpr (kSize == 16) copy16(to, src, left);
                            else copy4(to, src, left);
                        };
#pragma unroll
                        for (int i = 0; i < C::kPieces; ++i) {
                            const int q = lane + 32 * i;
                            if (ALIGNED || i + 1 < C::kPieces || q < kRowTile * C::kRowPieces)
                                clipped(piece_to(q), f_w, w_at[i] + byte0, p.u, w_pieces, q / C::kRowPieces < rows ? w_left[i] - byte0 : 0, std::integral_constant<int, 16>{});
                        }
#pragma unroll
                        for (int i = 0; i < kGroups / 2; ++i) {
                            const int q = lane + 32 * i, word = q % C::kScaleWords * 4, at = s_at[i] + grp * scale_bytes;
                            clipped(dst + C::kScaleAt + q * 4, f_s, (at & ~3) + word, static_cast<const uint8_t *>(p.s), s_words,
                                    q / C::kScaleWords < rows ? min(groups - grp, kGroups) * scale_bytes + (at & 3) - word : 0, std::integral_constant<int, 4>{});
                        }
                        if (p.z) {
#pragma unroll
                            for (int i = 0; i < C::kZeroWords / 2; ++i) {
                                const int q = lane + 32 * i, word = q % C::kZeroWords * 4, at = z_at[i] + grp;
                                clipped(dst + C::kZeroAt + q * 4, f_z, (at & ~3) + word, p.z, z_words, q / C::kZeroWords < rows ? min(groups - grp, kGroups) + (at & 3) - word : 0,
                                        std::integral_constant<int, 4>{});
                            }
                        }
                    }
                    f_stage = f_stage == C::kStages - 1 ? 0 : f_stage + 1;
                    if (++f_i == mine) {
                        f_i = 0;
                        f_tile += teams;
                        f_w += w_step;
                        f_s += s_step;
                        f_z += z_step;
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            const bool fresh = pass == t_begin || a.units > a.slab;  // x has to be laid out
            __syncthreads();  // the last slab's x has been used
            if (kWhole && fresh && threadIdx.x < C::kTokens) row_top[threadIdx.x] = 0;

            // One loop runs the copies ahead, then x once they are on their way, then unit after unit:
            // its code comes from memory, and a block runs little more than it once.
            uint32_t mask, magic;  // in registers: an instruction takes one constant
            asm volatile("mov.b32 %0, 0x000f000f;\n\tmov.b32 %1, %2;" : "=r"(mask), "=r"(magic) : "n"(kMagic));
            const uint8_t *x_lane[NT];  // of x: the columns behind the last one repeat it
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x_lane[nt] = xs + min(nt * 8 + g, cols - 1) * x_stride + c * 16;
            int tile = team, unit_i = 0, stage = 0;
            float total[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) total[nt][j] = 0.0f;
#pragma unroll 1
            for (int step = -C::kStages; step < 0 || tile < pass_tiles; ++step) {
            if (step < 0) {
                fetch();
                if (step < -1) continue;
                // ---- x: eight consecutive elements in the order of a word's codes, zero behind k; a thread takes
                // some such pieces at a time, whose loads are in flight together. For 32-bit x once before that: a row's
                // largest element sets its power of two, so that no part of x is lost at the ends of the range.
                if (fresh) {
                    constexpr int kBatch = kWhole ? 2 : 4, kRaw = kWhole ? 8 : 4;
                    const int pieces = slab_units * (kUnit / 8), count = pieces * tokens;  // pieces is a multiple of 32
                    uint32_t raw[kBatch][kRaw];
                    if (kWhole) __syncthreads();
#pragma unroll 1
                    for (int base = 0, look = kWhole; base < count; base += kBatch * kThreads) {
                        if (!kWhole || look || count > kBatch * kThreads) {  // else they are still there
#pragma unroll
                            for (int j = 0; j < kBatch; ++j) {
                                const int i = base + j * kThreads + threadIdx.x, tok = i / pieces, k0 = slab * kUnit + (i - tok * pieces) * 8;
                                const T *src = x + tok * p.ldx + k0;
                                if (i < count && k0 + 8 <= k && a.x_bytes == 16) {
#pragma unroll
                                    for (int e = 0; e < kRaw; e += 4) {
                                        const uint4 v = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint32_t *>(src) + e);
                                        raw[j][e] = v.x;
                                        raw[j][e + 1] = v.y;
                                        raw[j][e + 2] = v.z;
                                        raw[j][e + 3] = v.w;
                                    }
                                } else if (i < count && a.x_bytes >= 4) {  // words, the last one's second element behind k or not
                                    constexpr int kOf = 4 / sizeof(T);
#pragma unroll
                                    for (int e = 0; e < kRaw; ++e) {
                                        raw[j][e] = 0;
                                        if (k0 + kOf * (e + 1) <= k) raw[j][e] = reinterpret_cast<const uint32_t *>(src)[e];
                                        else if (kOf == 2 && k0 + 2 * e < k) raw[j][e] = reinterpret_cast<const uint16_t *>(src)[2 * e];
                                    }
                                } else if (i >= count || k0 >= k) {
#pragma unroll
                                    for (int e = 0; e < kRaw; ++e) raw[j][e] = 0;
                                } else {
                                    uint32_t part_of[kRaw];
                                    load_part<T>(src, k - k0, part_of);
#pragma unroll
                                    for (int e = 0; e < kRaw; ++e) raw[j][e] = part_of[e];
                                }
                            }
                        }
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) {
                            const int i = base + j * kThreads + threadIdx.x;
                            if (i >= count) break;
                            const int tok = i / pieces;
                            uint8_t *dst = xs + tok * C::kParts * x_stride + (i - tok * pieces) * 16;
                            if constexpr (kWhole) {
                                if (look) {
                                    unsigned top = 0;
#pragma unroll
                                    for (int e = 0; e < 8; ++e) top = max(top, raw[j][e] & 0x7fffffffu);
                                    top = __reduce_max_sync(0xffffffffu, top);
                                    if (lane == 0) atomicMax(&row_top[tok], top);
                                } else {
                                    const float up = __uint_as_float(static_cast<unsigned>(128 - exponent(row_top[tok])) << 23);
                                    uint32_t w[3][4];
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        uint16_t lo[3], hi[3];
                                        split3(__uint_as_float(raw[j][e]) * up, lo);
                                        split3(__uint_as_float(raw[j][e + 4]) * up, hi);
#pragma unroll
                                        for (int q = 0; q < 3; ++q) w[q][e] = lo[q] | static_cast<uint32_t>(hi[q]) << 16;
                                    }
#pragma unroll
                                    for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4 *>(dst + q * x_stride) = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
                                }
                            } else {
                                *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(raw[j][0], raw[j][2], 0x5410), __byte_perm(raw[j][0], raw[j][2], 0x7632),
                                                                             __byte_perm(raw[j][1], raw[j][3], 0x5410), __byte_perm(raw[j][1], raw[j][3], 0x7632));
                            }
                        }
                        if (look && base + kBatch * kThreads >= count) {
                            look = 0;
                            base = -kBatch * kThreads;
                            __syncthreads();
                        }
                    }
                }
                __syncthreads();
                continue;
            }
                // ---- a unit
                if (mine > 0) {
                    const int unit = part + unit_i * a.split;  // of the slab
                    asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 1) : "memory");
                    __syncwarp();
                    const uint8_t *const held = smem + warp * C::kRing + stage * C::kStage;
                    const int grp = group_of(slab + unit);
                    // a wide group goes on in the unit's second half, or the next one begins
                    const int second_half = GB < 4 || a.wide == 1 ? 1 : static_cast<int>(static_cast<unsigned>((slab + unit) * 2 + 1) / static_cast<unsigned>(a.wide)) - grp;
                    // lane c has the scales and zero points of groups c and c + 4 of rows g and g + 8
                    constexpr int kHeld = kGroups == 8 ? 2 : 1;
                    float held_s[kHeld][2];
                    uint32_t held_z[kHeld];
#pragma unroll
                    for (int j = 0; j < kHeld; ++j) {
                        const int of = min(c, kGroups - 1) + 4 * j;
                        uint32_t z[2] = {8, 8};
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const uint8_t *const at = held + C::kScaleAt + (g + 8 * r) * (C::kScaleWords * 4) + ((s_row[r] + grp * scale_bytes) & 3) + of * scale_bytes;
                            if (scale_bytes == 4) held_s[j][r] = *reinterpret_cast<const float *>(at);
                            else if (p.s_dtype == OM_F16) held_s[j][r] = __half2float(*reinterpret_cast<const __half *>(at));
                            else held_s[j][r] = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(at)) << 16);
                            if (p.z) z[r] = held[C::kZeroAt + (g + 8 * r) * (C::kZeroWords * 4) + ((z_row[r] + grp) & 3) + of];
                        }
                        held_z[j] = kMagic | z[0] | z[1] << 16;
                    }
                    // ALIGNED: the word of block 0; stages are whole multiples of 128 bytes
                    const uint32_t w_lane = ALIGNED ? g * 128 + (g & 7) * 16 + c * 4 : g * 144 + c * 4;
                    float acc[NT][4];
                    uint32_t off0 = 0, off1 = 0;
                    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        if (b % GB == 0) {  // a group begins
                            int j = b / GB;
                            if (GB == 4 && b == 4) j = second_half;
                            const int from = (lane & ~3) + j % 4;
                            s0 = __shfl_sync(0xffffffffu, held_s[b / GB / 4][0], from);
                            s1 = __shfl_sync(0xffffffffu, held_s[b / GB / 4][1], from);
                            const uint32_t z = __shfl_sync(0xffffffffu, held_z[b / GB / 4], from);
                            off0 = __byte_perm(z, 0, 0x1010);
                            off1 = __byte_perm(z, 0, 0x3232);
                        }
                        uint32_t w0, w1;
                        if constexpr (ALIGNED) {
                            const uint8_t *const at = held + (w_lane ^ (b * 16));
                            w0 = *reinterpret_cast<const uint32_t *>(at);
                            w1 = *reinterpret_cast<const uint32_t *>(at + 1024);  // (g + 8) ^ b: the same place
                        } else {
                            auto word = [&](const uint8_t *at, int off) {
                                return __funnelshift_r(*reinterpret_cast<const uint32_t *>(at + (off & ~3)), *reinterpret_cast<const uint32_t *>(at + ((off + 3) & ~3)), off * 8);
                            };
                            w0 = word(held + w_lane + b * 16, skew[0]);
                            w1 = word(held + w_lane + b * 16 + 8 * 144, skew[1]);
                        }
                        uint32_t f[2][4] = {{widen<0>(w0, mask, magic), widen<0>(w1, mask, magic), widen<1>(w0, mask, magic), widen<1>(w1, mask, magic)},
                                            {widen<2>(w0, mask, magic), widen<2>(w1, mask, magic), widen<3>(w0, mask, magic), widen<3>(w1, mask, magic)}};
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[q][e] = sub2<kHalf>(f[q][e], e & 1 ? off1 : off0);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(x_lane[nt] + (unit * 8 + b) * 64);
                            product<kHalf>(acc[nt], f[0], v.x, v.y, b % GB == 0);
                            product<kHalf>(acc[nt], f[1], v.z, v.w, false);
                        }
                        if (b % GB == GB - 1) {  // and ends
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                total[nt][0] = __fmaf_rn(s0, acc[nt][0], total[nt][0]);
                                total[nt][1] = __fmaf_rn(s0, acc[nt][1], total[nt][1]);
                                total[nt][2] = __fmaf_rn(s1, acc[nt][2], total[nt][2]);
                                total[nt][3] = __fmaf_rn(s1, acc[nt][3], total[nt][3]);
                            }
                        }
                    }
                    __syncwarp();  // the stage has been read by every lane
                    fetch();
                    stage = stage == C::kStages - 1 ? 0 : stage + 1;
                    if (++unit_i < mine) continue;
                    unit_i = 0;
                }
                // ---- the team's sums of the tile
                if constexpr (C::kJoins == 1) team_barrier();  // the last tile's sums have been read
                float4 *const sums = join + (C::kJoins == 1 ? 0 : (turn & 1) * (kWarps * NT * 32));
                ++turn;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) sums[(warp * NT + nt) * 32 + lane] = make_float4(total[nt][0], total[nt][1], total[nt][2], total[nt][3]);
                team_barrier();
                auto finish = [&](int tok, int r, float sum) {
                    sum *= 1.0f / kCode;
                    if constexpr (kWhole) {  // 2^(e - 1): e can be -126
                        const int e = exponent(row_top[tok]);
                        sum *= e > -126 ? __uint_as_float(static_cast<unsigned>(e + 126) << 23) : __uint_as_float(0x00400000u);
                    }
                    // the rows' sums of earlier slabs
                    float *const kept = acc_rows + (tile * C::kTokens + tok) * kRowTile + r;
                    if (slab > 0) sum += *kept;
                    if (slab + a.slab < a.units) {
                        *kept = sum;
                    } else {
                        const int row = (pass + tile) * kRowTile + r;
                        if (row < n) y[tok * p.ldy + row] = from_float<T>(sum);
                    }
                };
                // the joining warps take turns
                int first = part - turn * C::kJoinWarps;
                first = (first % a.split + a.split) % a.split;
                const float4 *const of_team = sums + team * a.split * NT * 32;
                if constexpr (kWhole) {
                    // two lanes an output, each half of the warps
                    for (int id = first * 32 + lane; id < 2 * kRowTile * tokens; id += a.split * 32) {
                        const int r = id % kRowTile, half = id / kRowTile % 2, tok = id / (2 * kRowTile);
                        float sum = 0.0f;
#pragma unroll
                        for (int j = 0; j < C::kParts; ++j) {
                            const int cc = tok * C::kParts + j;
                            const float *from = reinterpret_cast<const float *>(of_team + (cc / 8) * 32 + (r % 8) * 4 + cc % 8 / 2) + (cc & 1) + (r / 8) * 2;
#pragma unroll
                            for (int w = 0; w < 8; ++w)
                                if (w < a.split / 2) sum += from[(half * (a.split / 2) + w) * NT * 128];
                        }
                        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                        if (!half) finish(tok, r, sum);
                    }
                } else if (first < NT) {
                    // a lane's four sums: rows g and g + 8, columns 2 c and 2 c + 1
                    float4 sum = of_team[first * 32 + lane];
#pragma unroll 3
                    for (int w = 1; w < a.split; ++w) {
                        const float4 v = of_team[(w * NT + first) * 32 + lane];
                        sum.x += v.x;
                        sum.y += v.y;
                        sum.z += v.z;
                        sum.w += v.w;
                    }
                    const int tok = first * 8 + 2 * c;
                    if (tok < tokens) {
                        finish(tok, g, sum.x);
                        finish(tok, g + 8, sum.z);
                    }
                    if (tok + 1 < tokens) {
                        finish(tok + 1, g, sum.y);
                        finish(tok + 1, g + 8, sum.w);
                    }
                }
                tile += teams;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) total[nt][j] = 0.0f;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
    }
}

template <typename T>
__global__ void fill_zero_kernel(T *y, int64_t m, int64_t n, int64_t ldy) {
    const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (j < n) y[blockIdx.y * ldy + j] = from_float<T>(0.0f);
}

template <typename T, int NT, int GB, bool ALIGNED>
cudaError_t launch(Args a, cudaStream_t s) {
    using C = Config<T, NT, GB, ALIGNED>;
    static PerDevice ready;
    std::atomic<int> *const is_ready = ready.here();
    if (!is_ready || !is_ready->load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(w4_matvec_kernel<T, NT, GB, ALIGNED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
        if (is_ready) is_ready->store(1, std::memory_order_relaxed);
    }
    // x in shared memory: all of it, or as many units at a time as fit, in slabs of equal size
    const int64_t tokens = a.p.m < C::kTokens ? a.p.m : C::kTokens, cols = tokens * C::kParts, per_unit = cols * kUnit * 2;
    const int64_t most = (kMaxSmem - C::kFixed - cols * 64) / per_unit;
    static_assert(kMaxSmem - C::kFixed >= C::kCols * (kUnit * 2 + 64), "a unit of x fits");
    const int64_t slabs = (a.units + most - 1) / most;
    int64_t slab = ((a.units + slabs - 1) / slabs + 3) / 4 * 4;
    if (slab > most) slab = most;
    a.slab = static_cast<int>(a.units < slab ? a.units : slab);
    const int sms = num_sms();
    const dim3 grid(static_cast<unsigned>(a.tiles < sms ? a.tiles : sms), static_cast<unsigned>((a.p.m + C::kTokens - 1) / C::kTokens));
    // Warps that share a tile: the fewest rounds of units; of those the smallest team, which joins least.
    const int64_t of_block = (a.tiles + grid.x - 1) / grid.x;
    int64_t best = 0;
    for (int split = 4; split <= kWarps; split *= 2) {
        const int64_t rounds = (of_block + kWarps / split - 1) / (kWarps / split) * ((a.slab + split - 1) / split);
        if (split == 4 || rounds < best) {
            best = rounds;
            a.split = split;
        }
    }
    const int64_t smem = C::kFixed + cols * 64 + a.slab * per_unit;
    return launch_behind(w4_matvec_kernel<T, NT, GB, ALIGNED>, grid, dim3(kThreads), static_cast<size_t>(smem), s, a);
}

template <typename T, int NT, int GB>
cudaError_t by_alignment(const Args &a, cudaStream_t s) {
    return reinterpret_cast<uintptr_t>(a.p.u) % 16 == 0 && (a.p.n == 1 || a.p.ldu % 16 == 0) ? launch<T, NT, GB, true>(a, s) : launch<T, NT, GB, false>(a, s);
}

template <typename T, int NT>
cudaError_t by_group(const Args &a, cudaStream_t s) {
    if (a.p.group == 32) return by_alignment<T, NT, 1>(a, s);
    return a.p.group == 64 ? by_alignment<T, NT, 2>(a, s) : by_alignment<T, NT, 4>(a, s);
}

template <typename T>
cudaError_t run_w4_matvec(const W4Problem &p, cudaStream_t s) {
    if (p.k == 0) {
        fill_zero_kernel<T><<<dim3(static_cast<unsigned>((p.n + 255) / 256), static_cast<unsigned>(p.m)), 256, 0, s>>>(static_cast<T *>(p.y), p.m, p.n, p.ldy);
        return cudaGetLastError();
    }
    Args a{};
    a.p = p;
    a.tiles = static_cast<int>((p.n + kRowTile - 1) / kRowTile);
    a.units = static_cast<int>((p.k + kUnit - 1) / kUnit);
    a.wide = p.group >= 128 ? static_cast<int>(p.group / 128) : 1;
    const uintptr_t x_low = reinterpret_cast<uintptr_t>(p.x) | (p.m == 1 ? 0 : static_cast<uintptr_t>(p.ldx) * sizeof(T));
    a.x_bytes = x_low % 16 == 0 ? 16 : (x_low % 4 == 0 ? 4 : 2);
    constexpr int kParts = std::is_same_v<T, float> ? 3 : 1;
    if (p.m <= 8 / kParts) return by_group<T, 1>(a, s);
    return by_group<T, 2>(a, s);
}

}  // namespace
}  // namespace om
