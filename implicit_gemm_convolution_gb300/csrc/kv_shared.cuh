// kv_shared.cuh -- attention of many sequences to a prefix that they share, read once for all of them; one
// translation unit for each type of codes (kv_shared_*.cu). The sequences' own tokens are kv_attention.cuh's, as a part of
// the same softmax; kv_shared_join.cu puts the parts together.
//
// Mathematics. As in kv_attention.cuh: keys c_t a, values e_t s, x_t = (q . c_t) a scale log2(e),
// out = sum_t 2^(x_t - m) s e_t / sum_t 2^(x_t - m). The rows are the tokens of all sequences of a group times the
// query heads of a key head, so the products are as large as a library's and run on tcgen05: S = Q C^T, O += P E
// for 128 rows and a tile of 64 positions, sums in tensor memory. Codes are exact in 16-bit floats, queries are scaled
// by a power of two for each row (32-bit ones in two parts of 11 bits), weights 2^(x - m) s / u go in two parts of 11 bits
// with a power-of-two unit u for each row, set anew when a tile's largest weight leaves [2^-1, 2^15]: a weight is off by no more
// than 2^-22 of itself or 2^-24 of its tile's largest. Pages of one tile whose value scales are too far apart for one unit are
// taken one after the other: the tile comes again for each, with the others hidden.
//
// Block (16 warps, two blocks an SM for heads of up to 128), on tiles of 64 positions:
//   warps 0-3   a row of scores a thread: the tile's maximum from tensor memory, then weights, whose parts replace the scores as the
//               second product's operand; rows of sums are multiplied only when a unit or maximum changes; queries in, sums out. 32-bit calls' sums, and those
//               of long parts, leave tensor memory every few tiles: the tensor cores cut sums off, the more the longer they grow.
//   warps 4-11  codes of keys (4-7) and values from the pages, the next tile's on their way, to 16-bit floats in shared memory: rows of
//               128 bytes with the tensor cores' exclusive-or, the same layout for both (k-major and n-major operands).
//   warp 12     tensor memory, and one lane that issues the products: the next tile's scores beside the rows' work on this one.
//   warp 13     finds the block's parts of items;  warp 14 lays out the tiles' scales.
// Every mbarrier wait is bounded; on a timeout the block records the error, stops and frees its tensor memory.
//
// Split. The tiles of all items (group, key head, 128 rows) in equal shares of the blocks that fit at once, as lengths on the
// device give them. A block's part of a cut item goes to one of its two slots, a whole item to its rows' places;
// the join finds them by the same arithmetic. Nobody waits for another block.
//
// Bound and measured (GB300). What the rows issue: a score costs a maximum, an exponential, its part of a sum, two conversions to 16 bits and the
// difference between them, and two blocks an SM fill each other's waits. 64 sequences behind a prefix of 32768 tokens (8 key heads of 128, 8 query
// heads each, bfloat16): this kernel 118 us, with the own tokens and the join 154 us; the tensor cores are busy 57 % of it, issue slots 66 %. The
// prefix is read once (67 MB of keys and values, 10 us at the copy bandwidth). One token of each sequence over the same prefix by kv_attention.cuh
// reads it 64 times. 40 sequences with drafts of 32-bit queries, which go in two parts, behind three prefixes of 8001 tokens: 92 us of 132 (with all of a part's sums
// in tensor memory 53 of 90, and errors to 9e-6 behind long prefixes, where they are 2e-6 now). Tiles of 128 positions with one block an SM ran
// slower (nothing to fill the waits of the rows). Registers by warpgroup (88 for rows, 56 for copies): with equal shares the rows spill, and loads
// that wait for a spilled register no longer run ahead.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "attention_range.cuh"
#include "decode_device.cuh"
#include "kv_shared_items.cuh"
#include "om_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

// four warpgroups, which registers are handed out by: rows, keys, values, and the warps that steer
constexpr int kRowWarps = 4, kCopyWarps = 4;  // copy warps: of keys, and as many of values
constexpr int kProductWarp = kRowWarps + 2 * kCopyWarps, kWalkWarp = kProductWarp + 1, kScaleWarp = kWalkWarp + 1;
constexpr int kThreads = 512;
constexpr int kSharedFold = 4;  // tiles of 32-bit calls whose sums stay in tensor memory

// Instruction descriptor of tcgen05.mma kind::f16: D fp32 (bit 4), A and B fp16 (0), B n-major where
// asked (bit 16), N >> 3 in bits 17-22, M >> 4 in bits 24-28.
constexpr uint32_t descriptor_of(int n, bool b_n_major) {
    return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kSharedRows >> 4) << 24);
}

// PARTS: of a query. Shared memory holds two blocks of an SM (heads of 256: one), tensor memory the scores of two tiles and the sums.
template <int DIM, int PARTS>
struct Config {
    static constexpr int kPos = kSharedTile;
    static constexpr int kQPart = kSharedRows * DIM * 2;
    static constexpr int kQBytes = PARTS * kQPart;
    static constexpr int kTile = kPos * DIM * 2;
    static constexpr int kTiles = DIM * PARTS > 256 || (DIM == 128 && PARTS == 2) ? 1 : 2;  // of keys and of values: as many as fit
    static constexpr int kSmem = 1024 + kQBytes + 2 * kTiles * kTile;
    static constexpr int kColumns = 2 * kPos + DIM <= 256 ? 256 : 512;
    static constexpr int kGroups = kPos / 16;  // 16 positions have one page
    static constexpr uint32_t kScores = descriptor_of(kPos, false), kSums = descriptor_of(DIM, true);
};

// Shared-memory descriptor, 128-byte swizzle (layout 2), version 1: groups of 8 rows 1024 bytes apart (stride byte
// offset); n-major operands: 64 columns, then `block` bytes on to the next 64 (leading byte offset).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t block) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(block >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add, bool leader) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a),
                 "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
                 : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add, bool leader) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a),
                 "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)), "r"(static_cast<uint32_t>(leader))
                 : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar, bool leader) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
                 "r"(static_cast<uint32_t>(leader))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of a warp's lanes. What a load brings is there after tmem_loaded, through which the compiler sees it pass.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
                   "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]),
                   "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// work(g, columns of g, columns of g + 1) for each two groups of 16 columns from `at` on.
template <int GROUPS, typename F>
__device__ __forceinline__ void for_groups(uint32_t at, F work) {
#pragma unroll 1
    for (int g = 0; g < GROUPS; g += 2) {
        uint32_t a[16], b[16];
        tmem_load(at + g * 16, a);
        tmem_load(at + g * 16 + 16, b);
        tmem_loaded(a);
        tmem_loaded(b);
        work(g, a, b);
    }
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                 "r"(r[15]), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// Pairs of 32-bit floats as the paired instructions take them. What is the same for many of them is paired once.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair(float a, float b) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 apart(Pair p) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// A word's four codes as 16-bit floats, exactly. A whole number c becomes 1024 + (c + 128) by placing its byte (sign bit
// flipped) under the exponent byte 0x64, then loses 1152.
template <int KV>
__device__ __forceinline__ uint2 widen(uint32_t w) {
    uint2 o;
    if constexpr (KV == OM_I8) {
        w ^= 0x80808080u;
        const uint32_t u[2] = {__byte_perm(w, 0x64646464u, 0x4140), __byte_perm(w, 0x64646464u, 0x4342)};
        __half2 h[2], c = __half2half2(__ushort_as_half(0x6480));
        memcpy(h, u, 8);
        h[0] = __hsub2(h[0], c);
        h[1] = __hsub2(h[1], c);
        memcpy(&o, h, 8);
    } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(o.x), "=r"(o.y) : "r"(w));
    }
    return o;
}

// What a tile's groups of 16 positions have: scale of the keys, of the values (NaN if it is not finite), the log of its
// magnitude, visible positions.
struct TileScales {
    float4 group[kSharedTile / 16];
    float largest;  // magnitude of a visible group's value scale
    int kind;
};
// What kind of tile it is. kPlain: every position is visible, and larger products are larger scores. kAgain: the same positions' tile comes again, for
// pages of other scales. From kApart on: how many powers of two the value scales are apart. They share a unit up to kSpread; its largest
// weight has to stay so much higher for the weights of the smaller scales to keep their bits.
constexpr int kPlain = 1, kAgain = 2, kApart = 2, kSpread = 8;
// Barriers of what there are two of (tiles by their number's parity, items) belong to one of them: a wait for a phase never
// meets the phase after the next.
struct Bars {
    uint64_t q_full, k_full[2], scored[2], weighed[2], summed[2], drained;
    uint64_t item_full[2], item_free[2];
    SharedItem item[2];  // rows 0: there are no more
    TileScales scales[2];
    int again[4];  // kAgain of the last tiles, for the other roles: tile n + 4's replaces tile n's once the rows are done with tile n + 2
    uint32_t tmem;
    int abort;
};
__device__ __forceinline__ bool aborted(Bars *b) { return *reinterpret_cast<volatile int *>(&b->abort) != 0; }
// Bounded wait of a warp that also gives up once another role has failed. SLEEP: nanoseconds between tests, for the roles that are ahead;
// what a waiting warp issues, the working ones cannot.
template <int SLEEP>
__device__ __forceinline__ bool wait(Bars *b, uint64_t *bar, uint32_t parity, unsigned *status) {
    unsigned long long t0 = 0;
    bool ok = true;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 256; ++i) {
            if (mbar_try_wait(bar, parity)) goto arrived;
            if (SLEEP > 0) __nanosleep(SLEEP);
        }
        ok = !aborted(b);
        const unsigned long long now = global_ns();
        if (t0 == 0) t0 = now;
        if (ok && now - t0 > kWaitLimitNs) {
            atomicOr(status, kDevErrTimeout);
            *reinterpret_cast<volatile int *>(&b->abort) = 1;
            ok = false;
        }
        if (!ok) break;
    }
arrived:
    return __all_sync(0xffffffffu, ok);
}

// The page of a position, -1 behind the end. Nothing here looks at what was loaded, which would wait for it.
__device__ __forceinline__ int load_page(const int32_t *table, int pos, int len, int page_log) {
    int id;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tmov.s32 %0, -1;\n\t@p ld.global.s32 %0, [%1];\n\t}"
                 : "=&r"(id)
                 : "l"(table + (pos >> page_log)), "r"(static_cast<uint32_t>(pos < len)));
    return id;
}
// 16 codes, zeros where there are none.
__device__ __forceinline__ uint4 load_codes(const uint8_t *at, bool there) {
    uint4 x;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                 "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "=&r"(x.x), "=&r"(x.y), "=&r"(x.z), "=&r"(x.w)
                 : "l"(at), "r"(static_cast<uint32_t>(there)));
    return x;
}

// SEVERAL: pages are smaller than a tile, which then can come again. (As a choice at run time 64 conversations in pages of 64 took 163 us instead of 154.)
// FOLD: tiles whose sums stay in tensor memory before they are added to those in global memory, as rounded 32-bit sums (0: all of a part's)
template <int KV, int DIM, int PARTS, int FOLD, bool SEVERAL>
__global__ void __launch_bounds__(kThreads, DIM == 256 ? 1 : 2) kv_shared_kernel(const __grid_constant__ SharedProblem p) {
    using C = Config<DIM, PARTS>;
    constexpr int kPos = C::kPos, kGroups = C::kGroups, kBlocks = DIM / 64;
    extern __shared__ uint8_t raw_smem[];
    __shared__ Bars bars_;
    Bars *const bars = &bars_;
    uint8_t *const smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    const uint32_t q_at = smem_u32(smem), k_at = q_at + C::kQBytes, v_at = k_at + C::kTiles * C::kTile;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    unsigned *const status = p.status;
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, kRowWarps);
        mbar_init(&bars->drained, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->k_full[i], kCopyWarps);
            mbar_init(&bars->scored[i], 2);  // by the products, and by the warp that lays out the scales
            mbar_init(&bars->weighed[i], kRowWarps + kCopyWarps);  // by the weights' rows, and by the copies of the values
            mbar_init(&bars->summed[i], 1);
            mbar_init(&bars->item_full[i], 1);
            mbar_init(&bars->item_free[i], kRowWarps + 2 * kCopyWarps + 2);
        }
        bars->abort = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp == kProductWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem)), "n"(C::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = bars->tmem, sums = tmem + 2 * kPos;
    wait_for_earlier();

    const int page = static_cast<int>(p.c.page), page_log = 31 - __clz(page), heads = static_cast<int>(p.c.heads);
    const unsigned pages = static_cast<unsigned>(p.c.pages);
    auto there = [&](int id) { return static_cast<unsigned>(id) < pages; };
    int n = 0;  // tiles of this block so far
    int items = 0;
    bool ok = true;
    // waits for tile i at a barrier of two
    auto wait_tile = [&](auto sleep, uint64_t (&bar)[2], int i) { return wait<sleep.value>(bars, &bar[i & 1], i / 2 & 1, status); };
    // the block's next part of an item (rows 0: none), and the end of a warp's work on it
    auto take = [&]() -> const SharedItem & {
        ok = wait<32>(bars, &bars->item_full[items & 1], items / 2 & 1, status);
        return bars->item[items & 1];
    };
    constexpr std::integral_constant<int, 0> at_once{};
    constexpr std::integral_constant<int, 40> soon{};
    constexpr std::integral_constant<int, 400> ahead{};
    auto done = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_free[items & 1]);
        ++items;
    };

    // two blocks of 512 threads have 64 registers a thread: 256 for the four warpgroups
    if (warp < kRowWarps) {
        // ------------------------------------------------------------ rows
        if constexpr (DIM != 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        const int row = warp * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
#pragma unroll 1
        for (;;) {
            const SharedItem &it = take();
            if (!ok || it.rows == 0) break;
            // queries: raw to where their 16-bit floats will be (32-bit ones: four elements where the first parts of eight go, four where the
            // second parts go), then each lane scales its row by a power of two, in place
            constexpr int kElements = PARTS == 2 ? 4 : 8, kRaw = DIM / kElements;  // of 16 bytes; 16-byte chunks of a row
            const int bytes = PARTS == 2 ? 4 : 2, live = it.rows - warp * 32;
            auto chunk_at = [&](int r, int c) { return static_cast<uint32_t>(c / 8 * (kSharedRows * 128) + (warp * 32 + r) * 128 + ((c % 8 ^ (r & 7)) * 16)); };
            {
                const int R = it.row0 + row, token = R / p.group;
                const int64_t mine = (it.t0 + token) * p.q.ts + (static_cast<int64_t>(it.h) * p.group + R - token * p.group) * p.q.hs;
#pragma unroll 4
                for (int i = lane; i < 32 * kRaw; i += 32) {
                    const int r = i / kRaw, k = i % kRaw;
                    const uint8_t *const from = static_cast<const uint8_t *>(p.q.p) + (__shfl_sync(0xffffffffu, mine, r) + k * kElements) * bytes;
                    const uint32_t to = q_at + (PARTS == 2 ? k % 2 * C::kQPart + chunk_at(r, k / 2) : chunk_at(r, k));
                    if (p.q_sixteens) {
                        cp_async_16(to, r < live ? from : static_cast<const uint8_t *>(p.q.p), r < live ? 16 : 0);
                    } else {
#pragma unroll 1
                        for (int e = 0; e < kElements; ++e) {
                            if constexpr (PARTS == 2)
                                *reinterpret_cast<uint32_t *>(smem + (to - q_at) + 4 * e) = r < live ? reinterpret_cast<const uint32_t *>(from)[e] : 0;
                            else
                                *reinterpret_cast<uint16_t *>(smem + (to - q_at) + 2 * e) = r < live ? reinterpret_cast<const uint16_t *>(from)[e] : 0;
                        }
                    }
                }
                cp_async_wait_all();
                __syncwarp();
            }
            // eight elements of the lane's row
            auto eight = [&](int c, float (&v)[8]) {
                const uint4 a = *reinterpret_cast<const uint4 *>(smem + chunk_at(lane, c));
                const uint32_t w[4] = {a.x, a.y, a.z, a.w};
                if constexpr (PARTS == 2) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(smem + C::kQPart + chunk_at(lane, c));
                    const uint32_t z[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = __uint_as_float(w[e]);
                        v[4 + e] = __uint_as_float(z[e]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = p.dtype == OM_F16 ? unpack_half(w[e]) : make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
                        v[2 * e] = f.x;
                        v[2 * e + 1] = f.y;
                    }
                }
            };
            unsigned most = 0;
#pragma unroll 4
            for (int c = 0; c < DIM / 8; ++c) {
                float v[8];
                eight(c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
            }
            // the row's largest element to [2^13, 2^14)
            const int e2 = max(static_cast<int>(most >> 23) - 127, -100);
            const float up = power_of_two(13 - e2), factor = __fmul_rn(power_of_two(e2 - 13), __fmul_rn(p.scale, kLog2e));
#pragma unroll 4
            for (int c = 0; c < DIM / 8; ++c) {
                float v[8];
                eight(c, v);
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[2 * e] = __fmul_rn(v[2 * e], up);
                    v[2 * e + 1] = __fmul_rn(v[2 * e + 1], up);
                    x[e] = pack_half(v[2 * e], v[2 * e + 1]);
                }
                *reinterpret_cast<uint4 *>(smem + chunk_at(lane, c)) = make_uint4(x[0], x[1], x[2], x[3]);
                if constexpr (PARTS == 2) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = unpack_half(x[e]);
                        x[e] = pack_half(__fsub_rn(v[2 * e], y.x), __fsub_rn(v[2 * e + 1], y.y));
                    }
                    *reinterpret_cast<uint4 *>(smem + C::kQPart + chunk_at(lane, c)) = make_uint4(x[0], x[1], x[2], x[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full);

            float m = kNone, l = 0.0f, per_unit = 1.0f;
            const int first_tile = n;
            // four columns of the lane's row, of the sums that no longer are in tensor memory
            auto kept = [&](int c) {
                const int rows = static_cast<int>(p.slot_rows), first = warp * 32;
                return reinterpret_cast<float4 *>(p.kept + (static_cast<int64_t>(blockIdx.x) * rows + first) * DIM) + (c / 4 * min(rows - first, 32) + lane);
            };
#pragma unroll 1
            for (int left = it.to - it.from; left > 0; ++n) {
                const uint32_t scores = tmem + lanes + (n & 1) * kPos;
                const float4 *const groups = bars->scales[n & 1].group;
                ok = wait_tile(at_once, bars->scored, n);
                if (!ok) break;
                fence_after();
                const int kind = bars->scales[n & 1].kind;
                const bool plain = (kind & kPlain) != 0;
                left -= !SEVERAL || !(kind & kAgain);
                // the tile's largest score, and the largest log of a score's weight times its value scale; scores that are all NaN leave none
                float top = -INFINITY, heavy = -INFINITY;
                auto note = [&](float x, float log_scale) {
                    top = fmaxf(top, x);
                    heavy = fmaxf(heavy, __fadd_rn(x, log_scale));
                };
                if (plain) {
                    for_groups<kGroups>(scores, [&](int g, const uint32_t (&a)[16], const uint32_t (&b)[16]) {
                        const float4 of_a = groups[g], of_b = groups[g + 1];
                        float hi[2], lo[2];
                        auto at = [](const uint32_t (&s)[16], int i) { return __uint_as_float(s[i]); };
                        hi[0] = max3(at(a, 0), at(a, 1), at(a, 2));
                        lo[0] = max3(at(a, 3), at(a, 4), at(a, 5));
                        hi[1] = max3(at(b, 0), at(b, 1), at(b, 2));
                        lo[1] = max3(at(b, 3), at(b, 4), at(b, 5));
#pragma unroll
                        for (int i = 6; i < 14; i += 4) {
                            hi[0] = max3(hi[0], at(a, i), at(a, i + 1));
                            lo[0] = max3(lo[0], at(a, i + 2), at(a, i + 3));
                            hi[1] = max3(hi[1], at(b, i), at(b, i + 1));
                            lo[1] = max3(lo[1], at(b, i + 2), at(b, i + 3));
                        }
                        note(__fmul_rn(max3(hi[0], lo[0], fmaxf(at(a, 14), at(a, 15))), __fmul_rn(of_a.x, factor)), of_a.z);
                        note(__fmul_rn(max3(hi[1], lo[1], fmaxf(at(b, 14), at(b, 15))), __fmul_rn(of_b.x, factor)), of_b.z);
                    });
                } else {
                    for_groups<kGroups>(scores, [&](int g, const uint32_t (&a)[16], const uint32_t (&b)[16]) {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
                            const float4 of = groups[g + h];
                            const float kf = __fmul_rn(of.x, factor);
                            const int many = __float_as_int(of.w);
                            float hi = -INFINITY, lo = INFINITY;
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float s = __uint_as_float(h == 0 ? a[i] : b[i]);
                                if (i < many) {
                                    hi = fmaxf(hi, s);
                                    lo = fminf(lo, s);
                                }
                            }
                            if (hi >= lo) note(__fmul_rn(kf >= 0.0f ? hi : lo, kf), of.z);
                        }
                    });
                }
                // does the tile fit the row's maximum and unit
                float less = m - kBias;
                const bool live = heavy > -INFINITY;
                const float most_w = __fmul_rn(ex2(heavy - less), per_unit);
                const bool fits = (!live || most_w >= (SEVERAL ? power_of_two((kind >> kApart) - 1) : kLeast)) && most_w <= kMost && ex2(top - less) <= kMostExp;
                const bool fold = FOLD > 0 && n > first_tile && (n - first_tile) % (FOLD > 0 ? FOLD : 1) == 0;  // this tile's product starts new sums
                if (fold || !__all_sync(0xffffffffu, fits)) {
                    float by = 1.0f;  // what the sums are multiplied by
                    int raise = 0;    // the unit goes down by so many powers of two
                    if (!fits && top > kNone) {
                        if (top > m) {
                            by = ex2(m - top);
                            m = top;
                            l = __fmul_rn(l, by);
                        }
                        if (live) {
                            const float to = fmaxf(ex2(heavy - m), __fmul_rn(kLeastOfScale, bars->scales[n & 1].largest));
                            const unsigned unit = min(__float_as_uint(fmaxf(to, kLeastUnit)) & 0x7f800000u, kMostUnit);
                            raise = (static_cast<int>((254u << 23) - unit) - static_cast<int>(__float_as_uint(per_unit))) >> 23;
                        }
                    }
                    if (n > first_tile) {
                        const bool keeps = FOLD > 0 && n - first_tile > FOLD && row < it.rows;
                        // earlier tiles' sums are complete before they are touched
                        ok = wait_tile(at_once, bars->summed, n - 1);
                        if (!ok) break;
                        fence_after();
                        if (__any_sync(0xffffffffu, raise > 0)) {
                            unsigned most = 0;  // magnitudes compare as their bits
#pragma unroll 1
                            for (int c = 0; c < DIM; c += 16) {
                                uint32_t o[16];
                                tmem_load(sums + lanes + c, o);
                                tmem_loaded(o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) most = max(most, o[i] & 0x7fffffffu);
                            }
#pragma unroll 1
                            for (int c = 0; keeps && c < DIM; c += 4) {
                                const float4 o = __ldcg(kept(c));
                                most = max(most, max(max(__float_as_uint(o.x) & 0x7fffffffu, __float_as_uint(o.y) & 0x7fffffffu),
                                                     max(__float_as_uint(o.z) & 0x7fffffffu, __float_as_uint(o.w) & 0x7fffffffu)));
                            }
                            __syncwarp();
                            most = __float_as_uint(__fmul_rn(__uint_as_float(most), by));
                            raise = min(raise, max(227 - static_cast<int>(most >> 23), 0));
                        }
                        const int k = raise / 2;  // up to 2^252 either way: in two steps
                        const float one = __fmul_rn(by, power_of_two(k)), two = power_of_two(raise - k);
                        auto times = [&](float x) { return __fmul_rn(__fmul_rn(x, one), two); };
                        if (by != 1.0f || raise != 0) {
#pragma unroll 1
                            for (int c = 0; keeps && c < DIM; c += 4) {
                                const float4 o = __ldcg(kept(c));
                                __stcg(kept(c), make_float4(times(o.x), times(o.y), times(o.z), times(o.w)));
                            }
                        }
                        __syncwarp();
#pragma unroll 1
                        for (int c = 0; c < DIM; c += 16) {
                            uint32_t o[16];
                            tmem_load(sums + lanes + c, o);
                            tmem_loaded(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(times(__uint_as_float(o[i])));
                            if (!fold) {
                                tmem_store(sums + lanes + c, o);
                            } else if (row < it.rows) {
#pragma unroll
                                for (int i = 0; i < 16; i += 4) {
                                    const float4 x = make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]), __uint_as_float(o[i + 3]));
                                    // nobody else adds to them: their order is the thread's, which does not wait for the sums
                                    if (keeps)
                                        atomicAdd(kept(c + i), x);
                                    else
                                        __stcg(kept(c + i), x);
                                }
                            }
                            __syncwarp();
                        }
                        tmem_stored();
                    }
                    per_unit = __uint_as_float(__float_as_uint(per_unit) + (static_cast<unsigned>(raise) << 23));
                    less = m - kBias;
                }
                // weights: their parts take the scores' place, for 16 positions eight columns of the first and eight of the second
                Pair tile_sum[2] = {pair(0.0f, 0.0f), pair(0.0f, 0.0f)};
                const Pair base = pair(-less, -less), minus = pair(-1.0f, -1.0f);
                auto weigh = [&](auto every) {
                    for_groups<kGroups>(scores, [&](int g, const uint32_t (&a)[16], const uint32_t (&b)[16]) {
                        const float4 of[2] = {groups[g], groups[g + 1]};
                        Pair kf[2], vf[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float k = __fmul_rn(of[h].x, factor), v = of[h].y == of[h].y ? in_units(of[h].y, per_unit) : of[h].y;
                            kf[h] = pair(k, k);
                            vf[h] = pair(v, v);
                        }
                        uint32_t w[2][16];
                        // the groups side by side: two chains of operations for every pair
#pragma unroll
                        for (int i = 0; i < 16; i += 2)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const uint32_t s0 = h == 0 ? a[i] : b[i], s1 = h == 0 ? a[i + 1] : b[i + 1];
                                const float2 x = apart(fma2(pair(__uint_as_float(s0), __uint_as_float(s1)), kf[h], base));
                                float2 e = make_float2(ex2(x.x), ex2(x.y));
                                const int many = every.value ? 16 : __float_as_int(of[h].w);
                                if (!every.value) {
                                    if (i >= many) e.x = 0.0f;
                                    if (i + 1 >= many) e.y = 0.0f;
                                }
                                const Pair both = pair(e.x, e.y);
                                tile_sum[h] = add2(tile_sum[h], both);
                                Pair weights = mul2(both, vf[h]);
                                if (!every.value) {  // a scale that is not finite does not count where nothing is seen
                                    float2 y = apart(weights);
                                    if (i >= many) y.x = 0.0f;
                                    if (i + 1 >= many) y.y = 0.0f;
                                    weights = pair(y.x, y.y);
                                }
                                const float2 y = apart(weights);
                                w[h][i / 2] = pack_half(y.x, y.y);
                                const float2 z = unpack_half(w[h][i / 2]);
                                const float2 rest = apart(fma2(pair(z.x, z.y), minus, weights));  // there is no paired subtraction
                                w[h][8 + i / 2] = pack_half(rest.x, rest.y);
                            }
                        tmem_store(scores + g * 16, w[0]);
                        tmem_store(scores + g * 16 + 16, w[1]);
                    });
                };
                if (plain)
                    weigh(std::true_type{});
                else
                    weigh(std::false_type{});
                const float2 sum_a = apart(tile_sum[0]), sum_b = apart(tile_sum[1]);
                l = __fadd_rn(l, __fadd_rn(__fadd_rn(sum_a.x, sum_a.y), __fadd_rn(sum_b.x, sum_b.y)));
                tmem_stored();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->weighed[n & 1]);
            }
            if (!ok) break;
            // ---- the part's sums as weighted means (no larger than the values), by rows of 64 bytes through the queries' memory
            ok = wait_tile(at_once, bars->summed, n - 1);
            if (!ok) break;
            fence_after();
            const float inv = inverse(l), back = reciprocal(per_unit);
            const bool whole = it.from == 0 && it.to == it.units;
            const int slot = 2 * static_cast<int>(blockIdx.x) + !it.at_start;
            auto place = [&](int r) -> int64_t {
                const int R = it.row0 + r;
                return (it.t0 + R / p.group) * p.q_heads + static_cast<int64_t>(it.h) * p.group + R % p.group;
            };
            if (row < it.rows) {
                float2 *const to = whole ? p.whole_state + place(row) : p.slot_state + static_cast<int64_t>(slot) * p.slot_rows + row;
                *to = make_float2(m == kNone ? -INFINITY : m, l);
            }
            constexpr int kPitch = 20;  // floats of a row of 16, free of bank conflicts
            float *const stage = reinterpret_cast<float *>(smem + warp * 4096);  // where the warp's own queries were
            const bool keeps = FOLD > 0 && n - 1 - first_tile >= FOLD && row < it.rows;
            float4 more[4];
            if (keeps)
#pragma unroll
                for (int i = 0; i < 4; ++i) more[i] = __ldcg(kept(4 * i));
#pragma unroll 1
            for (int c = 0; c < DIM; c += 16) {
                uint32_t o[16];
                tmem_load(sums + lanes + c, o);
                tmem_loaded(o);
                if (keeps) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[4 * i] = __float_as_uint(__fadd_rn(__uint_as_float(o[4 * i]), more[i].x));
                        o[4 * i + 1] = __float_as_uint(__fadd_rn(__uint_as_float(o[4 * i + 1]), more[i].y));
                        o[4 * i + 2] = __float_as_uint(__fadd_rn(__uint_as_float(o[4 * i + 2]), more[i].z));
                        o[4 * i + 3] = __float_as_uint(__fadd_rn(__uint_as_float(o[4 * i + 3]), more[i].w));
                        if (c + 16 < DIM) more[i] = __ldcg(kept(c + 16 + 4 * i));
                    }
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    float4 x;
                    x.x = __fmul_rn(__fmul_rn(__uint_as_float(o[i]), inv), back);
                    x.y = __fmul_rn(__fmul_rn(__uint_as_float(o[i + 1]), inv), back);
                    x.z = __fmul_rn(__fmul_rn(__uint_as_float(o[i + 2]), inv), back);
                    x.w = __fmul_rn(__fmul_rn(__uint_as_float(o[i + 3]), inv), back);
                    *reinterpret_cast<float4 *>(stage + lane * kPitch + i) = x;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = i * 8 + lane / 4, R = warp * 32 + r;
                    if (R >= it.rows) continue;
                    float *const to = whole ? p.whole + place(R) * DIM : p.slots + (static_cast<int64_t>(slot) * p.slot_rows + R) * DIM;
                    *reinterpret_cast<float4 *>(to + c + lane % 4 * 4) = *reinterpret_cast<const float4 *>(stage + r * kPitch + lane % 4 * 4);
                }
            }
            // the tensor memory has been read before the next item's first product writes it, and the staging memory before queries take it
            fence_before();
            done();
        }
    } else if (warp < kRowWarps + 2 * kCopyWarps) {
        // ------------------------------------------------------------ codes
        if constexpr (DIM != 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        constexpr int kPieces = DIM / 16;                            // 16-byte pieces of a row
        constexpr int kRowsAtOnce = kCopyWarps * 32 / kPieces, kPasses = kPos / kRowsAtOnce;
        // four lanes take 64 dimensions of a row, the next four the row below: their stores of 16 bytes, of every other chunk, meet all banks
        const int tid = (threadIdx.x - kRowWarps * 32) % (kCopyWarps * 32), quad = tid / 4, block_of = quad / 2 % kBlocks, first_row = quad / 2 / kBlocks * 2 + quad % 2;
        const int piece = block_of * 4 + tid % 4;
        const uint32_t chunk = tid % 4 * 2;
        const int64_t page_bytes = static_cast<int64_t>(heads) * page * DIM;
        const bool values = warp >= kRowWarps + kCopyWarps;
#pragma unroll 1
        for (;;) {
            const SharedItem &it = take();
            if (!ok || it.rows == 0) break;
            const int len = it.len, to = it.to;
            const int32_t *const table = p.prefix_table + it.group * p.prefix_width;
            auto page_of = [&](int pos0) { return load_page(table, pos0 + lane * 16, lane < kGroups ? len : 0, page_log); };
            const int64_t head_at = static_cast<int64_t>(it.h) * page * DIM + piece * 16;
            auto load = [&](const void *codes, int pos0, int ids, uint4 (&x)[kPasses]) {
                const uint8_t *const base = static_cast<const uint8_t *>(codes) + head_at;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = i * kRowsAtOnce + first_row, pos = pos0 + r, id = __shfl_sync(0xffffffffu, ids, r / 16);
                    // positions that are not there: zeros, which no weight of zero can turn into a NaN
                    x[i] = load_codes(base + id * page_bytes + (pos & (page - 1)) * DIM, there(id) && pos < len);
                }
            };
            auto store = [&](uint8_t *tile, const uint4 (&x)[kPasses]) {
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = i * kRowsAtOnce + first_row;
                    const uint2 a = widen<KV>(x[i].x), b = widen<KV>(x[i].y), c = widen<KV>(x[i].z), d = widen<KV>(x[i].w);
                    uint8_t *const at = tile + block_of * (kPos * 128) + r * 128;
                    *reinterpret_cast<uint4 *>(at + ((chunk ^ (r & 7)) * 16)) = make_uint4(a.x, a.y, b.x, b.y);
                    *reinterpret_cast<uint4 *>(at + (((chunk + 1) ^ (r & 7)) * 16)) = make_uint4(c.x, c.y, d.x, d.y);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            const void *const codes = values ? p.c.v : p.c.k;
            int ids = page_of(it.from * kPos);
            uint4 x[kPasses];
            load(codes, it.from * kPos, ids, x);
            ids = page_of((it.from + 1) * kPos);
#pragma unroll 1
            for (int u = it.from; u < to; ++n) {  // n counts a tile that comes again, u does not
                // the products that read what this takes the place of
                const int last = n - C::kTiles, stage = n % C::kTiles;
                ok = last < 0 || wait_tile(ahead, values ? bars->summed : bars->scored, last);
                if (!ok) break;
                store(smem + C::kQBytes + ((values ? C::kTiles : 0) + stage) * C::kTile, x);
                if (lane == 0 && !(SEVERAL && values)) mbar_arrive(values ? &bars->weighed[n & 1] : &bars->k_full[stage]);
                if (u + 1 < to) load(codes, (u + 1) * kPos, ids, x);
                ids = page_of((u + 2) * kPos);
                if constexpr (SEVERAL) {
                    // Whether the tile comes again is known with its scores. Values are given away after that has been read: what is
                    // read is not replaced before.
                    ok = wait_tile(soon, bars->scored, n);
                    if (!ok) break;
                    const bool again = bars->again[n & 3] != 0;
                    __syncwarp();
                    if (lane == 0 && values) mbar_arrive(&bars->weighed[n & 1]);
                    if (again) {
                        load(codes, u * kPos, page_of(u * kPos), x);
                        ids = page_of((u + 1) * kPos);
                        continue;
                    }
                }
                ++u;
            }
            if (!ok) break;
            done();
        }
    } else {
        // ------------------------------------------------------------ products
        if constexpr (DIM != 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // one lane issues the products; the whole warp walks beside it, so that descriptors are uniform
        const bool leader = lane == 0;
        if (warp == kWalkWarp) {
            SharedItems walk;
            walk.start(p, blockIdx.x);
#pragma unroll 1
            for (bool more = true; ok && more; ++items) {
                if (items >= 2) ok = wait<100>(bars, &bars->item_free[items & 1], (items / 2 - 1) & 1, status);
                SharedItem it{};
                more = walk.next(p, &it);
                if (lane == 0) {
                    bars->item[items & 1] = it;
                    mbar_arrive(&bars->item_full[items & 1]);
                }
                __syncwarp();
            }
        } else if (warp == kScaleWarp) {
#pragma unroll 1
            for (;;) {
                const SharedItem &it = take();
                if (!ok || it.rows == 0) break;
                const int len = it.len, to = it.to;
                const int32_t *const table = p.prefix_table + it.group * p.prefix_width;
                // lane g has group g's page, a tile ahead
                auto page_of = [&](int pos0) { return load_page(table, pos0 + lane * 16, lane < kGroups ? len : 0, page_log); };
                int id = page_of(it.from * kPos);
#pragma unroll 1
                for (int u = it.from; u < to; ++u) {
                    const int id_next = page_of((u + 1) * kPos);
                    const int64_t at = static_cast<int64_t>(id) * heads + it.h;
                    const float ka = there(id) ? p.c.k_scale[at] : 0.0f, va = there(id) ? p.c.v_scale[at] : 0.0f;
                    const int many = there(id) ? min(max(len - (u * kPos + lane * 16), 0), 16) : 0;
                    const bool finite = fabsf(va) <= FLT_MAX;  // an infinite scale counts as NaN, and sets no unit
                    const float magnitude = finite ? fabsf(va) : 0.0f;
                    const bool grows = __fmul_rn(ka, p.scale) >= 0.0f;
                    // scales too far apart are taken one after the other, by their exponents below the largest one; groups without a magnitude with the first
                    const unsigned mine = many > 0 ? __float_as_uint(magnitude) : 0u;
                    unsigned largest = __reduce_max_sync(0xffffffffu, mine);
                    int below = 0;
                    unsigned passes = 1;  // a bit for each
                    int spread = 0;
                    if constexpr (SEVERAL) {
                        if (mine > 0) below = static_cast<int>(largest >> 23) - static_cast<int>(mine >> 23);
                        spread = 1 + __reduce_max_sync(0xffffffffu, below);
                        if (spread > kSpread) {
                            spread = kSpread;
                            below /= kSpread;
                            passes = __reduce_or_sync(0xffffffffu, 1u << below);
                        }
                    }
                    const bool several = passes != 1;
#pragma unroll 1
                    do {
                        int here = many;
                        if constexpr (SEVERAL) {
                            if (several) {
                                const bool takes = below == __ffs(passes) - 1;
                                here = takes ? many : 0;
                                largest = __reduce_max_sync(0xffffffffu, takes ? mine : 0u);
                            }
                            passes &= passes - 1;
                        }
                        const bool plain = __all_sync(0xffffffffu, lane >= kGroups || (here == 16 && grows));
                        ok = n < 2 || wait_tile(ahead, bars->weighed, n - 2);
                        if (!ok) break;
                        TileScales &s = bars->scales[n & 1];
                        if (lane < kGroups) s.group[lane] = make_float4(ka, finite ? va : __int_as_float(0x7FC00000), log2f(magnitude), __int_as_float(here));
                        if (lane == 0) {
                            s.largest = __uint_as_float(largest);
                            s.kind = (plain ? kPlain : 0) | (SEVERAL && passes != 0 ? kAgain : 0) | spread << kApart;
                            if constexpr (SEVERAL) bars->again[n & 3] = passes != 0;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->scored[n & 1]);
                        ++n;
                    } while (SEVERAL && passes != 0);
                    if (!ok) break;
                    id = id_next;
                }
                if (!ok) break;
                done();
            }
        } else if (warp == kProductWarp) {
#pragma unroll 1
            for (;;) {
                const SharedItem &it = take();
                if (!ok || it.rows == 0) break;
                const int from = it.from, to = it.to;
                // the scores of tile i
                auto score = [&](int i) {
                    const int stage = i % C::kTiles;
                    ok = wait<40>(bars, &bars->k_full[stage], i / C::kTiles & 1, status);
                    if (!ok) return;
                    fence_after();
                    const uint32_t to_scores = tmem + (i & 1) * kPos, keys = k_at + stage * C::kTile;
#pragma unroll
                    for (int j = 0; j < PARTS * kBlocks * 4; ++j) {
                        const int part = PARTS - 1 - j / (kBlocks * 4), b = j / 4 % kBlocks, k = j % 4;
                        mma_smem(to_scores, operand(q_at + part * C::kQPart + b * (kSharedRows * 128) + k * 32, 16), operand(keys + b * (kPos * 128) + k * 32, 16),
                                 C::kScores, j > 0, leader);
                    }
                    commit(&bars->scored[i & 1], leader);
                };
                ok = wait<40>(bars, &bars->q_full, items & 1, status);
                if (ok) score(n);
                const int first_tile = n;
#pragma unroll 1
                for (int u = from; ok && u < to; ++n) {
                    bool again = false;  // the same positions' tile
                    if constexpr (SEVERAL) {
                        ok = wait_tile(soon, bars->scored, n);
                        if (!ok) break;
                        again = bars->again[n & 3] != 0;
                        __syncwarp();
                    }
                    u += !again;
                    // The next tile's scores, beside the rows' work on this one. They take the place of the weights of the tile before, which its
                    // product reads until it is complete: products of one thread keep their order only where accumulator and shape are
                    // the same, and these differ in both. (Scores of an item's first tile follow its queries, which the rows bring after
                    // all products of the item before.)
                    if (u < to) {
                        ok = n == 0 || wait_tile(soon, bars->summed, n - 1);
                        if (!ok) break;
                        score(n + 1);
                    }
                    const int stage = n % C::kTiles;
                    ok = ok && wait_tile(soon, bars->weighed, n);
                    if (!ok) break;
                    fence_after();
                    const uint32_t values = v_at + stage * C::kTile, weights = tmem + (n & 1) * kPos;
#pragma unroll
                    for (int k = 0; k < kPos / 16; ++k) {  // small parts first
                        mma_tmem(sums, weights + k * 16 + 8, operand(values + k * 2048, kPos * 128), C::kSums, k > 0 || (FOLD > 0 ? (n - first_tile) % (FOLD > 0 ? FOLD : 1) != 0 : n > first_tile), leader);
                        mma_tmem(sums, weights + k * 16, operand(values + k * 2048, kPos * 128), C::kSums, true, leader);
                    }
                    commit(&bars->summed[n & 1], leader);
                }
                if (!ok) break;
                done();
            }
        }
        if (warp == kProductWarp) {
            // no product may still read shared memory or write tensor memory when the block frees them
            commit(&bars->drained, leader);
            (void)mbar_wait(&bars->drained, 0);
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kProductWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kColumns) : "memory");
}

template <int KV, int DIM, int PARTS, int FOLD, bool SEVERAL>
cudaError_t launch(const SharedProblem &p, cudaStream_t s) {
    constexpr int kSmem = Config<DIM, PARTS>::kSmem;
    static PerDevice ready;
    std::atomic<int> *const kept = ready.here();
    if (!kept || kept->load(std::memory_order_relaxed) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kv_shared_kernel<KV, DIM, PARTS, FOLD, SEVERAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (kept) kept->store(1, std::memory_order_relaxed);
    }
    return launch_behind(kv_shared_kernel<KV, DIM, PARTS, FOLD, SEVERAL>, dim3(static_cast<unsigned>(p.blocks)), dim3(kThreads), kSmem, s, p);
}

// The tensor cores cut their sums off. 16-bit calls leave a part's sums to them up to 256 tiles (values of one sign, weights alike: 3e-5 off);
// with the code for longer ones, 64 tiles at a time, 64 sequences behind 32768 tokens take 166 us instead of 154. 32-bit calls: see above.
template <int KV, bool SEVERAL, int DIM>
cudaError_t by_type(const SharedProblem &p, cudaStream_t s) {
    constexpr int64_t kLong = 256;
    if (p.dtype == OM_F32) return launch<KV, DIM, 2, kSharedFold, SEVERAL>(p, s);
    return p.most_tiles > kLong ? launch<KV, DIM, 1, 64, SEVERAL>(p, s) : launch<KV, DIM, 1, 0, SEVERAL>(p, s);
}

template <int KV, bool SEVERAL>
cudaError_t run_kv_shared(const SharedProblem &p, cudaStream_t s) {
    if (p.c.dim == 64) return by_type<KV, SEVERAL, 64>(p, s);
    return p.c.dim == 128 ? by_type<KV, SEVERAL, 128>(p, s) : by_type<KV, SEVERAL, 256>(p, s);
}

}  // namespace
}  // namespace om
