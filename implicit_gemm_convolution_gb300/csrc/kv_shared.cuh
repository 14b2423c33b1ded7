// kv_shared.cuh -- attention of many sequences to a prefix that they share, read once for all of them; one
// translation unit for each type of codes (kv_shared_*.cu). The sequences' own tokens are kv_attention.cuh's, as a part of
// the same softmax; kv_shared_join.cu puts the parts together.
//
// Mathematics. As in kv_attention.cuh: keys c_t a, values e_t s, x_t = (q . c_t) a scale log2(e),
// out = sum_t 2^(x_t - m) s e_t / sum_t 2^(x_t - m). The rows are the tokens of all sequences of a group times the
// query heads of a key head, so the products are as large as a library's and run on tcgen05: S = Q C^T, O += P E
// for 128 rows and a tile of 64 or 128 positions, sums in tensor memory. Codes are exact in 16-bit floats, queries are scaled
// by a power of two for each row (32-bit ones in two parts of 11 bits), weights 2^(x - m) s / u go in two parts of 11 bits
// with a power-of-two unit u for each row, set anew when a tile's largest weight leaves [2^-1, 2^15]: a weight is off by no more
// than 2^-22 of itself or 2^-24 of its tile's largest.
//
// Block (two an SM for heads of up to 128: one's products run beside the other's exponentials):
//   warps 0-3  a row of scores a thread: the tile's maxima from tensor memory, then weights, whose parts replace the scores as the
//              second product's operand; rows of sums are multiplied only when a unit or maximum changes; queries in, sums out.
//   warps 4-7  codes from the pages (values on their way beside a tile's scores, the next keys beside its weights) to 16-bit floats in shared memory, rows of 128 bytes with
//              the tensor cores' exclusive-or; keys and values have the same layout (as k-major and n-major operands).
//   warp 8     tensor memory, and one thread that issues the products.
// Every mbarrier wait is bounded; on a timeout the block records the error, stops and frees its tensor memory.
//
// Split. The tiles of all items (group, key head, 128 rows) in equal shares of the blocks that fit at once, as lengths on the
// device give them. A block's part of a cut item goes to one of its two slots, a whole item to its rows' places;
// the join finds them by the same arithmetic. Nobody waits for another block.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "decode_device.cuh"
#include "kv_shared_items.cuh"
#include "om_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kRowWarps = 4, kCopyWarps = 4;
constexpr int kThreads = 384;  // three warpgroups: registers are handed out by them
constexpr int kProductWarp = kRowWarps + kCopyWarps;
constexpr float kLog2e = 1.4426950408889634f;
// as in kv_attention.cuh
constexpr float kBias = 8.0f, kMost = 32768.0f, kLeast = 0.5f, kMostExp = 1099511627776.0f;
constexpr float kNone = -FLT_MAX;
constexpr float kLeastUnit = FLT_MIN, kLeastOfScale = 7.8886090522101181e-31f;
constexpr unsigned kMostUnit = 253u << 23;
__device__ __forceinline__ float in_units(float value, float per_unit) { return fminf(fmaxf(__fmul_rn(value, per_unit), -FLT_MAX), FLT_MAX); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }
__device__ __forceinline__ float reciprocal(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Instruction descriptor of tcgen05.mma kind::f16: D fp32 (bit 4), A and B fp16 (0), B n-major where
// asked (bit 16), N >> 3 in bits 17-22, M >> 4 in bits 24-28.
constexpr uint32_t descriptor_of(int n, bool b_n_major) {
    return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kSharedRows >> 4) << 24);
}

// PARTS: of a query. Positions of a tile: what leaves two blocks of an SM their shared and tensor memory (heads of 256: one block).
template <int DIM, int PARTS>
struct Config {
    static constexpr int kPos = shared_tile(DIM, PARTS);
    static constexpr int kQPart = kSharedRows * DIM * 2;
    static constexpr int kQBytes = PARTS * kQPart;
    static constexpr int kTile = kPos * DIM * 2;
    static constexpr int kSmem = 1024 + kQBytes + 2 * kTile;
    static constexpr int kColumns = kPos + DIM <= 256 ? 256 : 512;  // of tensor memory: scores, then sums
    static constexpr int kGroups = kPos / 16;                       // 16 positions have one page
    static constexpr uint32_t kScores = descriptor_of(kPos, false), kSums = descriptor_of(DIM, true);
};

// Shared-memory descriptor, 128-byte swizzle (layout 2), version 1: groups of 8 rows 1024 bytes apart (stride byte
// offset); n-major operands: 64 columns, then `block` bytes on to the next 64 (leading byte offset).
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t block) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(block >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b),
                 "r"(desc), "r"(static_cast<uint32_t>(add))
                 : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b),
                 "r"(desc), "r"(static_cast<uint32_t>(add))
                 : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 (16) columns of a warp's lanes; a load has arrived when it returns.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,"
        "%28,%29,%30,%31}, [%32];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
          "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
                   "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
        "%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
        "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
        : "memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
                 "r"(r[15]), "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

struct Bars {
    uint64_t q_full, k_full, v_full, scored, weighed, summed, drained;
    uint32_t tmem;
    int abort;
};
__device__ __forceinline__ bool aborted(Bars *b) { return *reinterpret_cast<volatile int *>(&b->abort) != 0; }
// Bounded wait that also gives up once another role has failed.
__device__ __forceinline__ bool wait(Bars *b, uint64_t *bar, uint32_t parity, unsigned *status) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (aborted(b)) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, kDevErrTimeout);
            *reinterpret_cast<volatile int *>(&b->abort) = 1;
            return false;
        }
    }
    return true;
}

// The same for all lanes of a warp.
__device__ __forceinline__ bool wait_warp(Bars *b, uint64_t *bar, uint32_t parity, unsigned *status) {
    return __all_sync(0xffffffffu, wait(b, bar, parity, status));
}

// Four elements of a row of queries.
template <int PARTS>
__device__ __forceinline__ void load_query(const SharedProblem &p, int64_t at, float *v) {
    if constexpr (PARTS == 2)
        p.q_fours ? load4<float, true>(static_cast<const float *>(p.q.p) + at, v) : load4<float, false>(static_cast<const float *>(p.q.p) + at, v);
    else if (p.dtype == OM_F16)
        p.q_fours ? load4<__half, true>(static_cast<const __half *>(p.q.p) + at, v) : load4<__half, false>(static_cast<const __half *>(p.q.p) + at, v);
    else
        p.q_fours ? load4<__nv_bfloat16, true>(static_cast<const __nv_bfloat16 *>(p.q.p) + at, v)
                  : load4<__nv_bfloat16, false>(static_cast<const __nv_bfloat16 *>(p.q.p) + at, v);
}

template <int KV, int DIM, int PARTS>
__global__ void __launch_bounds__(kThreads, DIM == 256 ? 1 : 2) kv_shared_kernel(const __grid_constant__ SharedProblem p) {
    using C = Config<DIM, PARTS>;
    constexpr int kPos = C::kPos, kGroups = C::kGroups, kBlocks = DIM / 64;
    extern __shared__ uint8_t raw_smem[];
    __shared__ Bars bars_;
    Bars *const bars = &bars_;
    uint8_t *const smem = raw_smem + ((1024u - (smem_u32(raw_smem) & 1023u)) & 1023u);
    const uint32_t q_at = smem_u32(smem), k_at = q_at + C::kQBytes, v_at = k_at + C::kTile;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    unsigned *const status = p.status;
    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, kRowWarps);
        mbar_init(&bars->k_full, kCopyWarps);
        mbar_init(&bars->v_full, kCopyWarps);
        mbar_init(&bars->scored, 1);
        mbar_init(&bars->weighed, kRowWarps);
        mbar_init(&bars->summed, 1);
        mbar_init(&bars->drained, 1);
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
    const uint32_t tmem = bars->tmem, sums = tmem + kPos;
    wait_for_earlier();

    __shared__ SharedItems walks[kProductWarp + 1];
    SharedItems &items = walks[min(warp, kProductWarp)];
    if (warp <= kProductWarp) items.start(p, blockIdx.x);
    const int page = static_cast<int>(p.c.page), page_log = 31 - __clz(page), heads = static_cast<int>(p.c.heads);
    int n = 0;  // tiles of this block so far, the phase of its barriers
    bool ok = true;

    // two blocks of 384 threads have 80 registers a thread: 240 for the three warpgroups
    if (warp < kRowWarps) {
        // ------------------------------------------------------------ rows
        if constexpr (DIM != 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        const int row = warp * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
#pragma unroll 1
        for (; ok && items.next(p);) {
            const SharedItem &it = items.item;
            // queries: 16 lanes a row, two rows at a time, scaled by a power of two
            constexpr int kEach = DIM / 16;
            float factor = 0.0f;
            const int half = lane / 16, q_d = lane % 16 * kEach;
#pragma unroll 2
            for (int i = 0; i < 16; ++i) {
                const int r = warp * 32 + 2 * i + half, R = it.row0 + r;
                float v[kEach];
                if (r < it.rows) {
                    const int64_t at = (it.t0 + R / p.group) * p.q.ts + (static_cast<int64_t>(it.h) * p.group + R % p.group) * p.q.hs + q_d;
#pragma unroll
                    for (int e = 0; e < kEach; e += 4) load_query<PARTS>(p, at + e, v + e);
                } else {
#pragma unroll
                    for (int e = 0; e < kEach; ++e) v[e] = 0.0f;
                }
                unsigned top = 0;
#pragma unroll
                for (int e = 0; e < kEach; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, x));
                // the row's largest element to [2^13, 2^14)
                int e2 = static_cast<int>(top >> 23) - 127;
                e2 = e2 < -100 ? -100 : e2;
                const float up = power_of_two(13 - e2);
                const float f = __shfl_sync(0xffffffffu, __fmul_rn(power_of_two(e2 - 13), __fmul_rn(p.scale, kLog2e)), (lane & 1) * 16);
                if (lane / 2 == i) factor = f;
#pragma unroll
                for (int e = 0; e < kEach; ++e) v[e] = __fmul_rn(v[e], up);
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int e = 0; e < kEach; e += 4) {
                        const int d = q_d + e;
                        const uint2 w = make_uint2(pack_half(v[e], v[e + 1]), pack_half(v[e + 2], v[e + 3]));
                        uint8_t *const to = smem + part * C::kQPart + d / 64 * (kSharedRows * 128) + r * 128 + ((d % 64 / 8 ^ (r & 7)) * 16) + d % 8 * 2;
                        *reinterpret_cast<uint2 *>(to) = w;
                        if (part + 1 < PARTS) {
                            const float2 y = unpack_half(w.x), z = unpack_half(w.y);
                            v[e] -= y.x;
                            v[e + 1] -= y.y;
                            v[e + 2] -= z.x;
                            v[e + 3] -= z.y;
                        }
                    }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full);

            float m = kNone, l = 0.0f, per_unit = 1.0f;
            // pages of the tile's groups of 16 positions: lane g has group g's, a tile ahead
            auto page_of = [&](int pos0) -> int {
                const int pos = pos0 + lane * 16;
                const int id = lane < kGroups && pos < it.len ? p.prefix_table[it.group * p.prefix_width + (pos >> page_log)] : -1;
                return id < p.c.pages ? id : -1;
            };
            auto scales_of = [&](int id, float *ka, float *va) {
                const int64_t at = static_cast<int64_t>(id) * heads + it.h;
                *ka = id < 0 ? 0.0f : p.c.k_scale[at];
                *va = id < 0 ? 0.0f : p.c.v_scale[at];
            };
            int id = page_of(it.from * kPos), id_next = page_of((it.from + 1) * kPos);
            float ka, va, ka_next, va_next;
            scales_of(id, &ka, &va);
#pragma unroll 1
            for (int u = it.from; ok && u < it.to; ++u, ++n) {
                scales_of(id_next, &ka_next, &va_next);
                const int id_after = page_of((u + 2) * kPos), pos0 = u * kPos;
                // positions that are visible in this lane's group
                const int mine = id < 0 ? 0 : min(max(it.len - (pos0 + lane * 16), 0), 16);
                const bool all = __all_sync(0xffffffffu, lane >= kGroups || mine == 16);
                ok = wait_warp(bars, &bars->scored, n & 1, status);
                if (!ok) break;
                fence_after();
                float xg[kGroups];
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < kPos / 32; ++c) {
                    uint32_t s[32];
                    tmem_load(tmem + lanes + c * 32, s);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * c + h;
                        float hi = -INFINITY, lo = INFINITY;
                        if (all) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                hi = fmaxf(hi, __uint_as_float(s[16 * h + i]));
                                lo = fminf(lo, __uint_as_float(s[16 * h + i]));
                            }
                        } else {
                            const int many = __shfl_sync(0xffffffffu, mine, g);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i < many) {
                                    hi = fmaxf(hi, __uint_as_float(s[16 * h + i]));
                                    lo = fminf(lo, __uint_as_float(s[16 * h + i]));
                                }
                        }
                        const float kf = __fmul_rn(__shfl_sync(0xffffffffu, ka, g), factor);
                        // nothing visible, or all of it NaN: -infinity either way
                        xg[g] = hi == -INFINITY && lo == INFINITY ? -INFINITY : __fmul_rn(kf >= 0.0f ? hi : lo, kf);
                        top = fmaxf(top, xg[g]);
                    }
                }
                // does the tile fit the row's maximum and unit
                const float odd_va = fabsf(va) <= FLT_MAX ? fabsf(va) : 0.0f;  // an infinite scale counts as NaN, and sets no unit
                float most_w = 0.0f;
                bool live = false;
                float less = m - kBias;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const float s = __shfl_sync(0xffffffffu, odd_va, g);
                    live |= s > 0.0f && xg[g] > -INFINITY;
                    most_w = fmaxf(most_w, __fmul_rn(__fmul_rn(ex2(xg[g] - less), s), per_unit));
                }
                const bool fits = (!live || most_w >= kLeast) && most_w <= kMost && ex2(top - less) <= kMostExp;
                if (!__all_sync(0xffffffffu, fits)) {
                    float by = 1.0f;  // what the sums are multiplied by
                    int raise = 0;    // the unit goes down by so many powers of two
                    if (!fits && top > kNone) {
                        if (top > m) {
                            by = ex2(m - top);
                            m = top;
                            l = __fmul_rn(l, by);
                        }
                    }
                    float to = 0.0f;
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const float s = __shfl_sync(0xffffffffu, odd_va, g);
                        if (s > 0.0f && xg[g] > -INFINITY) to = fmaxf(to, __fmul_rn(fmaxf(ex2(xg[g] - m), kLeastOfScale), s));
                    }
                    if (!fits && live && top > kNone) {
                        const unsigned unit = min(__float_as_uint(fmaxf(to, kLeastUnit)) & 0x7f800000u, kMostUnit);
                        raise = (static_cast<int>((254u << 23) - unit) - static_cast<int>(__float_as_uint(per_unit))) >> 23;
                    }
                    if (u > it.from) {
                        // earlier tiles' sums are complete before they are touched
                        ok = wait_warp(bars, &bars->summed, (n - 1) & 1, status);
                        if (!ok) break;
                        fence_after();
                        if (__any_sync(0xffffffffu, raise > 0)) {
                            unsigned most = 0;  // magnitudes compare as their bits
#pragma unroll 1
                            for (int c = 0; c < DIM; c += 16) {
                                uint32_t o[16];
                                tmem_load(sums + lanes + c, o);
#pragma unroll
                                for (int i = 0; i < 16; ++i) most = max(most, o[i] & 0x7fffffffu);
                            }
                            most = __float_as_uint(__fmul_rn(__uint_as_float(most), by));
                            raise = min(raise, max(227 - static_cast<int>(most >> 23), 0));
                        }
                        const int k = raise / 2;  // up to 2^252 either way: in two steps
                        const float one = __fmul_rn(by, power_of_two(k)), two = power_of_two(raise - k);
#pragma unroll 1
                        for (int c = 0; c < DIM; c += 16) {
                            uint32_t o[16];
                            tmem_load(sums + lanes + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(o[i]), one), two));
                            tmem_store(sums + lanes + c, o);
                        }
                        tmem_stored();
                    }
                    per_unit = __uint_as_float(__float_as_uint(per_unit) + (static_cast<unsigned>(raise) << 23));
                    less = m - kBias;
                }
                // weights: their parts take the scores' place, 16 columns of the first and 16 of the second for 32 positions
                float tile_sum = 0.0f;
#pragma unroll
                for (int c = 0; c < kPos / 32; ++c) {
                    uint32_t s[32], w[32];
                    tmem_load(tmem + lanes + c * 32, s);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int g = 2 * c + h;
                        const float kf = __fmul_rn(__shfl_sync(0xffffffffu, ka, g), factor), value = __shfl_sync(0xffffffffu, va, g);
                        const float vf = fabsf(value) <= FLT_MAX ? in_units(value, per_unit) : __int_as_float(0x7FC00000);
                        const int many = all ? 16 : __shfl_sync(0xffffffffu, mine, g);
                        float e[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            e[i] = ex2(__fmaf_rn(__uint_as_float(s[16 * h + i]), kf, -less));
                            if (!all && i >= many) e[i] = 0.0f;
                        }
                        float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            part = add2_rn(part, make_float2(e[i], e[i + 1]));
                            float a = __fmul_rn(e[i], vf), b = __fmul_rn(e[i + 1], vf);
                            if (!all) {  // a scale that is not finite does not count where nothing is seen
                                if (i >= many) a = 0.0f;
                                if (i + 1 >= many) b = 0.0f;
                            }
                            const uint32_t x = pack_half(a, b);
                            const float2 y = unpack_half(x);
                            w[8 * h + i / 2] = x;
                            w[16 + 8 * h + i / 2] = pack_half(__fsub_rn(a, y.x), __fsub_rn(b, y.y));
                        }
                        tile_sum = __fadd_rn(tile_sum, __fadd_rn(part.x, part.y));
                    }
                    tmem_store(tmem + lanes + c * 32, w);
                }
                l = __fadd_rn(l, tile_sum);
                tmem_stored();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->weighed);
                id = id_next;
                id_next = id_after;
                ka = ka_next;
                va = va_next;
            }
            if (!ok) break;
            // ---- the part's sums as weighted means (no larger than the values), by rows of 64 bytes through the queries' memory
            ok = wait_warp(bars, &bars->summed, (n - 1) & 1, status);
            if (!ok) break;
            fence_after();
            const float inv = shared_inverse(l), back = reciprocal(per_unit);
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
#pragma unroll 1
            for (int c = 0; c < DIM; c += 16) {
                uint32_t o[16];
                tmem_load(sums + lanes + c, o);
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
            __syncwarp();
        }
    } else if (warp < kRowWarps + kCopyWarps) {
        // ------------------------------------------------------------ codes
        if constexpr (DIM != 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        constexpr int kPieces = DIM / 16;                            // 16-byte pieces of a row
        constexpr int kRowsAtOnce = kCopyWarps * 32 / kPieces, kPasses = kPos / kRowsAtOnce;
        const int tid = threadIdx.x - kRowWarps * 32, piece = tid % kPieces, first_row = tid / kPieces;
        // a piece's 32 bytes of floats: two of a row's 16-byte chunks; pieces of every other 64 dimensions store them in the other
        // order, so that eight lanes meet all banks
        const int block_of = piece / 4, swap = block_of & 1;
        const uint32_t chunk = piece % 4 * 2;
        const int64_t page_bytes = static_cast<int64_t>(heads) * page * DIM;
#pragma unroll 1
        for (; ok && items.next(p);) {
            const SharedItem &it = items.item;
            auto page_of = [&](int pos0) -> int {
                const int pos = pos0 + lane * 16;
                const int id = lane < kGroups && pos < it.len ? p.prefix_table[it.group * p.prefix_width + (pos >> page_log)] : -1;
                return id < p.c.pages ? id : -1;
            };
            auto load = [&](const void *codes, int pos0, int ids, uint4 (&x)[kPasses]) {
                const uint8_t *const base = static_cast<const uint8_t *>(codes) + static_cast<int64_t>(it.h) * page * DIM + piece * 16;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = i * kRowsAtOnce + first_row, pos = pos0 + r, id = __shfl_sync(0xffffffffu, ids, r / 16);
                    // positions that are not there: zeros, which no weight of zero can turn into a NaN
                    x[i] = id >= 0 && pos < it.len ? __ldg(reinterpret_cast<const uint4 *>(base + id * page_bytes + (pos & (page - 1)) * DIM)) : make_uint4(0, 0, 0, 0);
                }
            };
            auto store = [&](uint8_t *tile, const uint4 (&x)[kPasses]) {
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int r = i * kRowsAtOnce + first_row;
                    const uint2 a = widen<KV>(x[i].x), b = widen<KV>(x[i].y), c = widen<KV>(x[i].z), d = widen<KV>(x[i].w);
                    const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(c.x, c.y, d.x, d.y);
                    uint8_t *const at = tile + block_of * (kPos * 128) + r * 128;
                    *reinterpret_cast<uint4 *>(at + (((chunk + swap) ^ (r & 7)) * 16)) = swap ? hi : lo;
                    *reinterpret_cast<uint4 *>(at + (((chunk + 1 - swap) ^ (r & 7)) * 16)) = swap ? lo : hi;
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            int ids = page_of(it.from * kPos);
            uint4 x[kPasses];
            load(p.c.k, it.from * kPos, ids, x);
#pragma unroll 1
            for (int u = it.from; u < it.to; ++u, ++n) {
                const int ids_next = page_of((u + 1) * kPos);
                ok = n == 0 || wait_warp(bars, &bars->scored, (n - 1) & 1, status);
                if (!ok) break;
                store(smem + C::kQBytes, x);
                if (lane == 0) mbar_arrive(&bars->k_full);
                load(p.c.v, u * kPos, ids, x);
                ok = n == 0 || wait_warp(bars, &bars->summed, (n - 1) & 1, status);
                if (!ok) break;
                store(smem + C::kQBytes + C::kTile, x);
                if (lane == 0) mbar_arrive(&bars->v_full);
                ids = ids_next;
                if (u + 1 < it.to) load(p.c.k, (u + 1) * kPos, ids, x);
            }
        }
    } else {
        // ------------------------------------------------------------ products
        if constexpr (DIM != 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        int segment = 0;
#pragma unroll 1
        for (; warp == kProductWarp && ok && items.next(p); ++segment) {
            const SharedItem &it = items.item;
            if (lane == 0) {
#pragma unroll 1
                for (int u = it.from; ok && u < it.to; ++u, ++n) {
                    ok = (u > it.from || wait(bars, &bars->q_full, segment & 1, status)) && wait(bars, &bars->k_full, n & 1, status) &&
                         (n == 0 || wait(bars, &bars->summed, (n - 1) & 1, status));  // the weights, in the scores' place, have been read
                    if (!ok) break;
                    fence_after();
                    bool add = false;
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                mma_smem(tmem, operand(q_at + part * C::kQPart + b * (kSharedRows * 128) + k * 32, 16), operand(k_at + b * (kPos * 128) + k * 32, 16), C::kScores, add);
                                add = true;
                            }
                    commit(&bars->scored);
                    ok = wait(bars, &bars->v_full, n & 1, status) && wait(bars, &bars->weighed, n & 1, status);
                    if (!ok) break;
                    fence_after();
                    add = u > it.from;
#pragma unroll
                    for (int k = 0; k < kPos / 16; ++k)
#pragma unroll
                        for (int part = 1; part >= 0; --part) {  // small parts first
                            mma_tmem(sums, tmem + k / 2 * 32 + part * 16 + k % 2 * 8, operand(v_at + k * 2048, kPos * 128), C::kSums, add);
                            add = true;
                        }
                    commit(&bars->summed);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (warp == kProductWarp && lane == 0) {
            // no product may still read shared memory or write tensor memory when the block frees them
            commit(&bars->drained);
            (void)mbar_wait(&bars->drained, 0);
        }
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kProductWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kColumns) : "memory");
}

template <int KV, int DIM, int PARTS>
cudaError_t launch(const SharedProblem &p, cudaStream_t s) {
    constexpr int kSmem = Config<DIM, PARTS>::kSmem;
    static PerDevice ready;
    std::atomic<int> *const kept = ready.here();
    if (!kept || kept->load(std::memory_order_relaxed) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(kv_shared_kernel<KV, DIM, PARTS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (kept) kept->store(1, std::memory_order_relaxed);
    }
    return launch_behind(kv_shared_kernel<KV, DIM, PARTS>, dim3(static_cast<unsigned>(p.blocks)), dim3(kThreads), kSmem, s, p);
}

template <int KV>
cudaError_t run_kv_shared(const SharedProblem &p, cudaStream_t s) {
    const bool two = p.dtype == OM_F32;
    if (p.c.dim == 64) return two ? launch<KV, 64, 2>(p, s) : launch<KV, 64, 1>(p, s);
    if (p.c.dim == 128) return two ? launch<KV, 128, 2>(p, s) : launch<KV, 128, 1>(p, s);
    return two ? launch<KV, 256, 2>(p, s) : launch<KV, 256, 1>(p, s);
}

}  // namespace
}  // namespace om
