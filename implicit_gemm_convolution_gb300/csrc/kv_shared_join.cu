// kv_shared_join.cu -- joins what attention to a shared prefix and to a sequence's own tokens left of each row: the
// weighted means, by weights sum 2^(maximum - best).
//
// One warp a row (token and query head), or some of a token's where there are many: it finds the blocks that had parts of its row from the lengths, as they cut
// them (kv_shared_items.cuh), takes the maximum over all parts, then one pass over their values. Order and arithmetic follow from
// the lengths alone.
//
// Bound: the latency of its lookups for few rows, L2 for many (4 dim bytes a row and part, written a moment before).
// Measured (GB300): 4096 rows of 128 in about three parts each 9 us behind the prefix's kernel; two rows a warp side by side ran slower.

#include <type_traits>

#include "attention_range.cuh"
#include "decode_device.cuh"
#include "kv_shared_items.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kThreads = 128;

template <int N>
__device__ __forceinline__ void load_values(const float *from, float (&v)[N]) {
    if constexpr (N == 2) {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(from));
        v[0] = x.x;
        v[1] = x.y;
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(from + e));
            v[e] = x.x;
            v[e + 1] = x.y;
            v[e + 2] = x.z;
            v[e + 3] = x.w;
        }
    }
}

// Where the parts of a token's rows are.
struct Parts {
    int t0, row_blocks, units, before;  // of its group; units 0: none
};

template <typename T, int DIM, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) kv_shared_join_kernel(const __grid_constant__ SharedProblem p, int rows_each) {
    constexpr int kEach = DIM / 32;
    const int lane = threadIdx.x & 31, heads = static_cast<int>(p.q_heads), rows = static_cast<int>(p.tokens) * heads;
    // a warp's rows are one token's, or a token's all
    const int begin = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * rows_each;
    wait_for_earlier();
    if (begin >= rows) return;
    const int t = begin / heads;
    // what does not depend on anything is asked for first
    float2 own = __ldcg(p.own_state + begin);
    float o[kEach];
    load_values(p.own + static_cast<int64_t>(begin) * DIM + lane * kEach, o);
    const int t_first = p.cu[0], t_last = p.cu[p.seqs];
    const SharedGroup mine_first = shared_group(p, lane);
    const int total = shared_units(p, mine_first), per = shared_per_block(p, total);
    if (t < t_first || t >= t_last) return;  // no sequence's
    // the token's group, and the units before it
    Parts parts{0, 0, 0, 0};
    if (total > 0) {
        int before = 0;
#pragma unroll 1
        for (int64_t base = 0; base < p.groups; base += 32) {
            const SharedGroup g = base == 0 ? mine_first : shared_group(p, base + lane);
            const int n = static_cast<int>(g.n);
            int up = n;
            if (p.groups > 1) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += x;
                }
            }
            const unsigned here = __ballot_sync(0xffffffffu, n > 0 && t >= g.t0 && (t - g.t0) * p.group < g.rows);
            if (here != 0) {
                const int from = __ffs(here) - 1;
                parts = Parts{__shfl_sync(0xffffffffu, g.t0, from), __shfl_sync(0xffffffffu, g.row_blocks, from), __shfl_sync(0xffffffffu, g.units, from),
                              before + __shfl_sync(0xffffffffu, up - n, from)};
                break;
            }
            before += __shfl_sync(0xffffffffu, up, 31);
        }
    }
#pragma unroll 1
    for (int row = begin; row < min(begin + rows_each, rows); ++row) {
        const int head = row - t * heads;
        int count = 0, first = 0, at = 0;
        if (parts.units > 0) {
            const int h = head / p.group, r = (t - parts.t0) * p.group + head - h * p.group;
            const int from = parts.before + (h * parts.row_blocks + r / kSharedRows) * parts.units, c = from / per;
            count = (from + parts.units - 1) / per - c + 1;
            first = 2 * c + (from > c * per);  // a part that does not start its block's share is in the second slot
            at = r % kSharedRows;
        }
        // part j of the prefix; an item that one block had is at its row's place
        const bool whole = count == 1;
        const int slot_rows = static_cast<int>(p.slot_rows);
        auto place = [&](int j) { return whole ? row : (j == 0 ? first : (first | 1) - 1 + 2 * j) * slot_rows + at; };
        const float2 *const states = whole ? p.whole_state : p.slot_state;
        const float *const values = whole ? p.whole : p.slots;
        if (row > begin) {
            own = __ldcg(p.own_state + row);
            load_values(p.own + static_cast<int64_t>(row) * DIM + lane * kEach, o);
        }
        float best = own.x;
        float2 mine = make_float2(-INFINITY, 0.0f);
#pragma unroll 1
        for (int j = lane; j < count; j += 32) {
            const float2 s = __ldcg(states + place(j));
            if (j < 32) mine = s;
            best = fmaxf(best, s.x);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, x));
        const float w_own = joined(own.y, own.x, best);
        float mass = w_own;
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] = __fmul_rn(o[e], w_own);
#pragma unroll 1
        for (int base = 0; base < count; base += 32) {
            if (base > 0) mine = base + lane < count ? __ldcg(states + place(base + lane)) : make_float2(-INFINITY, 0.0f);
            const float w = joined(mine.y, mine.x, best);
            const int many = min(count - base, 32), here = place(base + lane);
            constexpr int kAhead = 8;  // parts in flight
#pragma unroll 1
            for (int j0 = 0; j0 < many; j0 += kAhead) {
                float y[kAhead][kEach];
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (j0 + j < many) load_values(values + static_cast<int64_t>(__shfl_sync(0xffffffffu, here, j0 + j)) * DIM + lane * kEach, y[j]);
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const float wj = __shfl_sync(0xffffffffu, w, j0 + j);
                    if (j0 + j >= many) break;
                    mass = __fadd_rn(mass, wj);
#pragma unroll
                    for (int e = 0; e < kEach; ++e) o[e] = __fmaf_rn(y[j][e], wj, o[e]);
                }
            }
        }
        const float inv = inverse(mass);
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] = __fmul_rn(o[e], inv);
        T *const to = static_cast<T *>(const_cast<void *>(p.out.p)) + t * p.out.ts + head * p.out.hs + lane * kEach;
        if constexpr (kEach == 2) {
            to[0] = from_float<T>(o[0]);
            to[1] = from_float<T>(o[1]);
        } else {
#pragma unroll
            for (int e = 0; e < kEach; e += 4) store4<T, ALIGNED>(to + e, o + e);
        }
        if (p.lse && lane == 0) p.lse[row] = mass == 0.0f ? -INFINITY : __fmul_rn(__fadd_rn(best - kBias, log2f(mass)), 0.6931471805599453f);
    }
}

template <typename T, int DIM>
cudaError_t join_dim(const SharedProblem &p, cudaStream_t s) {
    const int64_t rows = p.tokens * p.q_heads, warps = kThreads / 32;
    const bool aligned = reinterpret_cast<uintptr_t>(p.out.p) % (4 * sizeof(T)) == 0 && p.out.ts % 4 == 0 && p.out.hs % 4 == 0;
    // rows of a warp: a divisor of the heads, as many as leave each SM eight warps
    int each = 1;
    while (each < 8 && p.q_heads % (2 * each) == 0 && rows >= static_cast<int64_t>(2 * each) * 8 * num_sms()) each *= 2;
    const int64_t blocks = (rows / each + warps - 1) / warps;
    return launch_behind(aligned ? kv_shared_join_kernel<T, DIM, true> : kv_shared_join_kernel<T, DIM, false>, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, p,
                         each);
}

template <typename T>
cudaError_t join_typed(const SharedProblem &p, cudaStream_t s) {
    if (p.c.dim == 64) return join_dim<T, 64>(p, s);
    return p.c.dim == 128 ? join_dim<T, 128>(p, s) : join_dim<T, 256>(p, s);
}

}  // namespace

cudaError_t launch_kv_shared_join(const SharedProblem &p, cudaStream_t s) {
    if (p.dtype == OM_F32) return join_typed<float>(p, s);
    return p.dtype == OM_F16 ? join_typed<__half>(p, s) : join_typed<__nv_bfloat16>(p, s);
}

}  // namespace om
