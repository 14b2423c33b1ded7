// kv_shared_join.cu -- joins what attention to a shared prefix and to a sequence's own tokens left of each row: the
// weighted means, by weights sum 2^(maximum - best).
//
// One warp a row (token and query head): it finds the blocks that had parts of its row from the lengths, as they cut
// them (kv_shared_items.cuh), takes the maximum over all parts, then one pass over their values. Order and arithmetic follow from
// the lengths alone.
//
// Bound: the latency of its lookups for few rows, L2 for many (4 dim bytes a row and part, written a moment before).

#include <type_traits>

#include "decode_device.cuh"
#include "kv_shared_items.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kThreads = 128;
constexpr float kBias = 8.0f;  // sums are 2^8 times the exponentials'

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Without a maximum a part saw nothing (its sum is 0) or scores that are all NaN (its sum is NaN, and stays).
__device__ __forceinline__ float joined(float sum, float top, float best) { return top == -INFINITY ? sum : __fmul_rn(sum, ex2(top - best)); }

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

template <typename T, int DIM, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) kv_shared_join_kernel(const __grid_constant__ SharedProblem p) {
    constexpr int kEach = DIM / 32;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, heads = static_cast<int>(p.q_heads);
    wait_for_earlier();
    if (row >= static_cast<int>(p.tokens) * heads) return;
    const int t = row / heads, head = row - t * heads;
    // what does not depend on anything is asked for first
    const float2 own = __ldcg(p.own_state + row);
    float o[kEach];
    load_values(p.own + static_cast<int64_t>(row) * DIM + lane * kEach, o);
    const int t_first = p.cu[0], t_last = p.cu[p.seqs];
    // the row's group, and the units before it
    const SharedGroup mine_first = shared_group(p, lane);
    const int total = shared_units(p, mine_first);
    if (t < t_first || t >= t_last) return;  // no sequence's
    int count = 0, first = 0, at = 0;
    if (total > 0) {
        const int per = shared_per_block(p, total);
        int before = 0;
#pragma unroll 1
        for (int64_t base = 0; base < p.groups; base += 32) {
            const SharedGroup g = base == 0 ? mine_first : shared_group(p, base + lane);
            const int n = static_cast<int>(g.n);
            int up = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            const unsigned here = __ballot_sync(0xffffffffu, n > 0 && t >= g.t0 && t < g.t0 + g.rows / p.group);
            if (here != 0) {
                const int from = __ffs(here) - 1;
                const int t0 = __shfl_sync(0xffffffffu, g.t0, from), blocks = __shfl_sync(0xffffffffu, g.row_blocks, from);
                const int units = __shfl_sync(0xffffffffu, g.units, from);
                before += __shfl_sync(0xffffffffu, up - n, from);
                const int h = head / p.group, r = (t - t0) * p.group + head % p.group;
                const int begin = before + (h * blocks + r / kSharedRows) * units;
                const int c = begin / per;
                count = (begin + units - 1) / per - c + 1;
                first = 2 * c + (begin > c * per);  // a part that does not start its block's share is in the second slot
                at = r % kSharedRows;
                break;
            }
            before += __shfl_sync(0xffffffffu, up, 31);
        }
    }
    // part j of the prefix; an item that one block had is at its row's place
    const bool whole = count == 1;
    auto place = [&](int j) -> int64_t { return whole ? static_cast<int64_t>(row) : static_cast<int64_t>(j == 0 ? first : (first | 1) - 1 + 2 * j) * p.slot_rows + at; };
    const float2 *const states = whole ? p.whole_state : p.slot_state;
    const float *const values = whole ? p.whole : p.slots;
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
        const int many = min(count - base, 32);
        constexpr int kAhead = 8;  // parts in flight
#pragma unroll 1
        for (int j0 = 0; j0 < many; j0 += kAhead) {
            float y[kAhead][kEach];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                load_values(values + place(min(base + j0 + j, count - 1)) * DIM + lane * kEach, y[j]);
            }
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
    const float inv = shared_inverse(mass);
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

template <typename T, int DIM>
cudaError_t join_dim(const SharedProblem &p, cudaStream_t s) {
    const int64_t rows = p.tokens * p.q_heads, warps = kThreads / 32;
    const bool aligned = reinterpret_cast<uintptr_t>(p.out.p) % (4 * sizeof(T)) == 0 && p.out.ts % 4 == 0 && p.out.hs % 4 == 0;
    return launch_behind(aligned ? kv_shared_join_kernel<T, DIM, true> : kv_shared_join_kernel<T, DIM, false>,
                         dim3(static_cast<unsigned>((rows + warps - 1) / warps)), dim3(kThreads), 0, s, p);
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
