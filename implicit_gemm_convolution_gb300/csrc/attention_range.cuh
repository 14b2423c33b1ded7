// attention_range.cuh -- what the kernels whose softmax parts are joined have to agree on (kv_attention.cuh, kv_shared.cuh,
// kv_shared_join.cu): the ranges of exponentials, weights and units, and what a part's sum is worth beside others.
#pragma once

#include <cfloat>
#include <cstdint>
#include <cstring>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace om {

constexpr float kLog2e = 1.4426950408889634f;
// A tile's largest weight is 2^8 as its unit is set, and may go to 2^15 and 2^-1 with the same one: inside 16-bit
// range, its second part above the subnormals. The maximum may lag behind while exponentials are below 2^40. Sums are 2^8 times
// the exponentials'.
constexpr float kBias = 8.0f, kMost = 32768.0f, kLeast = 0.5f, kMostExp = 1099511627776.0f;
constexpr float kNone = -FLT_MAX;  // the maximum of no scores
// Units from 2^-126 to 2^126, and no smaller than a value scale by 2^100; a smaller one may not raise sums above 2^100.
constexpr float kLeastUnit = FLT_MIN, kLeastOfScale = 7.8886090522101181e-31f;
constexpr unsigned kMostUnit = 253u << 23;

// A value scale in units, finite: a weight of 0 stays 0.
__device__ __forceinline__ float in_units(float value, float per_unit) { return fminf(fmaxf(__fmul_rn(value, per_unit), -FLT_MAX), FLT_MAX); }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<unsigned>(e + 127) << 23); }
__device__ __forceinline__ float reciprocal(float power) { return __uint_as_float((254u << 23) - __float_as_uint(power)); }

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

}  // namespace om
