// decode_device.cuh -- device helpers of the decoding operators: element and
// code conversions, and the ragged-batch lookups with their bounds checks.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "decode.h"

namespace om {

template <typename T>
__device__ __forceinline__ float to_float(T v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        return static_cast<float>(v);
    }
}

template <typename T>
__device__ __forceinline__ T from_float(float v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else if constexpr (std::is_same_v<T, __half>) {
        return __float2half_rn(v);
    } else {
        return __float2bfloat16_rn(v);
    }
}

// Four consecutive elements; p is aligned to them where ALIGNED.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void load4(const T *p, float *v) {
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_float(p[i]);
    } else if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        T e[4];
        memcpy(e, &w, 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_float(e[i]);
    }
}

template <typename T, bool ALIGNED>
__device__ __forceinline__ void store4(T *p, const float *v) {
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = from_float<T>(v[i]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        T e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = from_float<T>(v[i]);
        uint2 w;
        memcpy(&w, e, 8);
        *reinterpret_cast<uint2 *>(p) = w;
    }
}

// Codes. OM_I8: whole numbers -127 .. 127; OM_E4M3: 8-bit floats up to 448.
template <int KV>
__device__ __forceinline__ float code_top() {
    return KV == OM_I8 ? 127.0f : 448.0f;
}

// The nearest code of a finite value, ties to even, clamped to the range.
template <int KV>
__device__ __forceinline__ uint32_t encode(float x) {
    x = fminf(fmaxf(x, -code_top<KV>()), code_top<KV>());
    if constexpr (KV == OM_I8) {
        return static_cast<uint32_t>(__float2int_rn(x)) & 0xffu;
    } else {
        return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
    }
}

template <int KV>
__device__ __forceinline__ float decode(uint32_t byte) {
    if constexpr (KV == OM_I8) {
        return static_cast<float>(static_cast<int8_t>(byte & 0xffu));
    } else {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(byte & 0xffu), __NV_E4M3);
        return __half2float(__half(h));
    }
}

// The tokens of sequence b in a batch of `tokens`: [*lo, *hi), inside the
// batch whatever cu holds.
__device__ __forceinline__ void token_range(const int32_t *cu, int64_t b, int64_t tokens,
                                            int64_t *lo, int64_t *hi) {
    const int64_t a = cu[b], e = cu[b + 1];
    *lo = a < 0 ? 0 : (a > tokens ? tokens : a);
    *hi = e < *lo ? *lo : (e > tokens ? tokens : e);
}

// The sequence that token t belongs to, or seqs when none does; every thread of
// the block takes part. The count of sequences that end at or before t: one
// round of loads for up to blockDim.x sequences.
__device__ __forceinline__ int64_t block_sequence_of(const int32_t *cu, int64_t seqs, int64_t t) {
    int64_t b = 0;
    for (int64_t i = 0; i < seqs; i += blockDim.x) {
        const int64_t j = i + threadIdx.x;
        b += __syncthreads_count(j < seqs && cu[j + 1] <= t);
    }
    return b;
}

}  // namespace om
