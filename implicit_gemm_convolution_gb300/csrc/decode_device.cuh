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

// Waits until the kernels before this one in its stream have finished and their writes are visible, and lets the next
// kernel's blocks take the room that this one's leave (they wait here too): what it saves is the launch of
// a kernel between two short ones.
__device__ __forceinline__ void wait_for_earlier() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

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
// The nearest codes of four finite values, ties to even, clamped to the range; byte i is value i's.
template <int KV>
__device__ __forceinline__ uint32_t encode4(float x, float y, float z, float w) {
    if constexpr (KV == OM_I8) {
        // adding 1.5 * 2^23 rounds to a whole number, whose low byte is the code
        auto code = [](float v) { return __float_as_uint(__fadd_rn(fminf(fmaxf(v, -127.0f), 127.0f), 12582912.0f)); };
        return __byte_perm(__byte_perm(code(x), code(y), 0x0040), __byte_perm(code(z), code(w), 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(z, w), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
}

// The values of a word's four codes.
template <int KV>
__device__ __forceinline__ void decode4(uint32_t w, float *v) {
    if constexpr (KV == OM_I8) {
        // 2^23 + (code + 128), by its bits, less 2^23 + 128: exact
        w ^= 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7650 + i)), 8388736.0f);
    } else {
        uint32_t h[2];
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(h[0]), "=r"(h[1]) : "r"(w));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            __half2 x;
            memcpy(&x, &h[i], 4);
            const float2 f = __half22float2(x);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
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

}  // namespace om
