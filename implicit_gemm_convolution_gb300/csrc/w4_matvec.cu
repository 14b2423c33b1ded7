// w4_matvec.cu -- products of a few rows with 4-bit weights:
// y[i][j] = sum_p x[i][p] * (u[j][p] - z[j][p / group]) * s[j][p / group].

#include <type_traits>

#include "decode_device.cuh"
#include "om_internal.h"

namespace om {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float load_scale(const void *s, int dtype, int64_t i) {
    if (dtype == OM_F32) return static_cast<const float *>(s)[i];
    if (dtype == OM_F16) return __half2float(static_cast<const __half *>(s)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(s)[i]);
}

// One warp per output, its lanes over the bytes of the weight row.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) w4_simple_kernel(const __grid_constant__ W4Problem p) {
    const int lane = threadIdx.x & 31;
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32, i = blockIdx.y;
    if (j >= p.n) return;
    const T *x = static_cast<const T *>(p.x) + i * p.ldx;
    const uint8_t *u = p.u + j * p.ldu;
    float acc = 0.0f;
    for (int64_t c = lane; 2 * c < p.k; c += 32) {
        const int64_t g = 2 * c / p.group;  // groups are even: both codes of a byte share one
        const float s = load_scale(p.s, p.s_dtype, j * p.lds + g);
        const int z = p.z ? p.z[j * p.ldz + g] : 8, b = u[c];
        acc = __fmaf_rn(to_float(x[2 * c]), __fmul_rn(static_cast<float>((b & 15) - z), s), acc);
        if (2 * c + 1 < p.k) acc = __fmaf_rn(to_float(x[2 * c + 1]), __fmul_rn(static_cast<float>((b >> 4) - z), s), acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, o));
    if (lane == 0) static_cast<T *>(p.y)[i * p.ldy + j] = from_float<T>(acc);
}

template <typename T>
cudaError_t run(const W4Problem &p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.n + kWarps - 1) / kWarps), static_cast<unsigned>(p.m));
    w4_simple_kernel<T><<<grid, kWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4_matvec(const W4Problem &p, cudaStream_t s) {
    if (p.x_dtype == OM_F32) return run<float>(p, s);
    if (p.x_dtype == OM_F16) return run<__half>(p, s);
    return run<__nv_bfloat16>(p, s);
}

}  // namespace om
