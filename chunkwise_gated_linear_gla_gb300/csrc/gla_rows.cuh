// Eight values at a time from and to rows of bf16 or fp32, shared by the kernels that read and write rows.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace gla {

constexpr int VEC = 8;        // values per lane

// Eight values as loaded, and as fp32: a row waits in its own type (half the registers in bf16).
template <typename E> struct Raw;
template <> struct Raw<__nv_bfloat16> { typedef uint4 type; };
template <> struct Raw<float> { struct type { float4 a, b; }; };
__device__ __forceinline__ uint4 fetch(const __nv_bfloat16* p) {
    return p ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ Raw<float>::type fetch(const float* p) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    return p ? Raw<float>::type{__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1)}
             : Raw<float>::type{z, z};
}
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[VEC]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const Raw<float>::type& w, float (&x)[VEC]) {
    x[0] = w.a.x; x[1] = w.a.y; x[2] = w.a.z; x[3] = w.a.w; x[4] = w.b.x; x[5] = w.b.y; x[6] = w.b.z; x[7] = w.b.w;
}
__device__ __forceinline__ void save8(__nv_bfloat16* p, const float (&x)[VEC]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        u[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void save8(float* p, const float (&x)[VEC]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
}

// The sum over groups of LPR neighbouring lanes, in every lane.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// 1 / (1 + exp(-x)): 0 and 1 at the infinities.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + expf(-x)); }

}  // namespace gla
