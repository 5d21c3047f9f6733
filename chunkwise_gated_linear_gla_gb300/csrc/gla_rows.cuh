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

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) { float r; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x)); return r; }
__device__ __forceinline__ float rcp(float x) { float r; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x)); return r; }

// 1 / (1 + exp(-x)); the argument's rounding leaves |x| 2^-24 of it. 0 and 1 at the infinities.
__device__ __forceinline__ float sig(float x) { return rcp(1.f + ex2(-kLog2e * x)); }

// Pairs of fp32 values, as the packed instructions take them.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pk(float a, float b) { f2 r; asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b)); return r; }
__device__ __forceinline__ void up(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { f2 r; asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { f2 r; asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c)); return r; }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { f2 r; asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b)); return r; }
__device__ __forceinline__ f2 ex2_2(f2 v) { float a, b; up(v, a, b); return pk(ex2(a), ex2(b)); }

__device__ __forceinline__ f2 both(float c) { return pk(c, c); }
// sig of a pair.
__device__ __forceinline__ f2 sig(f2 x)
{
    float a, b;
    up(add2(ex2_2(mul2(x, both(-kLog2e))), both(1.f)), a, b);
    return pk(rcp(a), rcp(b));
}
__device__ __forceinline__ uint32_t bf16x2(f2 v)
{
    float a, b;
    uint32_t u;
    up(v, a, b);
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(b), "f"(a));
    return u;
}
// Eight values to p, rounded to its type.
__device__ __forceinline__ void keep8(float* p, const f2 (&r)[4])
{
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(r[0], r[1]);
    *(reinterpret_cast<ulonglong2*>(p) + 1) = make_ulonglong2(r[2], r[3]);
}
__device__ __forceinline__ void keep8(__nv_bfloat16* p, const f2 (&r)[4])
{
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(r[0]), bf16x2(r[1]), bf16x2(r[2]), bf16x2(r[3]));
}
// Eight loaded values as pairs.
__device__ __forceinline__ void wide(const uint4& w, f2 (&x)[4])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = pk(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
}
__device__ __forceinline__ void wide(const Raw<float>::type& w, f2 (&x)[4])
{
    x[0] = pk(w.a.x, w.a.y); x[1] = pk(w.a.z, w.a.w); x[2] = pk(w.b.x, w.b.y); x[3] = pk(w.b.z, w.b.w);
}
__device__ __forceinline__ float sum2(f2 v) { float a, b; up(v, a, b); return a + b; }

}  // namespace gla
