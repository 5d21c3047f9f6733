// The selective scan's device helpers and launchers, shared by its forward, backward and entry points.
#pragma once

#include <cuda_bf16.h>
#include <cstddef>
#include <cstdint>

#include "gla_internal.h"
#ifdef __CUDACC__
#include "gla_rows.cuh"
#endif

namespace gla {

constexpr int kSsmTile = 16;      // tokens per tile, and between two kept states of the backward

// What a pass over [B,T,D] channels reads and writes. Group g of the channels, Dg = D / G wide, reads row g of B and C.
struct SsmArgs {
    const void* x; const void* dt; const void* z; const void* Bm; const void* Cm;
    long long sx[2], sdt[2], sz[2], sB[2], sC[2];   // strides (b, t) in elements
    const float* A; const float* Dk; const float* bias; const float* S0;
    void* y; float* ST;
    int B, T, D, G, N, softplus;
    int nseg, seg;                // segments of the sequence, tokens in each (a multiple of kSsmTile)
    float* segS;                  // [B][nseg - 1][D][N] states: each segment's own, then those entering 1 .. nseg - 1
    float* sumd;                  // [B][nseg - 1][D] sums of delta
    float* keep;                  // KEEP: [B][ceil(T / kSsmTile)][D][N] states entering every tile
    // backward
    const void* dy; const float* dST;
    void* dx; void* ddt; void* dz; float* dS0;
    float* part_bc;               // [tiles per group][B][T][G][2 N]
    float* part_p;                // [B nseg][D N + 2 D]: dA, dD, ddt_bias
    float* segG;                  // [B][nseg - 1][D][N] gradients of the states after segments 0 .. nseg - 2
    int ctiles;                   // channel tiles per group
};

// What a walk over a segment does.
enum SsmMode {
    kSsmOut = 0,      // y and the last state
    kSsmState = 1,    // the segment's state from zero and its sum of delta (all segments but the last)
    kSsmKeep = 2,     // the state entering every tile
    kSsmRev = 3,      // backwards: the gradient of the state before the segment, from zero (all but the first)
};

cudaError_t launch_ssm_step(const SsmArgs& a, gla_dtype dtype, int sms, cudaStream_t s);
cudaError_t launch_ssm_walk(const SsmArgs& a, int mode, gla_dtype dtype, cudaStream_t s);
// The states entering the segments from each segment's own, in place; `rev`: from the last, into segG.
cudaError_t launch_ssm_scan(const SsmArgs& a, bool rev, int sms, cudaStream_t s);
cudaError_t launch_ssm_bwd(const SsmArgs& a, gla_dtype dtype, cudaStream_t s);
cudaError_t launch_ssm_bc_sum(const SsmArgs& a, void* dB, void* dC, gla_dtype dtype, int sms, cudaStream_t s);
int ssm_walk_channels(int N);     // channels per block of the walk, and of the backward
int ssm_bwd_channels(int N);
int ssm_walk_warps(int N);

#ifdef __CUDACC__

// log(1 + exp(v)): log(1 + u) = 2 atanh(s), s = u / (2 + u) <= 1/3, u = exp(-|v|), so that small steps keep their digits (a
// logarithm of the rounded 1 + u would lose them). atanh(s) / s in s^2 by Chebyshev interpolation at five points of [0, 1/9]: good to
// 8e-9 with its coefficients rounded. -inf gives 0.
__device__ __forceinline__ float softplus(float v)
{
    const float u = ex2(-kLog2e * fabsf(v)), s = u * rcp(2.f + u), q = s * s;
    float p = fmaf(q, 0.14078889787197113f, 0.13982579112052917f);
    p = fmaf(p, q, 0.20012298226356506f);
    p = fmaf(p, q, 0.3333316147327423f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// The same for a pair.
__device__ __forceinline__ f2 softplus(f2 v)
{
    float a, b, c, d;
    up(mul2(v, both(kLog2e)), a, b);
    const f2 u = pk(ex2(-fabsf(a)), ex2(-fabsf(b)));
    up(add2(u, both(2.f)), c, d);
    const f2 s = mul2(u, pk(rcp(c), rcp(d))), q = mul2(s, s);
    f2 p = fma2(q, both(2 * 0.14078889787197113f), both(2 * 0.13982579112052917f));
    p = fma2(p, q, both(2 * 0.20012298226356506f));
    p = fma2(p, q, both(2 * 0.3333316147327423f));
    p = fma2(p, q, both(2.f));
    up(v, a, b);
    return fma2(s, p, pk(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}

// S states from p, as fp32 pairs.
template <int S>
__device__ __forceinline__ void states(const __nv_bfloat16* p, f2 (&r)[S / 2])
{
    uint32_t u[S / 2];
    if constexpr (S == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
    } else {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        u[0] = q.x; u[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < S / 2; ++i) r[i] = pk(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
template <int S>
__device__ __forceinline__ void states(const float* p, f2 (&r)[S / 2])
{
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const ulonglong2 q = *(reinterpret_cast<const ulonglong2*>(p) + i);
        r[2 * i] = q.x;
        r[2 * i + 1] = q.y;
    }
}

// Eight parameters of channels c .. from p, zeros without.
__device__ __forceinline__ void params8(const float* p, bool in, f2 (&r)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = p && in ? pk(__ldg(p + 2 * i), __ldg(p + 2 * i + 1)) : 0ull;
}

__device__ __forceinline__ void copy16(void* smem, const void* g, bool ok)
{
    const unsigned d = (unsigned)__cvta_generic_to_shared(smem);
    const int n = ok ? 16 : 0;                     // the rest of the 16 bytes is zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(g), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// Copies of tiles of TT rows of W values each (a multiple of 16 bytes) by NT threads into shared memory [TT][W], tile after tile, forwards
// or backwards. A thread's pieces lie in one column, so a tile costs it an addition and a comparison a piece. Rows from
// t1 on and columns from `cols` on become zeros.
template <typename E, int TT, int W, int NT>
struct TileCopy {
    static constexpr int PER = 16 / sizeof(E), COLS = W / PER, ROWS = NT / COLS < TT ? NT / COLS : TT;
    static_assert(W % PER == 0 && (COLS >= NT || NT % COLS == 0) && TT % ROWS == 0, "whole pieces");
    const E* p;
    const E* any;                      // an address that can be read
    long long st;
    int row, col, t;
    bool in;
    // first: the first tile's first row
    __device__ __forceinline__ void start(const E* src, long long stride, int first, int cols)
    {
        col = threadIdx.x % COLS * PER;
        row = threadIdx.x / COLS;
        in = col < cols && row < TT;
        st = stride;
        any = src;
        t = first + row;
        p = src + t * stride + col;
    }
    __device__ __forceinline__ void go(E* smem, int t1, int step)
    {
        if (row < TT) {
#pragma unroll
            for (int k = 0; k < TT; k += ROWS) {
                const bool ok = in && t + k < t1;
                copy16(smem + (row + k) * W + col, ok ? p + k * st : any, ok);
            }
        }
        t += step;
        p += step * st;
    }
};

#endif
}  // namespace gla
