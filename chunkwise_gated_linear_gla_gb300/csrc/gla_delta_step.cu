// gla_delta_step: the gated delta rule token by token,
//
//     S~ = exp(log_g) S,   u = beta (v - k S~),   S <- S~ + k^T u,   o = scale q S,
//
// for single tokens (decoding), a few drafted ones, fp32 inputs and shapes outside the chunk
// form. A CTA owns CT columns of one head's state in registers; columns are independent, so
// nothing crosses CTAs. Thread (r, c) holds rows r RPT .. of four columns. Both products with
// the old state, k S and q S, are formed in one walk over the registers and reduced together
// (o = scale (exp(g) q S + (q . k) u)), so a token costs one block barrier.
//
// Bound by the state's bytes at small T: 4 dk dv read and written once per call. CT = 128
// columns by 256 threads keeps 16 16-byte loads per thread in flight at dk = 128; when the
// tiles are fewer than the SMs they narrow to 32 columns so that more SMs pull (the launcher).
#include <cuda_bf16.h>

#include "gla_delta_internal.h"

namespace gla {
namespace {

constexpr int NT = 256;
constexpr int NW = NT / 32;
constexpr int TB = 16;   // tokens staged in shared memory at a time

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

// N consecutive values from shared memory (16-byte aligned), as fp32.
template <int N>
__device__ __forceinline__ void read_row(const float* p, float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(p + i);
        x[i] = f.x; x[i + 1] = f.y; x[i + 2] = f.z; x[i + 3] = f.w;
    }
}
template <int N>
__device__ __forceinline__ void read_row(const __nv_bfloat16* p, float (&x)[N]) {
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[i + 2 * j] = __uint_as_float(u[j] << 16);
                x[i + 2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(p + i);
            x[i] = __uint_as_float(w.x << 16);
            x[i + 1] = __uint_as_float(w.x & 0xffff0000u);
            x[i + 2] = __uint_as_float(w.y << 16);
            x[i + 3] = __uint_as_float(w.y & 0xffff0000u);
        }
    }
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

// DK: keys padded to 64, 128 or 256 (rows from dk on are zero); CT: columns of the tile.
template <typename E, int DK, int CT>
__global__ void __launch_bounds__(NT) gla_delta_step_kernel(DeltaStep a)
{
    constexpr int CG = CT / 4;            // column groups (threads along the columns)
    constexpr int RG = NT / CG;           // row groups
    constexpr int RPT = DK / RG;          // rows per thread
    static_assert(CG <= 32 && RPT % 4 == 0, "thread layout");
    __shared__ __align__(16) E sq[TB][DK], sk[TB][DK], sv[TB][CT];
    __shared__ float sal[TB], sbe[TB];
    __shared__ __align__(16) float red[2][NW][2][CT];
    __shared__ float redqk[2][NW];

    const int tid = threadIdx.x, c = tid % CG, r = tid / CG, warp = tid / 32, lane = tid % 32;
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int c0 = blockIdx.y * CT, col = c0 + 4 * c;
    const bool in = col < a.dv;           // dv is a multiple of 16: a group of four is in or out
    const int row0 = r * RPT;

    float4 S[RPT];
    const size_t sbase = (size_t)bh * a.dk * a.dv + col;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        S[i] = a.S0 && in && row0 + i < a.dk
                   ? __ldcs(reinterpret_cast<const float4*>(a.S0 + sbase + (size_t)(row0 + i) * a.dv))
                   : make_float4(0.f, 0.f, 0.f, 0.f);

    const E* gq = static_cast<const E*>(a.q) + (size_t)bk * a.T * a.dk;
    const E* gk = static_cast<const E*>(a.k) + (size_t)bk * a.T * a.dk;
    const E* gv = static_cast<const E*>(a.v) + (size_t)bh * a.T * a.dv;
    E* go = a.O ? static_cast<E*>(a.O) + (size_t)bh * a.T * a.dv : nullptr;
    const int nkeep = (a.T + kDeltaKeep - 1) / kDeltaKeep;
    constexpr int V = 16 / sizeof(E);     // values per 16-byte piece

    for (int t0 = 0; t0 < a.T; t0 += TB) {
        const int n = min(TB, a.T - t0);
        __syncthreads();                  // the block before is read
        for (int i = tid; i < n * (DK / V); i += NT) {
            const int t = i / (DK / V), x = i % (DK / V) * V;
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
            const bool ok = x < a.dk;
            *reinterpret_cast<uint4*>(&sq[t][x]) =
                ok ? *reinterpret_cast<const uint4*>(gq + (size_t)(t0 + t) * a.dk + x) : z;
            *reinterpret_cast<uint4*>(&sk[t][x]) =
                ok ? *reinterpret_cast<const uint4*>(gk + (size_t)(t0 + t) * a.dk + x) : z;
        }
        for (int i = tid; i < n * (CT / V); i += NT) {
            const int t = i / (CT / V), x = i % (CT / V) * V;
            if (c0 + x < a.dv)
                *reinterpret_cast<uint4*>(&sv[t][x]) =
                    *reinterpret_cast<const uint4*>(gv + (size_t)(t0 + t) * a.dv + c0 + x);
        }
        if (tid < n) {
            sal[tid] = a.log_g ? expf(a.log_g[(size_t)bh * a.T + t0 + tid]) : 1.f;
            sbe[tid] = to_f(static_cast<const E*>(a.beta)[(size_t)bh * a.T + t0 + tid]);
        }
        __syncthreads();
        if (a.keep && in) {
            float* kp = a.keep + ((size_t)bh * nkeep + t0 / kDeltaKeep) * a.dk * a.dv + col;
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                if (row0 + i < a.dk) *reinterpret_cast<float4*>(kp + (size_t)(row0 + i) * a.dv) = S[i];
        }
        for (int t = 0; t < n; ++t) {
            float kr[RPT];
            float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
            float qk = 0.f;
            read_row<RPT>(&sk[t][row0], kr);
            {
                float qr[RPT];
                read_row<RPT>(&sq[t][row0], qr);
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    ks.x = fmaf(kr[i], S[i].x, ks.x); ks.y = fmaf(kr[i], S[i].y, ks.y);
                    ks.z = fmaf(kr[i], S[i].z, ks.z); ks.w = fmaf(kr[i], S[i].w, ks.w);
                    qs.x = fmaf(qr[i], S[i].x, qs.x); qs.y = fmaf(qr[i], S[i].y, qs.y);
                    qs.z = fmaf(qr[i], S[i].z, qs.z); qs.w = fmaf(qr[i], S[i].w, qs.w);
                    qk = fmaf(qr[i], kr[i], qk);
                }
            }
            // the row groups of one warp, then the warps through shared memory
#pragma unroll
            for (int o = CG; o < 32; o <<= 1) {
                ks.x += __shfl_xor_sync(~0u, ks.x, o); ks.y += __shfl_xor_sync(~0u, ks.y, o);
                ks.z += __shfl_xor_sync(~0u, ks.z, o); ks.w += __shfl_xor_sync(~0u, ks.w, o);
                qs.x += __shfl_xor_sync(~0u, qs.x, o); qs.y += __shfl_xor_sync(~0u, qs.y, o);
                qs.z += __shfl_xor_sync(~0u, qs.z, o); qs.w += __shfl_xor_sync(~0u, qs.w, o);
                qk += __shfl_xor_sync(~0u, qk, o);
            }
            const int bf = t & 1;         // two sets: a token's reads end before the token after next writes
            if (lane < CG) {
                *reinterpret_cast<float4*>(&red[bf][warp][0][4 * c]) = ks;
                *reinterpret_cast<float4*>(&red[bf][warp][1][4 * c]) = qs;
                if (lane == 0) redqk[bf][warp] = qk;
            }
            __syncthreads();
            ks = qs = make_float4(0.f, 0.f, 0.f, 0.f);
            qk = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(&red[bf][w][0][4 * c]);
                const float4 y = *reinterpret_cast<const float4*>(&red[bf][w][1][4 * c]);
                ks.x += x.x; ks.y += x.y; ks.z += x.z; ks.w += x.w;
                qs.x += y.x; qs.y += y.y; qs.z += y.z; qs.w += y.w;
                qk += redqk[bf][w];
            }
            const float al = sal[t], be = sbe[t];
            float vv[4] = {0.f, 0.f, 0.f, 0.f};
            if (in) read_row<4>(&sv[t][4 * c], vv);
            const float4 u = make_float4(be * (vv[0] - al * ks.x), be * (vv[1] - al * ks.y),
                                         be * (vv[2] - al * ks.z), be * (vv[3] - al * ks.w));
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                S[i].x = fmaf(kr[i], u.x, al * S[i].x); S[i].y = fmaf(kr[i], u.y, al * S[i].y);
                S[i].z = fmaf(kr[i], u.z, al * S[i].z); S[i].w = fmaf(kr[i], u.w, al * S[i].w);
            }
            if (go && r == 0 && in)
                store4(go + (size_t)(t0 + t) * a.dv + col,
                       make_float4(a.scale * fmaf(qk, u.x, al * qs.x), a.scale * fmaf(qk, u.y, al * qs.y),
                                   a.scale * fmaf(qk, u.z, al * qs.z), a.scale * fmaf(qk, u.w, al * qs.w)));
        }
    }
    if (a.ST && in) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (row0 + i < a.dk)
                __stcs(reinterpret_cast<float4*>(a.ST + sbase + (size_t)(row0 + i) * a.dv), S[i]);
    }
}

template <typename E, int DK>
cudaError_t launch_dk(const DeltaStep& a, cudaStream_t s) {
    // A thread holds at least four rows and at most 32 of them of four columns.
    constexpr int WIDE = DK <= 128 ? 128 : 64, NARROW = DK == 64 ? 64 : 32;
    const unsigned BH = (unsigned)(a.B * a.H);
    // Wide tiles move the most bytes per thread; with fewer of them than SMs, narrow ones put
    // more SMs on the same state.
    const long long wide = (long long)BH * ((a.dv + WIDE - 1) / WIDE);
    if (wide < a.sms || a.dv <= NARROW)
        gla_delta_step_kernel<E, DK, NARROW><<<dim3(BH, (a.dv + NARROW - 1) / NARROW), NT, 0, s>>>(a);
    else
        gla_delta_step_kernel<E, DK, WIDE><<<dim3(BH, (a.dv + WIDE - 1) / WIDE), NT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_e(const DeltaStep& a, cudaStream_t s) {
    if (a.dk <= 64) return launch_dk<E, 64>(a, s);
    if (a.dk <= 128) return launch_dk<E, 128>(a, s);
    return launch_dk<E, 256>(a, s);
}

}  // namespace

cudaError_t launch_delta_step(const DeltaStep& a, cudaStream_t s)
{
    return a.dtype == GLA_BF16 ? launch_e<__nv_bfloat16>(a, s) : launch_e<float>(a, s);
}

}  // namespace gla
