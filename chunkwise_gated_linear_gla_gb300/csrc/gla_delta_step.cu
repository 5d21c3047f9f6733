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
// dk = dv = 128, caches cold: the next token of 2048 heads 52 us, 5.2 TB/s; of 16 heads 6.2 us, launch latency;
// five tokens of 512 heads 25 us, two of them a token's barriers (calls back to back 24.1, with tiles of 64
// columns 26.7).
#include <cuda_bf16.h>

#include "gla_delta_dev.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using delta::fma2;
using delta::mul2;

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

// DK: keys padded to 64, 128 or 256 (rows from dk on are zero); CT: columns of the tile. Two CTAs per SM, of
// the half-size tiles three (4096 heads, dk = 64, dv = 128, one token: 60 us, with one CTA 101, with two 72).
template <typename E, int DK, int CT>
__global__ void __launch_bounds__(NT, DK * CT <= 8192 ? 3 : 2) gla_delta_step_kernel(DeltaStep a)
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

    float2 S[RPT][2];
    const size_t sbase = (size_t)bh * a.dk * a.dv + col;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
    {
        const float4 x = a.S0 && in && row0 + i < a.dk
                             ? __ldcs(reinterpret_cast<const float4*>(a.S0 + sbase + (size_t)(row0 + i) * a.dv))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
        S[i][0] = make_float2(x.x, x.y);
        S[i][1] = make_float2(x.z, x.w);
    }
    auto row4 = [&](int i) { return make_float4(S[i][0].x, S[i][0].y, S[i][1].x, S[i][1].y); };

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
                if (row0 + i < a.dk) *reinterpret_cast<float4*>(kp + (size_t)(row0 + i) * a.dv) = row4(i);
        }
        for (int t = 0; t < n; ++t) {
            float kr[RPT];
            float4 ks, qs;
            float qk = 0.f;
            read_row<RPT>(&sk[t][row0], kr);
            {
                float qr[RPT];
                read_row<RPT>(&sq[t][row0], qr);
                float2 kp[2] = {}, qp[2] = {};
#pragma unroll
                for (int i = 0; i < RPT; ++i) {
                    const float2 kk = make_float2(kr[i], kr[i]), qq = make_float2(qr[i], qr[i]);
                    kp[0] = fma2(kk, S[i][0], kp[0]);
                    kp[1] = fma2(kk, S[i][1], kp[1]);
                    qp[0] = fma2(qq, S[i][0], qp[0]);
                    qp[1] = fma2(qq, S[i][1], qp[1]);
                    qk = fmaf(qr[i], kr[i], qk);
                }
                ks = make_float4(kp[0].x, kp[0].y, kp[1].x, kp[1].y);
                qs = make_float4(qp[0].x, qp[0].y, qp[1].x, qp[1].y);
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
            const float2 u0 = make_float2(u.x, u.y), u1 = make_float2(u.z, u.w), aa = make_float2(al, al);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float2 kk = make_float2(kr[i], kr[i]);
                S[i][0] = fma2(kk, u0, mul2(aa, S[i][0]));
                S[i][1] = fma2(kk, u1, mul2(aa, S[i][1]));
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
                __stcs(reinterpret_cast<float4*>(a.ST + sbase + (size_t)(row0 + i) * a.dv), row4(i));
    }
}

__device__ __forceinline__ void cp16(void* dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

// The same recurrence for several tokens: nothing but the block's token loads is shared between
// warps, so no barrier stands between two tokens. A warp owns LC columns; lane (r, c) holds rows
// r RPT .. of one of them. A token's way from one state to the next is k S over 32 / LC lanes, two
// shuffles deep (three at dk = 256, where a lane cannot hold 64 rows of everything); o = scale q S of
// the token before, from the same state, is reduced beside it, and the next token's row is on its way
// from shared memory meanwhile. Bound by that latency: 256 tokens of two heads, fp32, dk = dv = 64,
// 37 us (59 with q . k formed ahead, three shuffles and nothing loaded early). Its state accesses
// are 32 bytes a row and warp, the reason why single tokens take the other kernel.
template <typename E, int DK>
__global__ void __launch_bounds__(DK <= 128 ? 128 : 256) gla_delta_tokens_kernel(DeltaStep a)
{
    constexpr int CT = 32, LC = DK <= 128 ? 8 : 4, NT = CT / LC * 32, RPT = DK * LC / 32, V = 16 / sizeof(E);
    __shared__ __align__(16) E sq[2][TB][DK], sk[2][TB][DK], sv[2][TB][CT];
    __shared__ float sal[2][TB], sbe[2][TB];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, c = lane % LC, r = lane / LC;
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int c0 = blockIdx.y * CT, lc = LC * warp + c, col = c0 + lc;
    const bool in = col < a.dv;
    const int row0 = r * RPT;

    const E* gq = static_cast<const E*>(a.q) + (size_t)bk * a.T * a.dk;
    const E* gk = static_cast<const E*>(a.k) + (size_t)bk * a.T * a.dk;
    const E* gv = static_cast<const E*>(a.v) + (size_t)bh * a.T * a.dv;
    E* go = a.O ? static_cast<E*>(a.O) + (size_t)bh * a.T * a.dv : nullptr;
    const int nkeep = (a.T + kDeltaKeep - 1) / kDeltaKeep;

    // tokens t0 .. of the sequence on their way to buffer f
    float next_g = 0.f, next_b = 0.f;
    auto fetch = [&](int t0, int f) {
        const int n = min(TB, a.T - t0);
        for (int i = tid; i < n * (DK / V); i += NT) {
            const int t = i / (DK / V), x = i % (DK / V) * V;
            if (x < a.dk) {
                cp16(&sq[f][t][x], gq + (size_t)(t0 + t) * a.dk + x);
                cp16(&sk[f][t][x], gk + (size_t)(t0 + t) * a.dk + x);
            }
        }
        for (int i = tid; i < n * (CT / V); i += NT) {
            const int t = i / (CT / V), x = i % (CT / V) * V;
            if (c0 + x < a.dv) cp16(&sv[f][t][x], gv + (size_t)(t0 + t) * a.dv + c0 + x);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (tid < n) {
            next_g = a.log_g ? a.log_g[(size_t)bh * a.T + t0 + tid] : 0.f;
            next_b = to_f(static_cast<const E*>(a.beta)[(size_t)bh * a.T + t0 + tid]);
        }
    };
    // the first warp's gates, once its block of tokens is done: waiting for them before it, that warp
    // came to every barrier a memory latency late
    auto put_gates = [&](int f) {
        if (tid < TB) {
            sal[f][tid] = expf(next_g);
            sbe[f][tid] = next_b;
        }
    };
    if (a.dk < DK)   // keys past dk are zero in both buffers, for good
        for (int i = tid; i < 2 * TB * (DK - a.dk); i += NT) {
            const int x = a.dk + i % (DK - a.dk), t = i / (DK - a.dk);
            (&sq[0][0][0])[t * DK + x] = E(0.f);
            (&sk[0][0][0])[t * DK + x] = E(0.f);
        }
    fetch(0, 0);
    put_gates(0);

    float2 S[RPT / 2];
    const size_t sbase = (size_t)bh * a.dk * a.dv + col;
#pragma unroll
    for (int i = 0; i < RPT / 2; ++i) {
        const int x = row0 + 2 * i;      // dk is a multiple of 16: a pair is in or out
        const bool ok = a.S0 && in && x < a.dk;
        S[i].x = ok ? a.S0[sbase + (size_t)x * a.dv] : 0.f;
        S[i].y = ok ? a.S0[sbase + (size_t)(x + 1) * a.dv] : 0.f;
    }

    // this lane's rows of x S
    auto sum = [&](const float (&x)[RPT]) {
        float2 z[2] = {};
#pragma unroll
        for (int i = 0; i < RPT / 2; ++i) z[i & 1] = fma2(make_float2(x[2 * i], x[2 * i + 1]), S[i], z[i & 1]);
        return (z[0].x + z[0].y) + (z[1].x + z[1].y);
    };
    const bool writes = go && r == 0 && in;
    size_t at = col;                     // of the next row of O to be written
    auto put = [&](float y) {
        if (writes) {
            if constexpr (sizeof(E) == 2) go[at] = __float2bfloat16_rn(a.scale * y);
            else go[at] = a.scale * y;
        }
        at += a.dv;
    };
    float q[RPT] = {};                   // of the token before
    for (int t0 = 0, f = 0; t0 < a.T; t0 += TB, f ^= 1) {
        const int n = min(TB, a.T - t0);
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (t0 + TB < a.T) fetch(t0 + TB, f ^ 1);
        if (a.keep && in) {
            float* kp = a.keep + ((size_t)bh * nkeep + t0 / kDeltaKeep) * a.dk * a.dv + col;
#pragma unroll
            for (int i = 0; i < RPT / 2; ++i)
                if (row0 + 2 * i < a.dk) {
                    kp[(size_t)(row0 + 2 * i) * a.dv] = S[i].x;
                    kp[(size_t)(row0 + 2 * i + 1) * a.dv] = S[i].y;
                }
        }
        // u = beta v - (beta alpha) k S: nothing but one fma waits for the sum
        float k[RPT], al, uv, ua;
        auto gate = [&](int t) {
            al = sal[f][t];
            uv = in ? sbe[f][t] * to_f(sv[f][t][lc]) : 0.f;
            ua = -sbe[f][t] * al;
        };
        gate(0);
        read_row<RPT>(&sk[f][0][row0], k);
#pragma unroll 4
        for (int t = 0; t < n; ++t) {
            float x = sum(k), y = sum(q);
            // what the next token takes (the row's last: itself again)
            const int nx = min(t + 1, n - 1);
            float kn[RPT];
            read_row<RPT>(&sk[f][nx][row0], kn);
            read_row<RPT>(&sq[f][t][row0], q);
#pragma unroll
            for (int o = LC; o < 32; o <<= 1) {
                const float x1 = __shfl_xor_sync(~0u, x, o), y1 = __shfl_xor_sync(~0u, y, o);
                x += x1;
                y += y1;
            }
            const float u = fmaf(ua, x, uv);
#pragma unroll
            for (int i = 0; i < RPT / 2; ++i)
                S[i] = fma2(make_float2(k[2 * i], k[2 * i + 1]), make_float2(u, u), mul2(make_float2(al, al), S[i]));
            gate(nx);
            if (t0 + t > 0) put(y);
#pragma unroll
            for (int i = 0; i < RPT; ++i) k[i] = kn[i];
        }
        put_gates(f ^ 1);
    }
    {
        float y = sum(q);
#pragma unroll
        for (int o = LC; o < 32; o <<= 1) y += __shfl_xor_sync(~0u, y, o);
        put(y);
    }
    if (a.ST && in) {
#pragma unroll
        for (int i = 0; i < RPT / 2; ++i)
            if (row0 + 2 * i < a.dk) {
                a.ST[sbase + (size_t)(row0 + 2 * i) * a.dv] = S[i].x;
                a.ST[sbase + (size_t)(row0 + 2 * i + 1) * a.dv] = S[i].y;
            }
    }
}

template <typename E, int DK>
cudaError_t launch_dk(const DeltaStep& a, cudaStream_t s) {
    // A thread holds at least four rows and at most 32 of them of four columns.
    constexpr int WIDE = DK <= 128 ? 128 : 64, NARROW = DK == 64 ? 64 : 32;
    const unsigned BH = (unsigned)(a.B * a.H);
    const long long wide = (long long)BH * ((a.dv + WIDE - 1) / WIDE);
    // Beyond a few tokens the barriers between them cost more than the tokens kernel's narrower state
    // accesses: with fewer wide tiles than SMs from three tokens on (dk = dv = 128, 16 heads, 5 tokens:
    // 8.9 us against 10.9), else from nine (512 heads, 8 tokens: 39.6 against 35.5, 12: 47.8 against 53.9).
    if (a.T > (wide < a.sms && DK <= 128 ? 2 : 8)) {
        gla_delta_tokens_kernel<E, DK><<<dim3((unsigned)(a.B * a.H), (a.dv + 31) / 32), DK <= 128 ? 128 : 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    // Wide tiles move the most bytes per thread; with fewer of them than SMs, narrow ones put
    // more SMs on the same state.
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
