// gla_delta_bwd_step: the gradients of the gated delta rule token by token, for fp32 inputs
// and shapes outside the chunk form. With S the state entering token t, S~ = exp(log_g) S,
// r = v - k S~, u = beta r, S+ = S~ + k^T u, and D the gradient of S+ (o's part included):
//
//     D   += scale q^T do           dq = scale do S+^T
//     du   = k D,  dbeta = du . r   dk = u D^T - dr S~^T
//     dr   = beta du = dv           D~ = D - k^T dr
//     dlog_g = <D~, S~>             D <- exp(log_g) D~   (the gradient of S)
//
// A CTA owns kDeltaBwdTile columns of one head; D stays in registers. The states entering the
// tokens come from the kept ones (one per kDeltaKeep tokens, left by the forward recurrence):
// each group of tokens is run forward again into a scratch that only its own threads read.
// Sums over the columns (dq, dk, dlog_g, dbeta) leave as partials per tile; gla_delta_bwd_sum
// adds them, and the heads that share a key row, in a fixed order: no atomics.
//
// Bound by instruction issue and by the reductions across lanes (two shuffled sums per row and
// token): 256 tokens of 64 fp32 heads, dk = dv = 128, 0.79 ms. This is the form for parity and odd
// shapes; bf16 training runs the chunk form.
#include <cuda_bf16.h>

#include "gla_delta_internal.h"

namespace gla {
namespace {

constexpr int NT = 256, NW = NT / 32, TB = kDeltaKeep, CT = kDeltaBwdTile;
constexpr int CG = CT / 4, RG = NT / CG;   // 16 lanes along the columns, 16 row groups

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

__device__ __forceinline__ float4 f4(float x) { return make_float4(x, x, x, x); }
__device__ __forceinline__ float4 fma4(float s, float4 a, float4 b) {
    return make_float4(fmaf(s, a.x, b.x), fmaf(s, a.y, b.y), fmaf(s, a.z, b.z), fmaf(s, a.w, b.w));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
}

template <typename E, int DK>
__global__ void __launch_bounds__(NT) gla_delta_bwd_step_kernel(DeltaBwdStep a)
{
    constexpr int RPT = DK / RG;
    __shared__ float sq[TB][DK], sk[TB][DK], sal[TB], sbe[TB];
    __shared__ __align__(16) float sv[TB][CT], sdo[TB][CT], red[2][NW][CT];
    __shared__ float reds[2][NW];

    const int tid = threadIdx.x, c = tid % CG, r = tid / CG, warp = tid / 32, lane = tid % 32;
    const int bh = blockIdx.x, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int tile = blockIdx.y, c0 = tile * CT, col = c0 + 4 * c;
    const bool in = col < a.dv;
    const int row0 = r * RPT;
    const size_t BH = (size_t)a.B * a.H;
    const int ngr = (a.T + TB - 1) / TB;

    float4 D[RPT];
    const size_t sbase = (size_t)bh * a.dk * a.dv + col;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        D[i] = a.dST && in && row0 + i < a.dk
                   ? *reinterpret_cast<const float4*>(a.dST + sbase + (size_t)(row0 + i) * a.dv) : f4(0.f);

    const E* gq = static_cast<const E*>(a.q) + (size_t)bk * a.T * a.dk;
    const E* gk = static_cast<const E*>(a.k) + (size_t)bk * a.T * a.dk;
    const E* gv = static_cast<const E*>(a.v) + (size_t)bh * a.T * a.dv;
    const E* gdo = static_cast<const E*>(a.dO) + (size_t)bh * a.T * a.dv;
    float* pq = a.part_q + ((size_t)tile * BH + bh) * a.T * a.dk;
    float* pk = a.part_k + ((size_t)tile * BH + bh) * a.T * a.dk;
    float* pg = a.part_g + ((size_t)tile * BH + bh) * a.T;
    float* pb = a.part_b + ((size_t)tile * BH + bh) * a.T;
    E* gdv = static_cast<E*>(a.dv_out) + (size_t)bh * a.T * a.dv;
    // this thread's own slots of the scratch: token, row
    float4* scr = reinterpret_cast<float4*>(a.scratch) + ((size_t)tile * BH + bh) * TB * RPT * NT + tid;

    int flip = 0;
    // sum over the rows of four columns' values, to every thread of the column group
    auto over_rows = [&](float4 x) -> float4 {
        x.x += __shfl_xor_sync(~0u, x.x, 16); x.y += __shfl_xor_sync(~0u, x.y, 16);
        x.z += __shfl_xor_sync(~0u, x.z, 16); x.w += __shfl_xor_sync(~0u, x.w, 16);
        if (lane < 16) *reinterpret_cast<float4*>(&red[flip][warp][4 * c]) = x;
        __syncthreads();
        x = f4(0.f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(&red[flip][w][4 * c]);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        flip ^= 1;
        return x;
    };
    auto over_cols = [&](float x) -> float {   // over the 16 lanes of a row group
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        return x;
    };

    for (int g = ngr - 1; g >= 0; --g) {
        const int t0 = g * TB, n = min(TB, a.T - t0);
        __syncthreads();
        for (int i = tid; i < n * DK; i += NT) {
            const int t = i / DK, x = i % DK;
            sq[t][x] = x < a.dk ? to_f(gq[(size_t)(t0 + t) * a.dk + x]) : 0.f;
            sk[t][x] = x < a.dk ? to_f(gk[(size_t)(t0 + t) * a.dk + x]) : 0.f;
        }
        for (int i = tid; i < n * CT; i += NT) {
            const int t = i / CT, x = i % CT;
            const bool ok = c0 + x < a.dv;
            sv[t][x] = ok ? to_f(gv[(size_t)(t0 + t) * a.dv + c0 + x]) : 0.f;
            sdo[t][x] = ok ? to_f(gdo[(size_t)(t0 + t) * a.dv + c0 + x]) : 0.f;
        }
        if (tid < n) {
            sal[tid] = a.log_g ? expf(a.log_g[(size_t)bh * a.T + t0 + tid]) : 1.f;
            sbe[tid] = to_f(static_cast<const E*>(a.beta)[(size_t)bh * a.T + t0 + tid]);
        }
        __syncthreads();
        // forward over the group: the decayed state S~ of every token to the scratch, and v
        // becomes the token's r = v - k S~
        float4 S[RPT];
        const float* kp = a.keep + ((size_t)bh * ngr + g) * a.dk * a.dv + col;
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            S[i] = in && row0 + i < a.dk ? *reinterpret_cast<const float4*>(kp + (size_t)(row0 + i) * a.dv) : f4(0.f);
        for (int t = 0; t < n; ++t) {
            const float al = sal[t];
            float4 ks = f4(0.f);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                S[i] = make_float4(al * S[i].x, al * S[i].y, al * S[i].z, al * S[i].w);
                scr[((size_t)t * RPT + i) * NT] = S[i];
                ks = fma4(sk[t][row0 + i], S[i], ks);
            }
            ks = over_rows(ks);
            const float4 v = *reinterpret_cast<const float4*>(&sv[t][4 * c]);
            const float4 rr = make_float4(v.x - ks.x, v.y - ks.y, v.z - ks.z, v.w - ks.w);
            const float be = sbe[t];
#pragma unroll
            for (int i = 0; i < RPT; ++i)
                S[i] = fma4(be * sk[t][row0 + i], rr, S[i]);
            __syncthreads();              // every row group has read v
            if (r == 0) *reinterpret_cast<float4*>(&sv[t][4 * c]) = rr;
        }
        __syncthreads();
        for (int t = n - 1; t >= 0; --t) {
            const float al = sal[t], be = sbe[t];
            const float4 rr = *reinterpret_cast<const float4*>(&sv[t][4 * c]);
            const float4 go = *reinterpret_cast<const float4*>(&sdo[t][4 * c]);
            float4 Sd[RPT], du = f4(0.f);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                Sd[i] = scr[((size_t)t * RPT + i) * NT];
                const float k = sk[t][row0 + i];
                D[i] = fma4(a.scale * sq[t][row0 + i], go, D[i]);
                du = fma4(k, D[i], du);
            }
            du = over_rows(du);
            const float4 dr = make_float4(be * du.x, be * du.y, be * du.z, be * du.w);
            float dg = 0.f;
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float k = sk[t][row0 + i];
                const float4 Sn = fma4(be * k, rr, Sd[i]);   // S+
                const float q = over_cols(dot4(Sn, go)) * a.scale;
                const float kk = over_cols(be * dot4(D[i], rr) - dot4(Sd[i], dr));
                if (c == 0 && row0 + i < a.dk) {
                    pq[(size_t)(t0 + t) * a.dk + row0 + i] = q;
                    pk[(size_t)(t0 + t) * a.dk + row0 + i] = kk;
                }
                D[i] = fma4(-k, dr, D[i]);
                dg += dot4(D[i], Sd[i]);
                D[i] = make_float4(al * D[i].x, al * D[i].y, al * D[i].z, al * D[i].w);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dg += __shfl_xor_sync(~0u, dg, o);
            const float db = over_cols(dot4(du, rr));   // every row group holds the same du and r
            if (lane == 0) reds[t & 1][warp] = dg;
            if (r == 0 && in) {
                E* o = gdv + (size_t)(t0 + t) * a.dv + col;
                put(o, dr.x); put(o + 1, dr.y); put(o + 2, dr.z); put(o + 3, dr.w);
            }
            __syncthreads();
            if (tid == 0) {
                float x = 0.f;
#pragma unroll
                for (int w = 0; w < NW; ++w) x += reds[t & 1][w];
                pg[t0 + t] = x;
                pb[t0 + t] = db;
            }
        }
    }
    if (a.dS0 && in) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (row0 + i < a.dk) *reinterpret_cast<float4*>(a.dS0 + sbase + (size_t)(row0 + i) * a.dv) = D[i];
    }
}

// dq, dk: one thread per four values of a key row; dlog_g, dbeta: one per token and head.
template <typename E>
__global__ void __launch_bounds__(256) gla_delta_bwd_sum_kernel(DeltaBwdSum a)
{
    const long long nrow4 = (long long)a.B * a.Hk * a.T * (a.dk / 4), BHT = (long long)a.B * a.H * a.T;
    const int share = a.H / a.Hk;
    const long long step = (long long)gridDim.x * blockDim.x, first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (a.dq || a.dk_out)
        for (long long i = first; i < nrow4; i += step) {
            const long long x = i * 4, per = (long long)a.T * a.dk;
            const long long bk = x / per, rest = x % per;
            float4 q = f4(0.f), k = f4(0.f);
            for (int s = 0; s < share; ++s)
                for (int t = 0; t < a.tiles; ++t) {
                    const long long at = (t * (long long)a.B * a.H + bk * share + s) * per + rest;
                    const float4 u = *reinterpret_cast<const float4*>(a.part_q + at);
                    const float4 w = *reinterpret_cast<const float4*>(a.part_k + at);
                    q.x += u.x; q.y += u.y; q.z += u.z; q.w += u.w;
                    k.x += w.x; k.y += w.y; k.z += w.z; k.w += w.w;
                }
            if (a.dq) {
                E* o = static_cast<E*>(a.dq) + x;
                put(o, q.x); put(o + 1, q.y); put(o + 2, q.z); put(o + 3, q.w);
            }
            if (a.dk_out) {
                E* o = static_cast<E*>(a.dk_out) + x;
                put(o, k.x); put(o + 1, k.y); put(o + 2, k.z); put(o + 3, k.w);
            }
        }
    if (a.dlog_g || a.dbeta)
        for (long long i = first; i < BHT; i += step) {
            float g = 0.f, be = 0.f;
            for (int t = 0; t < a.tiles; ++t) {
                g += a.part_g[t * BHT + i];
                be += a.part_b[t * BHT + i];
            }
            if (a.dlog_g) a.dlog_g[i] = g;
            if (a.dbeta) put(static_cast<E*>(a.dbeta) + i, be);
        }
}

template <typename E>
cudaError_t launch_e(const DeltaBwdStep& a, cudaStream_t s) {
    const dim3 g((unsigned)(a.B * a.H), (a.dv + CT - 1) / CT);
    if (a.dk <= 64) gla_delta_bwd_step_kernel<E, 64><<<g, NT, 0, s>>>(a);
    else if (a.dk <= 128) gla_delta_bwd_step_kernel<E, 128><<<g, NT, 0, s>>>(a);
    else gla_delta_bwd_step_kernel<E, 256><<<g, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_bwd_step(const DeltaBwdStep& a, cudaStream_t s)
{
    return a.dtype == GLA_BF16 ? launch_e<__nv_bfloat16>(a, s) : launch_e<float>(a, s);
}

cudaError_t launch_delta_bwd_sum(const DeltaBwdSum& a, cudaStream_t s)
{
    const long long n = (long long)a.B * a.Hk * a.T * (a.dk / 4), m = (long long)a.B * a.H * a.T;
    const long long want = ((n > m ? n : m) + 255) / 256, most = (long long)a.sms * 8;
    const unsigned g = (unsigned)(want < most ? (want > 0 ? want : 1) : most);
    if (a.dtype == GLA_BF16) gla_delta_bwd_sum_kernel<__nv_bfloat16><<<g, 256, 0, s>>>(a);
    else gla_delta_bwd_sum_kernel<float><<<g, 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace gla
