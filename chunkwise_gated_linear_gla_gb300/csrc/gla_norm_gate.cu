// gla_norm_gate: the rows of every head's output on their way to the output projection, [B,H,T,d] to
// [B,T,H,d], normed and gated in one pass:
//
//     y = w (.) x / n(x) (.) act(g),    or, with the gate first,   u = x (.) act(g),  y = w (.) u / n(u),
//
// n the 2-norm sqrt(sum x^2 + eps), the root mean square or 1; act silu or the sigmoid. Backward, x^ = x / n, N = 1
// (2-norm) or d, and r(z) = (z - x^ (sum z (.) x^) / N) / n the norm's own gradient:
//
//     dx = r(dy (.) w (.) act),  dg = dy (.) w (.) x^ (.) act',  dw = sum dy (.) x^ (.) act;
//     gate first: du = r(dy (.) w),  dx = du (.) act,  dg = du (.) x (.) act',  dw = sum dy (.) u^.
//
// Bound by HBM: x and g read, y written once (backward: x, g and dy read, dx and dg written). A row is LPR lanes of
// K pieces of eight values, the rows in the order of y (a token's heads side by side); two rows' loads are in flight per
// thread. The weight's gradient is summed in fp32 over a thread's rows, its block, then the blocks, each in a fixed order.
#include <cmath>
#include <cstring>

#include "gla_internal.h"
#include "gla_rows.cuh"
#include "gla_span.h"

namespace gla {
namespace {

constexpr int NT = 256;

struct GateArgs {
    const void* x; const void* g; const float* w; void* y;
    const void* dy; void* dx; void* dg; float* part;
    long long sx[3], sg[3], sdx[3], sdg[3];   // strides (b, h, t) in elements
    long long rows;
    int H, T, d, norm, act, first;
    float eps;
};

__device__ __forceinline__ float act_of(float g, int silu, float& slope)
{
    const float s = sigmoid(g);
    if (silu) {
        slope = fmaf(g * s, 1.f - s, s);
        return g * s;
    }
    slope = s * (1.f - s);
    return s;
}

template <typename E, int LPR, int K, bool BWD, bool FIRST>
__global__ void __launch_bounds__(NT, K > 2 ? (BWD ? 1 : 2) : BWD ? 2 : 4) gla_norm_gate_kernel(GateArgs a)
{
    constexpr int RPB = NT / LPR, U = BWD || K > 1 ? 1 : 2;
    __shared__ float red[BWD ? RPB : 1][BWD ? LPR * K * VEC : 1];
    const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
    float w[K][VEC], dw[K][VEC];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int lo = (k * LPR + l) * VEC;
        in[k] = lo < a.d;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            w[k][j] = a.w && in[k] ? a.w[lo + j] : 1.f;
            dw[k][j] = 0.f;
        }
    }
    const float invn = a.norm == GLA_NORM_RMS ? 1.f / (float)a.d : 1.f;
    for (long long r0 = (long long)blockIdx.x * RPB * U; r0 < a.rows; r0 += (long long)gridDim.x * RPB * U) {
        typename Raw<E>::type xr[U][K], gr[U][K], yr[U][K];
        long long xo[U], go[U], dxo[U], dgo[U], yo[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long r = r0 + u * RPB + row;
            on[u] = r < a.rows;
            const long long q = on[u] ? r : 0;
            long long bt, b;
            int h, t;
            if (a.rows <= 0x7fffffff) {
                const unsigned n = (unsigned)q / (unsigned)a.H;
                h = (int)((unsigned)q - n * (unsigned)a.H);
                b = n / (unsigned)a.T;
                t = (int)(n - (unsigned)b * (unsigned)a.T);
            } else {
                bt = q / a.H;
                h = (int)(q - bt * a.H);
                b = bt / a.T;
                t = (int)(bt - b * a.T);
            }
            xo[u] = b * a.sx[0] + h * a.sx[1] + t * a.sx[2];
            go[u] = b * a.sg[0] + h * a.sg[1] + t * a.sg[2];
            yo[u] = q * a.d;
            if constexpr (BWD) {
                dxo[u] = b * a.sdx[0] + h * a.sdx[1] + t * a.sdx[2];
                dgo[u] = b * a.sdg[0] + h * a.sdg[1] + t * a.sdg[2];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int lo = (k * LPR + l) * VEC;
                const bool ok = on[u] && in[k];
                xr[u][k] = fetch(ok ? static_cast<const E*>(a.x) + xo[u] + lo : nullptr);
                gr[u][k] = fetch(ok && a.g ? static_cast<const E*>(a.g) + go[u] + lo : nullptr);
                if constexpr (BWD) yr[u][k] = fetch(ok ? static_cast<const E*>(a.dy) + yo[u] + lo : nullptr);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[K][VEC], ac[K][VEC], sl[K][VEC], xin[K][VEC];
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                unpack(xr[u][k], x[k]);
                unpack(gr[u][k], ac[k]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (a.g) ac[k][j] = act_of(ac[k][j], a.act == GLA_ACT_SILU, sl[k][j]);
                    else { ac[k][j] = 1.f; sl[k][j] = 0.f; }
                    if constexpr (BWD) xin[k][j] = x[k][j];
                    if (FIRST) x[k][j] *= ac[k][j];
                    s = fmaf(x[k][j], x[k][j], s);
                }
            }
            float inv = 1.f;
            if (a.norm != GLA_NORM_NONE) {
                inv = rsqrtf(fmaf(row_sum<LPR>(s), invn, a.eps));
                if (BWD && !on[u]) inv = 0.f;      // a row that is none holds zeros: with eps = 0, 1 / 0
            }
            if constexpr (!BWD) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        x[k][j] *= inv * w[k][j];
                        if (!FIRST) x[k][j] *= ac[k][j];
                    }
                    if (on[u] && in[k]) save8(static_cast<E*>(a.y) + yo[u] + (k * LPR + l) * VEC, x[k]);
                }
            } else {
                float z[K][VEC], m = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    unpack(yr[u][k], z[k]);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        x[k][j] *= inv;                                        // x^
                        const float dyx = z[k][j] * x[k][j];
                        dw[k][j] = fmaf(dyx, FIRST ? 1.f : ac[k][j], dw[k][j]);
                        sl[k][j] *= FIRST ? xin[k][j] : dyx * w[k][j];       // dg, or what du is multiplied by
                        z[k][j] *= FIRST ? w[k][j] : w[k][j] * ac[k][j];
                        m = fmaf(z[k][j], x[k][j], m);
                    }
                }
                if (a.norm != GLA_NORM_NONE) m = row_sum<LPR>(m) * invn;
                else m = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int lo = (k * LPR + l) * VEC;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        z[k][j] = inv * fmaf(-x[k][j], m, z[k][j]);
                        if (FIRST) {
                            sl[k][j] *= z[k][j];
                            z[k][j] *= ac[k][j];
                        }
                    }
                    if (on[u] && in[k]) {
                        save8(static_cast<E*>(a.dx) + dxo[u] + lo, z[k]);
                        if (a.g) save8(static_cast<E*>(a.dg) + dgo[u] + lo, sl[k]);
                    }
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) red[row][(k * LPR + l) * VEC + j] = dw[k][j];
        __syncthreads();
        for (int i = threadIdx.x; i < a.d; i += NT) {
            float s = 0.f;
            for (int k = 0; k < RPB; ++k) s += red[k][i];
            a.part[(size_t)blockIdx.x * a.d + i] = s;
        }
    }
}

long long blocks_of(const GateArgs& a, int sms, bool bwd)
{
    const int lpr = a.d <= 64 ? 8 : a.d <= 128 ? 16 : 32, u = bwd || a.d > 256 ? 1 : 2;
    const long long per = NT / lpr * u, n = (a.rows + per - 1) / per;
    const long long most = bwd ? 4LL * sms : 1LL << 30;    // backward: few blocks, few partials
    return n < most ? n : most;
}

template <typename E, bool BWD, bool FIRST>
cudaError_t launch(const GateArgs& a, int sms, cudaStream_t s)
{
    const unsigned g = (unsigned)blocks_of(a, sms, BWD);
    if (a.d <= 64) gla_norm_gate_kernel<E, 8, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else if (a.d <= 128) gla_norm_gate_kernel<E, 16, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else if (a.d <= 256) gla_norm_gate_kernel<E, 32, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else if (a.d <= 512) gla_norm_gate_kernel<E, 32, 2, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else gla_norm_gate_kernel<E, 32, 4, BWD, FIRST><<<g, NT, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename E, bool BWD>
cudaError_t launch(const GateArgs& a, int sms, cudaStream_t s)
{
    return a.first ? launch<E, BWD, true>(a, sms, s) : launch<E, BWD, false>(a, sms, s);
}

gla_status check(const gla_norm_gate_params* p)
{
    if (!p || p->B <= 0 || p->H <= 0 || p->T < 0 || p->d <= 0 || p->d % 16 != 0) return GLA_ERR_INVALID_ARG;
    if (p->dtype != GLA_BF16 && p->dtype != GLA_FP32) return GLA_ERR_INVALID_ARG;
    if (p->norm != GLA_NORM_NONE && p->norm != GLA_NORM_L2 && p->norm != GLA_NORM_RMS) return GLA_ERR_INVALID_ARG;
    if (p->activation != GLA_ACT_SILU && p->activation != GLA_ACT_SIGMOID) return GLA_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && !p->x) return GLA_ERR_INVALID_ARG;
    if ((long long)p->B * p->T > (1LL << 40) / p->H) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (int i = 0; i < 3; ++i)
        if (p->x_stride[i] * (long long)e % 16 != 0 || p->gate_stride[i] * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;
    for (const void* x : {p->x, p->gate})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(p->w, 4)) return GLA_ERR_INVALID_ARG;
    if (p->d > 1024) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

GateArgs common(const gla_norm_gate_params* p)
{
    GateArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = p->x; a.g = p->gate; a.w = p->w;
    for (int i = 0; i < 3; ++i) { a.sx[i] = p->x_stride[i]; a.sg[i] = p->gate_stride[i]; }
    a.rows = (long long)p->B * p->H * p->T;
    a.H = p->H; a.T = p->T; a.d = p->d; a.norm = p->norm; a.act = p->activation; a.first = p->gate_first != 0;
    a.eps = p->eps;
    return a;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

gla_status gla_norm_gate(const gla_norm_gate_params* p, void* y, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if ((p->T > 0 && !y) || !aligned(y, 16)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    const Span in[] = {span(p->x, p->x_stride, p->B, p->H, p->T, p->d, e),
                       span(p->gate, p->gate_stride, p->B, p->H, p->T, p->d, e), flat(p->w, p->d * 4)};
    for (const Span& s : in)
        if (overlap(flat(y, (size_t)p->B * p->H * p->T * p->d * e), s)) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK || p->T == 0) return st;
    GateArgs a = common(p);
    a.y = y;
    const cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16, false>(a, sms, stream) : launch<float, false>(a, sms, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

size_t gla_norm_gate_bwd_workspace_size(const gla_norm_gate_params* p)
{
    int sms = 0;
    if (check(p) != GLA_OK || p->T == 0 || !p->w) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    return (size_t)blocks_of(common(p), sms, true) * p->d * 4;
}

gla_status gla_norm_gate_bwd(const gla_norm_gate_params* p, const gla_norm_gate_grads* g, void* workspace,
                             size_t workspace_bytes, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (!g || (p->T > 0 && (!g->grad_y || !g->grad_x || (p->gate && !g->grad_gate)))) return GLA_ERR_INVALID_ARG;
    if ((g->grad_w && !p->w) || (g->grad_gate && !p->gate)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (int i = 0; i < 3; ++i)
        if (g->x_stride[i] * (long long)e % 16 != 0 || g->gate_stride[i] * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;
    for (const void* x : {g->grad_y, (const void*)g->grad_x, (const void*)g->grad_gate})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(g->grad_w, 4) || !aligned(workspace, 256)) return GLA_ERR_INVALID_ARG;
    const Span in[] = {span(p->x, p->x_stride, p->B, p->H, p->T, p->d, e),
                       span(p->gate, p->gate_stride, p->B, p->H, p->T, p->d, e), flat(p->w, p->d * 4),
                       flat(g->grad_y, (size_t)p->B * p->H * p->T * p->d * e)};
    // grad_x and grad_gate may be interleaved slices of one tensor (their rows apart): only equal starts are
    // refused between them
    const Span out[] = {span(g->grad_x, g->x_stride, p->B, p->H, p->T, p->d, e),
                        span(g->grad_gate, g->gate_stride, p->B, p->H, p->T, p->d, e), flat(g->grad_w, p->d * 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return GLA_ERR_INVALID_ARG;
        if (i < 2 && overlap(out[i], out[2])) return GLA_ERR_INVALID_ARG;
    }
    if (p->T > 0 && g->grad_x == g->grad_gate) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!apart(g->x_stride, p->B, p->H, p->T, p->d) ||
                     (p->gate && !apart(g->gate_stride, p->B, p->H, p->T, p->d))))
        return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    if (p->T == 0) {
        const cudaError_t r = g->grad_w ? cudaMemsetAsync(g->grad_w, 0, p->d * 4, stream) : cudaSuccess;
        return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
    }
    GateArgs a = common(p);
    const long long blocks = blocks_of(a, sms, true);
    if (g->grad_w && (!workspace || workspace_bytes < (size_t)blocks * p->d * 4)) return GLA_ERR_WORKSPACE;
    a.dy = g->grad_y; a.dx = g->grad_x; a.dg = g->grad_gate;
    for (int i = 0; i < 3; ++i) { a.sdx[i] = g->x_stride[i]; a.sdg[i] = g->gate_stride[i]; }
    a.part = g->grad_w ? static_cast<float*>(workspace) : nullptr;
    cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16, true>(a, sms, stream) : launch<float, true>(a, sms, stream);
    if (r == cudaSuccess && g->grad_w) r = launch_column_sum(a.part, blocks, p->d, ColumnOuts{{{g->grad_w, p->d}}}, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
