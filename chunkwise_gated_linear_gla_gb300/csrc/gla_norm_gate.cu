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
// K pieces of eight values; a thread keeps its token and takes the token's heads one after the other, so that a row's address
// is a sum (the division into batch row and token is done once; once per row it was a third of the instructions, 49 us for the
// layer), two heads' loads in flight (of heads above 256 one, but twice the blocks: 65536 rows of 512 47 us with two, 39 so). 8 x 2048 tokens
// of 16 heads of 128: 33 us, 6.1 TB/s, 0.90 of the copy rate. The backward has one head in flight, asked for after the last one's stores, and two
// blocks an SM: too few bytes, 3.1 to 3.9 TB/s in bf16 up to 256 values (3.6 at 128), 4.2 to 5.6 in fp32. The weight's gradient is summed in fp32 over a thread's rows, its
// block, then the blocks, each in a fixed order.
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
    long long tokens;
    int H, T, d, norm, act, first;
    int hsplit;                               // heads per block
    float eps;
};

// act(g) and its slope.
__device__ __forceinline__ f2 act_of(f2 g, int silu, f2& slope)
{
    const f2 s = sig(g), left = fma2(s, both(-1.f), both(1.f));      // 1 - s
    if (silu) {
        const f2 a = mul2(g, s);
        slope = fma2(a, left, s);
        return a;
    }
    slope = mul2(s, left);
    return s;
}

template <typename E, int LPR, int K, bool BWD, bool FIRST>
__global__ void __launch_bounds__(NT, BWD ? (K > 2 ? 1 : 2) : K > 2 ? 2 : 4) gla_norm_gate_kernel(GateArgs a)
{
    constexpr int RPB = NT / LPR, U = BWD || K > 1 ? 1 : 2;
    __shared__ __align__(16) float red[BWD ? RPB : 1][BWD ? LPR * K * VEC : 4];
    const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
    f2 w[K][4], dw[K][4];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int lo = (k * LPR + l) * VEC;
        in[k] = lo < a.d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            w[k][j] = a.w && in[k] ? pk(a.w[lo + 2 * j], a.w[lo + 2 * j + 1]) : both(1.f);
            dw[k][j] = 0ull;
        }
    }
    const float invn = a.norm == GLA_NORM_RMS ? 1.f / (float)a.d : 1.f;
    const int h0 = blockIdx.y * a.hsplit, h1 = min(a.H, h0 + a.hsplit);
    for (long long t0 = (long long)blockIdx.x * RPB; t0 < a.tokens; t0 += (long long)gridDim.x * RPB) {
        const bool on = t0 + row < a.tokens;
        const long long tok = on ? t0 + row : 0;
        const long long b = a.tokens <= 0x7fffffff ? (unsigned)tok / (unsigned)a.T : tok / a.T, t = tok - b * a.T;
        const E* xp = static_cast<const E*>(a.x) + b * a.sx[0] + h0 * a.sx[1] + t * a.sx[2] + l * VEC;
        const E* gp = a.g ? static_cast<const E*>(a.g) + b * a.sg[0] + h0 * a.sg[1] + t * a.sg[2] + l * VEC : nullptr;
        const long long yo = (tok * a.H + h0) * a.d + l * VEC;
        E* yp = BWD ? nullptr : static_cast<E*>(a.y) + yo;
        const E* dyp = BWD ? static_cast<const E*>(a.dy) + yo : nullptr;
        E* dxp = BWD ? static_cast<E*>(a.dx) + b * a.sdx[0] + h0 * a.sdx[1] + t * a.sdx[2] + l * VEC : nullptr;
        E* dgp = BWD && a.g ? static_cast<E*>(a.dg) + b * a.sdg[0] + h0 * a.sdg[1] + t * a.sdg[2] + l * VEC : nullptr;
        for (int h = h0; h < h1; h += U) {
            typename Raw<E>::type xr[U][K], gr[U][K], yr[U][K];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const bool ok = on && in[k] && h + u < h1;
                    const int lo = k * LPR * VEC;
                    xr[u][k] = fetch(ok ? xp + u * a.sx[1] + lo : nullptr);
                    gr[u][k] = fetch(ok && gp ? gp + u * a.sg[1] + lo : nullptr);
                    if constexpr (BWD) yr[u][k] = fetch(ok ? dyp + u * a.d + lo : nullptr);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool row_on = on && h + u < h1;
                f2 x[K][4], ac[K][4], sl[K][4], s2 = 0ull;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    wide(xr[u][k], x[k]);
                    wide(gr[u][k], ac[k]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (gp) ac[k][j] = act_of(ac[k][j], a.act == GLA_ACT_SILU, sl[k][j]);
                        else { ac[k][j] = both(1.f); sl[k][j] = 0ull; }
                        if (FIRST) x[k][j] = mul2(x[k][j], ac[k][j]);
                        s2 = fma2(x[k][j], x[k][j], s2);
                    }
                }
                float inv = 1.f;
                if (a.norm != GLA_NORM_NONE) {
                    inv = rsqrtf(fmaf(row_sum<LPR>(sum2(s2)), invn, a.eps));
                    if (BWD && !row_on) inv = 0.f;      // a row that is none holds zeros: with eps = 0, 1 / 0
                }
                if constexpr (!BWD) {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[k][j] = mul2(x[k][j], mul2(w[k][j], both(inv)));
                            if (!FIRST) x[k][j] = mul2(x[k][j], ac[k][j]);
                        }
                        if (row_on && in[k]) keep8(yp + u * a.d + k * LPR * VEC, x[k]);
                    }
                } else {
                    f2 z[K][4], m2 = 0ull;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        f2 xin[4];
                        wide(yr[u][k], z[k]);
                        if (FIRST) wide(xr[u][k], xin);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            x[k][j] = mul2(x[k][j], both(inv));                     // x^
                            const f2 dyx = mul2(z[k][j], x[k][j]);
                            dw[k][j] = FIRST ? add2(dw[k][j], dyx) : fma2(dyx, ac[k][j], dw[k][j]);
                            // dg, or what du is multiplied by
                            sl[k][j] = mul2(sl[k][j], FIRST ? xin[j] : mul2(dyx, w[k][j]));
                            z[k][j] = mul2(z[k][j], FIRST ? w[k][j] : mul2(w[k][j], ac[k][j]));
                            m2 = fma2(z[k][j], x[k][j], m2);
                        }
                    }
                    const float m = a.norm != GLA_NORM_NONE ? row_sum<LPR>(sum2(m2)) * invn : 0.f;
#pragma unroll
                    for (int k = 0; k < K; ++k) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            z[k][j] = mul2(both(inv), fma2(x[k][j], both(-m), z[k][j]));
                            if (FIRST) {
                                sl[k][j] = mul2(sl[k][j], z[k][j]);
                                z[k][j] = mul2(z[k][j], ac[k][j]);
                            }
                        }
                        if (row_on && in[k]) {
                            keep8(dxp + k * LPR * VEC, z[k]);
                            if (gp) keep8(dgp + k * LPR * VEC, sl[k]);
                        }
                    }
                }
            }
            xp += U * a.sx[1];
            if (gp) gp += U * a.sg[1];
            if constexpr (BWD) {
                dyp += U * a.d;
                dxp += U * a.sdx[1];
                if (gp) dgp += U * a.sdg[1];
            } else {
                yp += U * a.d;
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
#pragma unroll
        for (int k = 0; k < K; ++k) keep8(&red[row][(k * LPR + l) * VEC], dw[k]);
        __syncthreads();
        const size_t blk = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
        for (int i = threadIdx.x; i < a.d; i += NT) {
            float s = 0.f;
            for (int k = 0; k < RPB; ++k) s += red[k][i];
            a.part[blk * a.d + i] = s;
        }
    }
}

// The heads are spread over blocks until every SM has two (3 x 1531 tokens of 4 heads of 512: 10.5 us, with four 12.5, with eight 16.5: the weights
// are read for one head, not two; 777 tokens of 16 heads of 256 4.8, 5.5 and 8.4); backward: as many blocks as are resident, few partials.
dim3 grid_of(GateArgs& a, int sms, bool bwd)
{
    const int lpr = a.d <= 16 ? 2 : a.d <= 32 ? 4 : a.d <= 64 ? 8 : a.d <= 128 ? 16 : 32, rows = NT / lpr;
    const long long tg = (a.tokens + rows - 1) / rows;
    const long long want = 2LL * sms;
    int split = 1;
    while (split < a.H && tg * split < want) split *= 2;
    if (split > a.H) split = a.H;
    a.hsplit = (a.H + split - 1) / split;
    const int gy = (a.H + a.hsplit - 1) / a.hsplit;
    long long gx = tg;
    const long long most = bwd ? (want + gy - 1) / gy : 1LL << 30;
    if (gx > most) gx = most;
    return dim3((unsigned)gx, gy);
}

template <typename E, bool BWD, bool FIRST>
cudaError_t launch(GateArgs a, int sms, cudaStream_t s)
{
    const dim3 g = grid_of(a, sms, BWD);
    if (a.d <= 16) gla_norm_gate_kernel<E, 2, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else if (a.d <= 32) gla_norm_gate_kernel<E, 4, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
    else if (a.d <= 64) gla_norm_gate_kernel<E, 8, 1, BWD, FIRST><<<g, NT, 0, s>>>(a);
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
    if ((long long)p->B * p->T > (1LL << 40) / p->H || p->H > 65535) return GLA_ERR_INVALID_ARG;
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
    a.tokens = (long long)p->B * p->T;
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
    GateArgs a = common(p);
    const dim3 g = grid_of(a, sms, true);
    return (size_t)g.x * g.y * p->d * 4;
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
    const dim3 grid = grid_of(a, sms, true);
    const long long blocks = (long long)grid.x * grid.y;
    if (g->grad_w && (!workspace || workspace_bytes < (size_t)blocks * p->d * 4)) return GLA_ERR_WORKSPACE;
    a.dy = g->grad_y; a.dx = g->grad_x; a.dg = g->grad_gate;
    for (int i = 0; i < 3; ++i) { a.sdx[i] = g->x_stride[i]; a.sdg[i] = g->gate_stride[i]; }
    a.part = g->grad_w ? static_cast<float*>(workspace) : nullptr;
    cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16, true>(a, sms, stream) : launch<float, true>(a, sms, stream);
    if (r == cudaSuccess && g->grad_w) r = launch_column_sum(a.part, blocks, p->d, ColumnOuts{{{g->grad_w, p->d}}}, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
