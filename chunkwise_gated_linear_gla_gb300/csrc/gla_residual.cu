// gla_residual_norm: what lies between two blocks of a layer stack, in one pass over the rows: the block's output x
// goes into the residual r, scaled and, if wanted, normed first, and the next block's normed input comes out,
//
//     u = x or x / n(x),   h = r + alpha scale (.) u,   y = w (.) h / n(h),   n(x) = sqrt(mean x^2 + eps).
//
// Backward, h^ = h / n(h), u^ = x / n(x), means over the row:
//
//     dr = dh + (dy (.) w - h^ mean(dy (.) w (.) h^)) / n(h),   dw = sum dy (.) h^,
//     du = alpha scale (.) dr,  dscale = alpha sum dr (.) u,    dx = du or (du - u^ mean(du (.) u^)) / n(x).
//
// The norm reads h as summed in fp32, before its rounding to the residual's type, and the backward forms it again
// from r and x, so that no gradient carries that rounding.
//
// Bound by HBM: x and r read, h and y written once (backward: x, r, dh, dy read, dx and dr written). Rows of up to 512
// values are a warp's, with shuffles for the sums; wider rows a block's, K pieces of eight values per thread: two pieces, as every sum
// over the row costs a thread 60 instructions (with one piece 51 us for the rows below). The vectors' gradients are summed in
// fp32 over a thread's rows, then over the blocks, each in a fixed order. 16384 bf16 rows of 2048 values, post norm and scale: 40 us,
// 6.7 TB/s, 0.98 of the copy rate; backward 77 us, 0.77, and above 4096 values, with a block an SM and no load between the row's sums, 2.7 to
// 3.2 TB/s in bf16 (fp32 3.1 to 4.1).
#include <cmath>
#include <cstring>

#include "gla_internal.h"
#include "gla_rows.cuh"
#include "gla_span.h"

namespace gla {
namespace {

constexpr int kWarpD = 512;          // the widest row that one warp takes
constexpr int kWarps = 8;            // warps (rows) per block of that form
constexpr int kMaxD = 16384;

struct ResArgs {
    const void* x; const void* r; const float* w; const float* scale;
    void* h; void* y;
    const void* dh; const void* dy; void* dx; void* dr; float* part;
    long long rows;
    int D, post;
    float alpha, eps;
};

// The sum of a value, or of two, over the row's threads, in every one of them.
template <int NTR, bool TWO>
__device__ __forceinline__ void sum_row(float& a, float& b, float2 (*red)[NTR / 32 + 1], int& turn)
{
    a = row_sum<32>(a);
    if (TWO) b = row_sum<32>(b);
    if constexpr (NTR > 32) {
        // two buffers in turn: a warp may be one sum ahead of another, not two
        if (threadIdx.x % 32 == 0) red[turn][threadIdx.x / 32] = make_float2(a, b);
        __syncthreads();
        a = 0.f;
        if (TWO) b = 0.f;
#pragma unroll
        for (int i = 0; i < NTR / 32; ++i) {
            const float2 v = red[turn][i];
            a += v.x;
            if (TWO) b += v.y;
        }
        turn ^= 1;
    }
}

template <typename E, typename R, int NTR, int K, bool BWD>
__global__ void __launch_bounds__(NTR == 32 ? 32 * kWarps : NTR, NTR == 32 ? (BWD ? 2 : 1) : BWD ? K < 4 ? 512 / NTR : 1 : NTR == 512 && K < 4 ? 2 : 1)
gla_residual_norm_kernel(ResArgs a)
{
    __shared__ float2 red[2][NTR / 32 + 1];
    int turn = 0;
    constexpr int RPB = NTR == 32 ? kWarps : 1;
    // The widest rows have one block to an SM. Its registers take the next row as soon as h is formed, before the row's sum and stores
    // (4096 bf16 rows of 16384 values 127 us a row at a time, 96 so); backward the vectors' sums lie in shared memory, each thread's
    // in places of its own (326 us with what the registers do not hold spilled, 271 so). Clusters of two and four blocks to a row, each
    // with 4096 values of it, wait longer for each other's sums: 194 and 594 us.
    constexpr bool AHEAD = !BWD && K == 4, SHARED = BWD && K == 4;
    extern __shared__ __align__(16) ulonglong2 sums_of[];         // [dw, ds][K][2][NTR]
    const int l = threadIdx.x % NTR;
    const float invn = 1.f / (float)a.D;
    bool in[K];
    f2 dw[BWD && !SHARED ? K : 1][4], ds[BWD && !SHARED ? K : 1][4];
    auto sums = [&](int which, int k, int half) -> ulonglong2& { return sums_of[((which * K + k) * 2 + half) * NTR + threadIdx.x]; };
#pragma unroll
    for (int k = 0; k < K; ++k) in[k] = (k * NTR + l) * VEC < a.D;
    if constexpr (BWD) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (SHARED) {
                sums(0, k, 0) = sums(0, k, 1) = sums(1, k, 0) = sums(1, k, 1) = make_ulonglong2(0ull, 0ull);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) dw[k][j] = ds[k][j] = 0ull;
            }
        }
    }
    // eight values of a vector (1 without it), times c
    auto vec = [&](const float* p, int k, float c, f2 (&f)[4]) {
        const float* q = p + (k * NTR + l) * VEC;
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            if (p && in[k]) {
                const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2*>(q + 2 * j));
                f[j] = v.x; f[j + 1] = v.y;
            } else {
                f[j] = f[j + 1] = both(1.f);
            }
        }
        if (c != 1.f)
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], both(c));
    };

    const long long step = (long long)gridDim.x * RPB;
    long long row = (long long)blockIdx.x * RPB + (NTR == 32 ? threadIdx.x / 32 : 0);
    typename Raw<E>::type xr[K], yr[BWD ? K : 1];
    typename Raw<R>::type rr[K], hr[BWD ? K : 1];
    auto load = [&](auto& to, const auto* from, long long of) {
#pragma unroll
        for (int k = 0; k < K; ++k) to[k] = fetch(from && in[k] && of < a.rows ? from + of * a.D + (k * NTR + l) * VEC : nullptr);
    };
    auto load_xr = [&](long long of) {
        load(xr, static_cast<const E*>(a.x), of);
        load(rr, static_cast<const R*>(a.r), of);
    };
    if (AHEAD) load_xr(row);
    for (; row < a.rows; row += step) {
        const long long at = row * a.D + l * VEC;
        if (!AHEAD) load_xr(row);
        if constexpr (BWD) {
            load(yr, static_cast<const E*>(a.dy), row);
            if (!SHARED) load(hr, static_cast<const R*>(a.dh), row);
        }
        float invx = 1.f, none = 0.f;
        if (a.post) {
            f2 s = 0ull;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 x[4];
                wide(xr[k], x);
#pragma unroll
                for (int j = 0; j < 4; ++j) s = fma2(x[j], x[j], s);
            }
            float t = sum2(s);
            sum_row<NTR, false>(t, none, red, turn);
            invx = rsqrtf(fmaf(t, invn, a.eps));
        }
        // h, its squares' sum and (backward) that of dy w h
        f2 h[K][4], s2 = 0ull, m2 = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f2 x[4], sc[4];
            wide(xr[k], x);
            wide(rr[k], h[k]);
            vec(a.scale, k, a.alpha * invx, sc);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[k][j] = fma2(x[j], sc[j], h[k][j]);
                s2 = fma2(h[k][j], h[k][j], s2);
            }
            if constexpr (BWD) {
                f2 wv[4], g[4];
                vec(a.w, k, 1.f, wv);
                wide(yr[k], g);
#pragma unroll
                for (int j = 0; j < 4; ++j) m2 = fma2(mul2(g[j], wv[j]), h[k][j], m2);
            }
        }
        if (AHEAD) load_xr(row + step);
        if constexpr (SHARED) load(hr, static_cast<const R*>(a.dh), row);      // (into r's registers)
        float s = sum2(s2), m = sum2(m2);
        sum_row<NTR, BWD>(s, m, red, turn);
        const float inv = rsqrtf(fmaf(s, invn, a.eps));
        if constexpr (!BWD) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k]) continue;
                const long long o = at + k * NTR * VEC;
                if (a.h) keep8(static_cast<R*>(a.h) + o, h[k]);
                f2 wv[4];
                vec(a.w, k, inv, wv);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[k][j] = mul2(h[k][j], wv[j]);
                keep8(static_cast<E*>(a.y) + o, h[k]);
            }
        } else {
            const f2 i2 = both(inv), mm = both(-m * inv * invn);        // -mean(dy w h^)
            f2 q2 = 0ull;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                f2 x[4], sc[4], wv[4], g[4], d[4];
                wide(xr[k], x);
                wide(yr[k], g);
                wide(hr[k], d);
                vec(a.w, k, 1.f, wv);
                vec(a.scale, k, 1.f, sc);
                f2 dwk[4], dsk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 hh = mul2(h[k][j], i2);
                    if constexpr (SHARED) dwk[j] = mul2(g[j], hh);
                    else dw[k][j] = fma2(g[j], hh, dw[k][j]);
                    h[k][j] = fma2(i2, fma2(hh, mm, mul2(g[j], wv[j])), d[j]);        // dr
                    const f2 p = mul2(h[k][j], x[j]);
                    if constexpr (SHARED) dsk[j] = mul2(p, both(invx));
                    else ds[k][j] = fma2(p, both(invx), ds[k][j]);
                    q2 = fma2(p, sc[j], q2);
                }
                if constexpr (SHARED) {
                    if (a.part) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ulonglong2 &u = sums(0, k, half), &v = sums(1, k, half);
                            u = make_ulonglong2(add2(u.x, dwk[2 * half]), add2(u.y, dwk[2 * half + 1]));
                            v = make_ulonglong2(add2(v.x, dsk[2 * half]), add2(v.y, dsk[2 * half + 1]));
                        }
                    }
                }
                if (in[k] && a.dr) keep8(static_cast<R*>(a.dr) + at + k * NTR * VEC, h[k]);
            }
            float q = 0.f;
            if (a.post) {
                q = sum2(q2);
                sum_row<NTR, false>(q, none, red, turn);
                q *= invx * invx * invn;                               // mean(du u^) / n(x)
            }
            if (a.dx) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (!in[k]) continue;
                    f2 x[4], sc[4];
                    wide(xr[k], x);
                    vec(a.scale, k, 1.f, sc);
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = mul2(both(a.alpha * invx), fma2(x[j], both(-q), mul2(h[k][j], sc[j])));
                    keep8(static_cast<E*>(a.dx) + at + k * NTR * VEC, x);
                }
            }
        }
    }
    if constexpr (BWD) {
        if (!a.part) return;
        if constexpr (!SHARED) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) ds[k][j] = mul2(ds[k][j], both(a.alpha));
        }
        if constexpr (SHARED) {
            float* p = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k]) continue;
                const ulonglong2 u = sums(0, k, 0), v = sums(0, k, 1), y = sums(1, k, 0), z = sums(1, k, 1);
                const f2 dwk[4] = {u.x, u.y, v.x, v.y}, al = both(a.alpha);
                const f2 dsk[4] = {mul2(y.x, al), mul2(y.y, al), mul2(z.x, al), mul2(z.y, al)};
                keep8(p + (k * NTR + l) * VEC, dwk);
                keep8(p + a.D + (k * NTR + l) * VEC, dsk);
            }
        } else if constexpr (NTR > 32) {
            float* p = a.part + (size_t)blockIdx.x * 2 * a.D;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k]) continue;
                keep8(p + (k * NTR + l) * VEC, dw[k]);
                keep8(p + a.D + (k * NTR + l) * VEC, ds[k]);
            }
        } else {
            __shared__ float sums[kWarps][K * 32 * VEC];
            for (int z = 0; z < 2; ++z) {
                __syncthreads();
#pragma unroll
                for (int k = 0; k < K; ++k) keep8(&sums[threadIdx.x / 32][(k * 32 + l) * VEC], z ? ds[k] : dw[k]);
                __syncthreads();
                for (int i = threadIdx.x; i < a.D; i += 32 * kWarps) {
                    float t = 0.f;
                    for (int k = 0; k < kWarps; ++k) t += sums[k][i];
                    a.part[((size_t)blockIdx.x * 2 + z) * a.D + i] = t;
                }
            }
        }
    }
}

long long blocks_of(long long rows, int D, int sms, bool bwd)
{
    const long long n = D <= kWarpD ? (rows + kWarps - 1) / kWarps : rows;
    // backward: as many blocks as are resident, a partial row of both sums each
    const long long per = D <= kWarpD ? 2 : D <= 1024 ? 8 : D <= 2048 ? 4 : D <= 4096 ? 2 : 1;
    const long long most = bwd ? per * sms : D > 8192 ? sms : 0x7fffffff;
    return n < most ? n : most;
}

template <typename E, typename R, bool BWD>
cudaError_t launch_widest(const ResArgs& a, unsigned blocks, cudaStream_t s)
{
    constexpr int NTR = 512, K = 4, n = BWD ? 2 * K * 2 * NTR * (int)sizeof(ulonglong2) : 0;
    const cudaError_t r = cudaFuncSetAttribute(gla_residual_norm_kernel<E, R, NTR, K, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    if (r != cudaSuccess) return r;
    gla_residual_norm_kernel<E, R, NTR, K, BWD><<<blocks, NTR, n, s>>>(a);
    return cudaGetLastError();
}
template <typename E, typename R, bool BWD>
cudaError_t launch(const ResArgs& a, int sms, cudaStream_t s)
{
    const unsigned g = (unsigned)blocks_of(a.rows, a.D, sms, BWD);
    if (a.D <= 256) gla_residual_norm_kernel<E, R, 32, 1, BWD><<<g, 32 * kWarps, 0, s>>>(a);
    else if (a.D <= 512) gla_residual_norm_kernel<E, R, 32, 2, BWD><<<g, 32 * kWarps, 0, s>>>(a);
    else if (a.D <= 1024) gla_residual_norm_kernel<E, R, 64, 2, BWD><<<g, 64, 0, s>>>(a);
    else if (a.D <= 2048) gla_residual_norm_kernel<E, R, 128, 2, BWD><<<g, 128, 0, s>>>(a);
    else if (a.D <= 4096) gla_residual_norm_kernel<E, R, 256, 2, BWD><<<g, 256, 0, s>>>(a);
    else if (a.D <= 8192) gla_residual_norm_kernel<E, R, 512, 2, BWD><<<g, 512, 0, s>>>(a);
    else return launch_widest<E, R, BWD>(a, g, s);
    return cudaGetLastError();
}
template <bool BWD>
cudaError_t launch(const gla_residual_params* p, const ResArgs& a, int sms, cudaStream_t s)
{
    if (p->dtype == GLA_FP32) return launch<float, float, BWD>(a, sms, s);
    return p->residual_dtype == GLA_FP32 ? launch<__nv_bfloat16, float, BWD>(a, sms, s)
                                         : launch<__nv_bfloat16, __nv_bfloat16, BWD>(a, sms, s);
}

gla_status check(const gla_residual_params* p)
{
    if (!p || p->rows < 0 || p->D <= 0 || p->D % 16 != 0) return GLA_ERR_INVALID_ARG;
    if (p->dtype != GLA_BF16 && p->dtype != GLA_FP32) return GLA_ERR_INVALID_ARG;
    if (p->residual_dtype != GLA_FP32 && p->residual_dtype != p->dtype) return GLA_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !std::isfinite(p->eps) || !std::isfinite(p->alpha)) return GLA_ERR_INVALID_ARG;
    if (p->rows > 0 && !p->x) return GLA_ERR_INVALID_ARG;
    for (const void* x : {p->x, p->residual, (const void*)p->w, (const void*)p->scale})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (p->D > kMaxD || p->rows > (1LL << 40) / p->D) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

ResArgs common(const gla_residual_params* p)
{
    ResArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = p->x; a.r = p->residual; a.w = p->w; a.scale = p->scale;
    a.rows = p->rows; a.D = p->D; a.post = p->post_norm != 0; a.alpha = p->alpha; a.eps = p->eps;
    return a;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

gla_status gla_residual_norm(const gla_residual_params* p, void* h, void* y, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if ((p->rows > 0 && !y) || !aligned(h, 16) || !aligned(y, 16)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, er = p->residual_dtype == GLA_BF16 ? 2 : 4, n = (size_t)p->rows * p->D;
    const Span r = flat(p->residual, n * er), in[] = {flat(p->x, n * e), flat(p->w, p->D * 4), flat(p->scale, p->D * 4)};
    const Span ho = flat(h, n * er), yo = flat(y, n * e);
    for (const Span& s : in)
        if (overlap(ho, s) || overlap(yo, s)) return GLA_ERR_INVALID_ARG;
    if ((overlap(ho, r) && h != p->residual) || overlap(yo, r) || overlap(ho, yo)) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK || p->rows == 0) return st;
    ResArgs a = common(p);
    a.h = h; a.y = y;
    return launch<false>(p, a, sms, stream) == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

size_t gla_residual_norm_bwd_workspace_size(const gla_residual_params* p)
{
    int sms = 0;
    if (check(p) != GLA_OK || p->rows == 0 || (!p->w && !p->scale)) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    return (size_t)blocks_of(p->rows, p->D, sms, true) * 2 * p->D * 4;
}

gla_status gla_residual_norm_bwd(const gla_residual_params* p, const gla_residual_grads* g, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (!g || (g->grad_w && !p->w) || (g->grad_scale && !p->scale) || (g->grad_residual && !p->residual)) return GLA_ERR_INVALID_ARG;
    for (const void* x : {g->grad_h, g->grad_y, (const void*)g->grad_x, (const void*)g->grad_residual})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(g->grad_w, 4) || !aligned(g->grad_scale, 4) || !aligned(workspace, 256)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, er = p->residual_dtype == GLA_BF16 ? 2 : 4, n = (size_t)p->rows * p->D;
    const Span in[] = {flat(p->x, n * e), flat(p->residual, n * er), flat(p->w, p->D * 4), flat(p->scale, p->D * 4),
                       flat(g->grad_h, n * er), flat(g->grad_y, n * e)};
    const Span out[] = {flat(g->grad_x, n * e), flat(g->grad_residual, n * er), flat(g->grad_w, p->D * 4), flat(g->grad_scale, p->D * 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return GLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j])) return GLA_ERR_INVALID_ARG;
    }
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    cudaError_t r = cudaSuccess;
    if (p->rows == 0) {
        if (g->grad_w) r = cudaMemsetAsync(g->grad_w, 0, p->D * 4, stream);
        if (r == cudaSuccess && g->grad_scale) r = cudaMemsetAsync(g->grad_scale, 0, p->D * 4, stream);
        return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
    }
    const bool sums = g->grad_w || g->grad_scale;
    const long long blocks = blocks_of(p->rows, p->D, sms, true);
    if (sums && (!workspace || workspace_bytes < (size_t)blocks * 2 * p->D * 4)) return GLA_ERR_WORKSPACE;
    ResArgs a = common(p);
    a.dh = g->grad_h; a.dy = g->grad_y; a.dx = g->grad_x; a.dr = g->grad_residual;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    r = launch<true>(p, a, sms, stream);
    if (r == cudaSuccess && sums)
        r = launch_column_sum(a.part, blocks, 2LL * p->D, ColumnOuts{{{g->grad_w, p->D}, {g->grad_scale, p->D}}}, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
