// gla_conv_fwd: the short causal convolution of every channel c of a layer's rows, with the state that
// carries its last W - 1 inputs from call to call,
//
//     y_t = act(a_t),   a_t = bias + sum_j w_j x_{t-W+1+j},   x_{-(W-1)..-1} from S0 (or zero),
//
// act the identity or silu, and S_T the last W - 1 of (S0, x). Backward, with da_t = dy_t act'(a_t) and da_t = 0
// from T on:
//
//     dx_s = sum_j w_j da_{s+W-1-j} (+ dS_T where row s is in S_T; s < 0: dS0),   dw_j = sum da_t x_{t-W+1+j},
//     dbias = sum da_t.
//
// Bound by HBM: x read and y written once (backward: x and dy read, dx written). A thread takes eight
// channels (16 bytes in bf16; four in the backward, whose sums and windows fill the registers) and walks a run of tokens with
// the window in registers; a run's first W - 1 rows are read again, from L2. Reads go through strides (a
// projection's slice, head by head), writes are dense. Sums are fp32; S_T is a copy of inputs.
#include <cmath>
#include <cstring>

#include "gla_internal.h"
#include "gla_rows.cuh"
#include "gla_span.h"

namespace gla {
namespace {

constexpr int NT = 256;
constexpr int LANES = 32;                // lanes across channels
constexpr int RUNS = NT / LANES;         // runs of tokens per block
constexpr int UNR = 4;                   // rows in flight per thread

struct ConvArgs {
    const void* x; const float* w; const float* bias; const void* S0;
    void* y; void* ST;
    const void* dy; const void* dST; void* dx; void* dS0; float* part;
    long long sx[3], sdx[3];             // strides (b, h, t) in elements
    int B, H, T, d, D, silu;
    int run;                             // tokens per thread
    int tblocks;                         // blocks along the tokens
};

// V values of a row from p (zeros from nullptr), as loaded.
template <typename E, int V> struct Row;
template <> struct Row<__nv_bfloat16, 8> { uint4 u; };
template <> struct Row<float, 8> { float4 a, b; };
template <> struct Row<__nv_bfloat16, 4> { uint2 u; };
template <> struct Row<float, 4> { float4 a; };
__device__ __forceinline__ void get(Row<__nv_bfloat16, 8>& r, const __nv_bfloat16* p) { r.u = p ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void get(Row<__nv_bfloat16, 4>& r, const __nv_bfloat16* p) { r.u = p ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0); }
__device__ __forceinline__ void get(Row<float, 4>& r, const float* p) { r.a = p ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0); }
__device__ __forceinline__ void get(Row<float, 8>& r, const float* p) {
    r.a = p ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0);
    r.b = p ? *(reinterpret_cast<const float4*>(p) + 1) : make_float4(0, 0, 0, 0);
}
__device__ __forceinline__ void two(uint32_t u, float& a, float& b) { a = __uint_as_float(u << 16); b = __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ void open(const Row<__nv_bfloat16, 8>& r, float (&x)[8]) {
    two(r.u.x, x[0], x[1]); two(r.u.y, x[2], x[3]); two(r.u.z, x[4], x[5]); two(r.u.w, x[6], x[7]);
}
__device__ __forceinline__ void open(const Row<__nv_bfloat16, 4>& r, float (&x)[4]) { two(r.u.x, x[0], x[1]); two(r.u.y, x[2], x[3]); }
__device__ __forceinline__ void open(const Row<float, 4>& r, float (&x)[4]) { x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w; }
__device__ __forceinline__ void open(const Row<float, 8>& r, float (&x)[8]) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w; x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&x)[4]) { *reinterpret_cast<uint2*>(p) = make_uint2(pack(x[0], x[1]), pack(x[2], x[3])); }
__device__ __forceinline__ void put(float* p, const float (&x)[4]) { *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void put(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(x[4], x[5], x[6], x[7]);
}

// The thread's place: channels c.. of batch row b, tokens [t0, t1).
template <int V>
struct Place {
    int b, c, h, off, t0, t1;
    bool on, first;
    __device__ explicit Place(const ConvArgs& a)
    {
        const int lane = threadIdx.x % LANES, r = threadIdx.x / LANES;
        const unsigned q = blockIdx.x / a.tblocks;
        b = blockIdx.y + blockIdx.z * 65535;
        c = (q * LANES + lane) * V;
        const long long at = ((long long)(blockIdx.x % a.tblocks) * RUNS + r) * a.run;
        on = c < a.D && b < a.B && (at < a.T || at == 0);
        t0 = (int)(at < a.T ? at : 0);
        t1 = (int)(at + a.run < a.T ? at + a.run : a.T);
        first = at == 0;
        h = on ? c / a.d : 0;
        off = c - h * a.d;
    }
};

template <typename E, int W>
__global__ void __launch_bounds__(NT, 4) gla_conv_fwd_kernel(ConvArgs a)
{
    constexpr int V = 8;
    const Place<V> at(a);
    if (!at.on) return;
    float w[W][V], bias[V];
    {
        float f[W * V];
#pragma unroll
        for (int i = 0; i < W * V; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.w + (size_t)at.c * W + i));
            f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = f[v * W + j];
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = a.bias ? __ldg(a.bias + at.c + v) : 0.f;
    }
    const E* xp = static_cast<const E*>(a.x) + at.b * a.sx[0] + at.h * a.sx[1] + at.off;
    const E* s0 = a.S0 ? static_cast<const E*>(a.S0) + (size_t)at.b * (W - 1) * a.D + at.c : nullptr;
    E* yp = static_cast<E*>(a.y) + ((size_t)(at.b * a.H + at.h) * a.T + at.t0) * a.d + at.off;

    Row<E, V> win[W - 1];        // rows t - W + 1 .. t - 1
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int s = at.t0 - (W - 1) + i;
        get(win[i], s >= 0 ? xp + s * a.sx[2] : s0 ? s0 + (size_t)(s + W - 1) * a.D : nullptr);
    }
    if (at.first && a.ST) {
        // S_T may lie in S0's place: its rows are read above, by this thread alone
        Row<E, V> last[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int s = a.T - (W - 1) + i;
            if (s >= 0) {
                get(last[i], xp + s * a.sx[2]);
            } else {
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    if (s + W - 1 == k) last[i] = win[k];
            }
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            float f[V];
            open(last[i], f);
            put(static_cast<E*>(a.ST) + ((size_t)at.b * (W - 1) + i) * a.D + at.c, f);
        }
    }
    float x[W][V];               // x[j]: row t - W + 1 + j
#pragma unroll
    for (int i = 0; i < W - 1; ++i) open(win[i], x[i]);
    for (int t = at.t0; t < at.t1; t += UNR) {
        Row<E, V> in[UNR];
#pragma unroll
        for (int u = 0; u < UNR; ++u) get(in[u], t + u < at.t1 ? xp + (t + u) * a.sx[2] : nullptr);
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
            open(in[u], x[W - 1]);
            float y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                y[v] = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) y[v] = fmaf(w[j][v], x[j][v], y[v]);
                if (a.silu) y[v] *= sigmoid(y[v]);
            }
            if (t + u < at.t1) put(yp, y);
            yp += a.d;
#pragma unroll
            for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) x[j][v] = x[j + 1][v];
        }
    }
}

// The backward walks W - 1 tokens past its run: dx of the run's rows needs their da. Weight sums are its own run's.
template <typename E, int W>
__global__ void __launch_bounds__(NT, 2) gla_conv_bwd_kernel(ConvArgs a)
{
    constexpr int V = 4;
    __shared__ float red[RUNS][LANES * V * (W + 1)];
    const Place<V> at(a);
    float w[W][V], bias[V], dw[W + 1][V];
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
    if (at.on) {
        float f[W * V];
#pragma unroll
        for (int i = 0; i < W * V; i += 4) {
            const float4 q = __ldg(reinterpret_cast<const float4*>(a.w + (size_t)at.c * W + i));
            f[i] = q.x; f[i + 1] = q.y; f[i + 2] = q.z; f[i + 3] = q.w;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = f[v * W + j];
#pragma unroll
        for (int v = 0; v < V; ++v) bias[v] = a.bias ? __ldg(a.bias + at.c + v) : 0.f;
        const E* xp = static_cast<const E*>(a.x) + at.b * a.sx[0] + at.h * a.sx[1] + at.off;
        const E* s0 = a.S0 ? static_cast<const E*>(a.S0) + (size_t)at.b * (W - 1) * a.D + at.c : nullptr;
        const E* gp = static_cast<const E*>(a.dy) + (size_t)(at.b * a.H + at.h) * a.T * a.d + at.off;
        const E* dst = a.dST ? static_cast<const E*>(a.dST) + (size_t)at.b * (W - 1) * a.D + at.c : nullptr;
        E* dxp = static_cast<E*>(a.dx) + at.b * a.sdx[0] + at.h * a.sdx[1] + at.off;
        E* ds0 = a.dS0 ? static_cast<E*>(a.dS0) + (size_t)at.b * (W - 1) * a.D + at.c : nullptr;
        float x[W][V], da[W][V];     // x[j]: row t - W + 1 + j; da[j]: of row t - j
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int s = at.t0 - (W - 1) + i;
            Row<E, V> r;
            get(r, s >= 0 ? xp + s * a.sx[2] : s0 ? s0 + (size_t)(s + W - 1) * a.D : nullptr);
            open(r, x[i]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) da[j][v] = 0.f;
        const int end = at.t1 + W - 1;
        for (int t = at.t0; t < end; t += UNR) {
            Row<E, V> in[UNR], ing[UNR];
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                const bool ok = t + u < a.T && t + u < end;
                get(in[u], ok ? xp + (t + u) * a.sx[2] : nullptr);
                get(ing[u], ok ? gp + (size_t)(t + u) * a.d : nullptr);
            }
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                const int tt = t + u;
                open(in[u], x[W - 1]);
                float g[V];
                open(ing[u], g);             // (zero from T on)
#pragma unroll
                for (int j = W - 1; j > 0; --j)
#pragma unroll
                    for (int v = 0; v < V; ++v) da[j][v] = da[j - 1][v];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    da[0][v] = g[v];
                    if (a.silu) {
                        float z = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) z = fmaf(w[j][v], x[j][v], z);
                        const float s = sigmoid(z);
                        da[0][v] = g[v] * fmaf(z * s, 1.f - s, s);
                    }
                }
                if (tt < at.t1) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][v] = fmaf(da[0][v], x[j][v], dw[j][v]);
                        dw[W][v] += da[0][v];
                    }
                }
                const int s = tt - (W - 1);
                if (tt < end && (s >= at.t0 || (at.first && s < 0))) {
                    float o[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        o[v] = 0.f;
#pragma unroll
                        for (int j = 0; j < W; ++j) o[v] = fmaf(w[j][v], da[j][v], o[v]);
                    }
                    const int k = s - a.T + W - 1;
                    if (dst && k >= 0) {
                        Row<E, V> r;
                        float f[V];
                        get(r, dst + (size_t)k * a.D);
                        open(r, f);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += f[v];
                    }
                    if (s >= 0) put(dxp + s * a.sdx[2], o);
                    else if (ds0) put(ds0 + (size_t)(s + W - 1) * a.D, o);
                }
#pragma unroll
                for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) x[j][v] = x[j + 1][v];
            }
        }
    }
    if (!a.part) return;
    // over the block's runs, in order; a block leaves [D][W] of dw, then [D] of dbias
    const int lane = threadIdx.x % LANES, r = threadIdx.x / LANES;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j <= W; ++j) red[r][(v * (W + 1) + j) * LANES + lane] = dw[j][v];
    __syncthreads();
    const int cols = (W + 1) * a.D, c0 = (blockIdx.x / a.tblocks) * LANES * V;
    const long long blk = (long long)(blockIdx.y + blockIdx.z * 65535) * a.tblocks + blockIdx.x % a.tblocks;
    for (int i = threadIdx.x; i < LANES * V * (W + 1); i += NT) {
        const int ch = i / (W + 1), j = i % (W + 1);
        if (c0 + ch >= a.D || blockIdx.y + blockIdx.z * 65535 >= (unsigned)a.B) continue;
        float s = 0.f;
        for (int k = 0; k < RUNS; ++k) s += red[k][(ch % V * (W + 1) + j) * LANES + ch / V];
        a.part[blk * cols + (j < W ? (c0 + ch) * W + j : a.D * W + c0 + ch)] = s;
    }
}

// Tokens per thread: long runs read fewer rows twice and leave fewer partials, short ones fill the chip.
dim3 grid_of(ConvArgs& a, int V, int sms, bool bwd)
{
    const long long ct = (a.D + LANES * V - 1) / (LANES * V);
    int run = bwd ? 64 : 32;
    while (run > UNR && ct * a.B * ((a.T + (long long)run * RUNS - 1) / ((long long)run * RUNS)) < 4LL * sms) run /= 2;
    a.run = run;
    const long long tb = (a.T + (long long)run * RUNS - 1) / ((long long)run * RUNS);
    a.tblocks = (int)(tb > 1 ? tb : 1);
    return dim3((unsigned)(ct * a.tblocks), a.B < 65535 ? a.B : 65535, (a.B + 65534) / 65535);
}

template <typename E, int W>
cudaError_t launch(ConvArgs a, int sms, bool bwd, cudaStream_t s)
{
    const dim3 g = grid_of(a, bwd ? 4 : 8, sms, bwd);
    if (bwd) gla_conv_bwd_kernel<E, W><<<g, NT, 0, s>>>(a);
    else gla_conv_fwd_kernel<E, W><<<g, NT, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename E>
cudaError_t launch(const ConvArgs& a, int W, int sms, bool bwd, cudaStream_t s)
{
    return W == 2 ? launch<E, 2>(a, sms, bwd, s) : W == 3 ? launch<E, 3>(a, sms, bwd, s) : launch<E, 4>(a, sms, bwd, s);
}

gla_status check(const gla_conv_params* p)
{
    if (!p || p->B <= 0 || p->H <= 0 || p->T < 0 || p->d <= 0) return GLA_ERR_INVALID_ARG;
    if (p->d % 16 != 0 || (p->dtype != GLA_BF16 && p->dtype != GLA_FP32)) return GLA_ERR_INVALID_ARG;
    if (p->activation != GLA_ACT_NONE && p->activation != GLA_ACT_SILU) return GLA_ERR_INVALID_ARG;
    if (p->W < 1 || !p->w || (p->T > 0 && !p->x)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (const long long s : p->x_stride)
        if (s * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;   // every row starts on 16 bytes
    for (const void* x : {p->x, (const void*)p->w, p->S0})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(p->bias, 4)) return GLA_ERR_INVALID_ARG;
    if (p->W < 2 || p->W > 4 || (long long)p->H * p->d > (1 << 24) || p->T > (1 << 30)) return GLA_ERR_UNSUPPORTED;
    if ((long long)p->B * p->T > (1LL << 40) / ((long long)p->H * p->d)) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

ConvArgs common(const gla_conv_params* p)
{
    ConvArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = p->x; a.w = p->w; a.bias = p->bias; a.S0 = p->S0;
    for (int i = 0; i < 3; ++i) a.sx[i] = p->x_stride[i];
    a.B = p->B; a.H = p->H; a.T = p->T; a.d = p->d; a.D = p->H * p->d;
    a.silu = p->activation == GLA_ACT_SILU;
    return a;
}

size_t part_bytes(const gla_conv_params* p, int sms, long long* blocks)
{
    ConvArgs a = common(p);
    grid_of(a, 4, sms, true);
    *blocks = (long long)a.tblocks * p->B;
    return (size_t)*blocks * a.D * (p->W + 1) * 4;
}

struct Sizes { size_t dense, state, w, bias; };
Sizes sizes_of(const gla_conv_params* p)
{
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, D = (size_t)p->H * p->d;
    return Sizes{(size_t)p->B * p->T * D * e, (size_t)p->B * (p->W - 1) * D * e, D * p->W * 4, D * 4};
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

gla_status gla_conv_fwd(const gla_conv_params* p, void* y, void* ST, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if ((p->T > 0 && !y) || !aligned(y, 16) || !aligned(ST, 16)) return GLA_ERR_INVALID_ARG;
    const Sizes n = sizes_of(p);
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    const Span x = span(p->x, p->x_stride, p->B, p->H, p->T, p->d, e), s0 = flat(p->S0, n.state);
    const Span in[] = {x, s0, flat(p->w, n.w), flat(p->bias, n.bias)};
    const Span out = flat(y, n.dense), so = flat(ST, n.state);
    for (const Span& s : in) {
        if (overlap(out, s)) return GLA_ERR_INVALID_ARG;
        if (overlap(so, s) && ST != p->S0) return GLA_ERR_INVALID_ARG;
    }
    if (overlap(out, so) || (ST == p->S0 && overlap(so, x))) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK || (p->T == 0 && (!ST || ST == p->S0))) return st;
    ConvArgs a = common(p);
    a.y = y; a.ST = ST;
    const cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16>(a, p->W, sms, false, stream)
                                               : launch<float>(a, p->W, sms, false, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

size_t gla_conv_bwd_workspace_size(const gla_conv_params* p)
{
    int sms = 0;
    long long blocks;
    if (check(p) != GLA_OK) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    return part_bytes(p, sms, &blocks);
}

gla_status gla_conv_bwd(const gla_conv_params* p, const gla_conv_grads* g, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (!g || (p->T > 0 && (!g->grad_y || !g->grad_x))) return GLA_ERR_INVALID_ARG;
    if (g->grad_bias && !p->bias) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (const long long s : g->x_stride)
        if (s * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;
    for (const void* x : {g->grad_y, g->grad_ST, (const void*)g->grad_x, (const void*)g->grad_S0})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(g->grad_w, 4) || !aligned(g->grad_bias, 4) || !aligned(workspace, 256)) return GLA_ERR_INVALID_ARG;
    const Sizes n = sizes_of(p);
    const Span in[] = {span(p->x, p->x_stride, p->B, p->H, p->T, p->d, e), flat(p->S0, n.state), flat(p->w, n.w),
                       flat(p->bias, n.bias), flat(g->grad_y, n.dense), flat(g->grad_ST, n.state)};
    const Span out[] = {span(g->grad_x, g->x_stride, p->B, p->H, p->T, p->d, e), flat(g->grad_S0, n.state),
                        flat(g->grad_w, n.w), flat(g->grad_bias, n.bias)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return GLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlap(out[i], out[j])) return GLA_ERR_INVALID_ARG;
    }
    if (p->T > 0 && !apart(g->x_stride, p->B, p->H, p->T, p->d)) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    const bool sums = g->grad_w || g->grad_bias;
    long long blocks = 0;
    const size_t need = part_bytes(p, sms, &blocks);
    if (sums && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
    ConvArgs a = common(p);
    a.dy = g->grad_y; a.dST = g->grad_ST; a.dx = g->grad_x; a.dS0 = g->grad_S0;
    for (int i = 0; i < 3; ++i) a.sdx[i] = g->x_stride[i];
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16>(a, p->W, sms, true, stream)
                                         : launch<float>(a, p->W, sms, true, stream);
    if (r == cudaSuccess && sums)
        r = launch_column_sum(a.part, blocks, a.D * (p->W + 1), ColumnOuts{{{g->grad_w, (long long)a.D * p->W}, {g->grad_bias, a.D}}}, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
