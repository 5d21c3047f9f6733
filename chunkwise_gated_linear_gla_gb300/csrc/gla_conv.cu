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
// Bytes: x read and y written once (backward: x and dy read, dx written). A thread takes four channels of a row (with eight
// the weights and windows do not fit the registers: 69 us for the layer below, 33 then), two in the backward, whose sums and
// windows are twice as many (75 us then, 85 with four), and walks a run of tokens with the window in registers; a run's first W - 1
// rows are read again, from L2. A warp is 128 (64) channels of a run of one batch row, a block eight warps, runs of all rows in one
// order, so that single tokens of many rows fill it too (128 rows of 4096 channels 5.5 us, 16 with a block to a row). Reads go through
// strides (a projection's slice, head by head), writes are dense. Sums are fp32; S_T is a copy of inputs. 8 x 2048 tokens of
// 2048 channels: 25.5 us, 5.3 TB/s, 0.78 of the copy rate; backward 61 us, 0.49 (eight rows are loaded, then computed with none in flight; bf16
// spills 92 bytes at its 80 registers), and 5 for the sums of the weights' partials.
#include <cmath>
#include <cstring>
#include <type_traits>

#include "gla_internal.h"
#include "gla_rows.cuh"
#include "gla_span.h"

namespace gla {
namespace {

constexpr int NT = 256;
constexpr int LANES = 32;                // lanes across channels
constexpr int RUNS = NT / LANES;         // runs of tokens per block
constexpr int kFwdPairs = 2, kBwdPairs = 1;    // pairs of channels per thread
constexpr int UNR = 4;                   // rows in flight per thread; long runs take eight

struct ConvArgs {
    const void* x; const float* w; const float* bias; const void* S0;
    void* y; void* ST;
    const void* dy; const void* dST; void* dx; void* dS0; float* part;
    long long sx[3], sdx[3];             // strides (b, h, t) in elements
    int B, H, T, d, D, silu;
    int run, runs;                       // tokens of a run, runs of a batch row
    int ctiles;                          // channel tiles
};

// P pairs of values of a row from p (zeros from nullptr), as loaded, and as pairs.
template <typename E, int P> struct Row { uint32_t u[P * sizeof(E) / 2]; };
template <typename E, int P>
__device__ __forceinline__ void get(Row<E, P>& r, const E* p)
{
    constexpr int WORDS = P * sizeof(E) / 2;
    if constexpr (WORDS == 1) {
        r.u[0] = p ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    } else if constexpr (WORDS == 2) {
        const uint2 q = p ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
        r.u[0] = q.x; r.u[1] = q.y;
    } else {
        const uint4 q = p ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
        r.u[0] = q.x; r.u[1] = q.y; r.u[2] = q.z; r.u[3] = q.w;
    }
}
template <int P>
__device__ __forceinline__ void open(const Row<__nv_bfloat16, P>& r, f2 (&x)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = pk(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xffff0000u));
}
template <int P>
__device__ __forceinline__ void open(const Row<float, P>& r, f2 (&x)[P])
{
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = pk(__uint_as_float(r.u[2 * i]), __uint_as_float(r.u[2 * i + 1]));
}
template <int P>
__device__ __forceinline__ void put(__nv_bfloat16* p, const f2 (&x)[P])
{
    if constexpr (P == 1) *reinterpret_cast<uint32_t*>(p) = bf16x2(x[0]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(bf16x2(x[0]), bf16x2(x[1]));
}
template <int P>
__device__ __forceinline__ void put(float* p, const f2 (&x)[P])
{
    if constexpr (P == 1) *reinterpret_cast<f2*>(p) = x[0];
    else *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x[0], x[1]);
}

// The thread's channels c .., from the block's channel tile.
template <int P>
struct Channels {
    int c, h, off;
    bool in;
    __device__ explicit Channels(const ConvArgs& a)
    {
        c = ((int)(blockIdx.x % a.ctiles) * LANES + threadIdx.x % LANES) * 2 * P;
        in = c < a.D;
        h = in ? c / a.d : 0;
        off = in ? c - h * a.d : 0;
    }
};
// A warp's run: tokens [t0, t1) of batch row b, the r-th of all.
struct Run {
    int b, t0, t1;
    bool on, first;
    __device__ Run(const ConvArgs& a, long long r)
    {
        on = r < (long long)a.B * a.runs;
        const long long q = on ? r : 0;
        b = (int)(q / a.runs);
        t0 = (int)(q - (long long)b * a.runs) * a.run;
        first = t0 == 0;
        t1 = a.T - t0 < a.run ? a.T : t0 + a.run;
    }
};
// W weights of each of the thread's channels, and its bias.
template <int W, int P>
__device__ __forceinline__ void weights(const ConvArgs& a, const Channels<P>& ch, f2 (&w)[W][P], f2 (&bias)[P])
{
    float f[W * 2 * P];
#pragma unroll
    for (int i = 0; i < W * 2 * P; i += 2 * P) {             // (2 P channels' weights start on 8 P bytes)
        const float* q = a.w + (size_t)ch.c * W + i;
        if constexpr (P == 2) {
            const float4 v = ch.in ? __ldg(reinterpret_cast<const float4*>(q)) : make_float4(0, 0, 0, 0);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        } else {
            const float2 v = ch.in ? __ldg(reinterpret_cast<const float2*>(q)) : make_float2(0, 0);
            f[i] = v.x; f[i + 1] = v.y;
        }
    }
#pragma unroll
    for (int v = 0; v < P; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = pk(f[2 * v * W + j], f[(2 * v + 1) * W + j]);
        bias[v] = a.bias && ch.in ? pk(__ldg(a.bias + ch.c + 2 * v), __ldg(a.bias + ch.c + 2 * v + 1)) : 0ull;
    }
}

template <typename E, int W, int UNR>
__global__ void __launch_bounds__(NT, UNR > 4 && sizeof(E) > 2 ? 3 : 4) gla_conv_fwd_kernel(ConvArgs a)
{
    constexpr int P = kFwdPairs;
    const Channels<P> ch(a);
    const Run at(a, (long long)(blockIdx.x / a.ctiles) * RUNS + threadIdx.x / LANES);
    if (!ch.in || !at.on) return;
    f2 w[W][P], bias[P];
    weights<W>(a, ch, w, bias);
    const E* xp = static_cast<const E*>(a.x) + at.b * a.sx[0] + ch.h * a.sx[1] + ch.off;
    const E* s0 = a.S0 ? static_cast<const E*>(a.S0) + (size_t)at.b * (W - 1) * a.D + ch.c : nullptr;
    E* yp = static_cast<E*>(a.y) + ((size_t)(at.b * (long long)a.H + ch.h) * a.T + at.t0) * a.d + ch.off;

    Row<E, P> win[W - 1];        // rows t - W + 1 .. t - 1
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int s = at.t0 - (W - 1) + i;
        get(win[i], s >= 0 ? xp + s * a.sx[2] : s0 ? s0 + (size_t)(s + W - 1) * a.D : nullptr);
    }
    if (at.first && a.ST) {
        // S_T may lie in S0's place: its rows are read above, by this thread alone
        Row<E, P> last[W - 1];
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
            f2 f[P];
            open(last[i], f);
            put(static_cast<E*>(a.ST) + ((size_t)at.b * (W - 1) + i) * a.D + ch.c, f);
        }
    }
    f2 x[W][P];                  // x[j]: row t - W + 1 + j
#pragma unroll
    for (int i = 0; i < W - 1; ++i) open(win[i], x[i]);
    const E* in_p = xp + at.t0 * a.sx[2];
    for (int t = at.t0; t < at.t1; t += UNR) {
        Row<E, P> in[UNR];
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
            get(in[u], t + u < at.t1 ? in_p : nullptr);
            in_p += a.sx[2];
        }
#pragma unroll
        for (int u = 0; u < UNR; ++u) {
            open(in[u], x[W - 1]);
            f2 y[P];
#pragma unroll
            for (int v = 0; v < P; ++v) {
                y[v] = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) y[v] = fma2(w[j][v], x[j][v], y[v]);
                if (a.silu) y[v] = mul2(y[v], sig(y[v]));
            }
            if (t + u < at.t1) put(yp, y);
            yp += a.d;
#pragma unroll
            for (int j = 0; j + 1 < W; ++j)
#pragma unroll
                for (int v = 0; v < P; ++v) x[j][v] = x[j + 1][v];
        }
    }
}

// The backward walks W - 1 tokens past its run: dx of the run's rows needs their da. Weight sums are its own run's. A block
// takes several groups of runs, so that it leaves one partial sum of them all.
template <typename E, int W, int UNR>
__global__ void __launch_bounds__(NT, UNR > 4 && sizeof(E) > 2 ? 2 : 3) gla_conv_bwd_kernel(ConvArgs a)
{
    constexpr int P = kBwdPairs, V = 2 * P;
    __shared__ float red[RUNS][LANES * V * (W + 1)];
    const Channels<P> ch(a);
    const int groups = gridDim.x / a.ctiles;
    const long long all = (long long)a.B * a.runs;
    f2 w[W][P], bias[P], dw[W + 1][P];
    weights<W>(a, ch, w, bias);
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < P; ++v) dw[j][v] = 0ull;
    for (long long r0 = (long long)(blockIdx.x / a.ctiles) * RUNS; r0 < all; r0 += (long long)groups * RUNS) {
        const Run at(a, r0 + threadIdx.x / LANES);
        if (!at.on || !ch.in) break;
        const E* xp = static_cast<const E*>(a.x) + at.b * a.sx[0] + ch.h * a.sx[1] + ch.off;
        const E* s0 = a.S0 ? static_cast<const E*>(a.S0) + (size_t)at.b * (W - 1) * a.D + ch.c : nullptr;
        const E* gp = static_cast<const E*>(a.dy) + ((size_t)(at.b * (long long)a.H + ch.h) * a.T + at.t0) * a.d + ch.off;
        f2 x[W][P], da[W][P];        // x[j]: row t - W + 1 + j; da[j]: of row t - j
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int s = at.t0 - (W - 1) + i;
            Row<E, P> r;
            get(r, s >= 0 ? xp + s * a.sx[2] : s0 ? s0 + (size_t)(s + W - 1) * a.D : nullptr);
            open(r, x[i]);
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < P; ++v) da[j][v] = 0ull;
        const int end = at.t1 + W - 1;
        xp += at.t0 * a.sx[2];
        E* out = static_cast<E*>(a.dx) + at.b * a.sdx[0] + ch.h * a.sdx[1] + ch.off + (at.t0 - (W - 1)) * a.sdx[2];   // of row t - W + 1
        // UNR tokens from t; INSIDE: all are the run's own and their rows of dx the run's
        auto tokens = [&](int t, auto inside) {
            constexpr bool INSIDE = decltype(inside)::value;
            Row<E, P> in[UNR], ing[UNR];
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                const bool given = INSIDE || (t + u < a.T && t + u < end);
                get(in[u], given ? xp : nullptr);
                get(ing[u], given ? gp : nullptr);           // (zeros from T on)
                xp += a.sx[2];
                gp += a.d;
            }
#pragma unroll
            for (int u = 0; u < UNR; ++u) {
                const int tt = t + u;
                f2 g[P], o[P];
                open(in[u], x[W - 1]);
                open(ing[u], g);
#pragma unroll
                for (int v = 0; v < P; ++v) {
#pragma unroll
                    for (int j = W - 1; j > 0; --j) da[j][v] = da[j - 1][v];
                    da[0][v] = g[v];
                    if (a.silu) {
                        f2 z = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) z = fma2(w[j][v], x[j][v], z);
                        const f2 s = sig(z);
                        da[0][v] = mul2(g[v], fma2(mul2(z, s), fma2(s, both(-1.f), both(1.f)), s));
                    }
                    if (INSIDE || tt < at.t1) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][v] = fma2(da[0][v], x[j][v], dw[j][v]);
                        dw[W][v] = add2(dw[W][v], da[0][v]);
                    }
                    o[v] = mul2(w[0][v], da[0][v]);
#pragma unroll
                    for (int j = 1; j < W; ++j) o[v] = fma2(w[j][v], da[j][v], o[v]);
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) x[j][v] = x[j + 1][v];
                }
                if constexpr (INSIDE) {
                    put(out, o);
                } else {
                    const int s = tt - (W - 1);
                    if (tt < end && (s >= at.t0 || (at.first && s < 0))) {
                        if (a.dST && tt >= a.T) {
                            Row<E, P> r;
                            f2 f[P];
                            get(r, static_cast<const E*>(a.dST) + ((size_t)at.b * (W - 1) + tt - a.T) * a.D + ch.c);
                            open(r, f);
#pragma unroll
                            for (int v = 0; v < P; ++v) o[v] = add2(o[v], f[v]);
                        }
                        if (s >= 0) put(out, o);
                        else if (a.dS0) put(static_cast<E*>(a.dS0) + ((size_t)at.b * (W - 1) + tt) * a.D + ch.c, o);
                    }
                }
                out += a.sdx[2];
            }
        };
#pragma unroll 1
        for (int t = at.t0; t < end; t += UNR) {
            if (t >= at.t0 + W - 1 && t + UNR <= at.t1) tokens(t, std::true_type());
            else tokens(t, std::false_type());
        }
    }
    if (!a.part) return;
    // over the block's warps, in order; a block leaves [D][W] of dw, then [D] of dbias
    const int lane = threadIdx.x % LANES, r = threadIdx.x / LANES;
#pragma unroll
    for (int v = 0; v < P; ++v)
#pragma unroll
        for (int j = 0; j <= W; ++j) up(dw[j][v], red[r][(2 * v * (W + 1) + j) * LANES + lane], red[r][((2 * v + 1) * (W + 1) + j) * LANES + lane]);
    __syncthreads();
    const int c0 = (int)(blockIdx.x % a.ctiles) * LANES * V;
    float* part = a.part + (size_t)(blockIdx.x / a.ctiles) * (W + 1) * a.D;
    for (int i = threadIdx.x; i < LANES * V * (W + 1); i += NT) {
        const int c = i / (W + 1), j = i % (W + 1);
        if (c0 + c >= a.D) continue;
        float s = 0.f;
        for (int k = 0; k < RUNS; ++k) s += red[k][(c % V * (W + 1) + j) * LANES + c / V];
        part[j < W ? (c0 + c) * W + j : a.D * W + c0 + c] = s;
    }
}

// Tokens per run, and the groups of runs (the blocks of a channel tile). Long runs read fewer rows twice, short ones fill the chip;
// blocks come in rounds of as many as are resident, and the run is the one whose rounds end first, a run of
// its tokens and a few more that start and end it. Backward a block takes its rounds' groups one after the other, for few partials
// (8 x 2048 tokens of 2048 channels: 75 us with 64 tokens in three rounds, 63 so; fp32 82 and 77; forward 32.7 with 16 in four, 25.6 so).
// Forward in fp32 it is bytes, and runs above 32 tokens lose a little (two taps: 42 us, 45 with more).
int grid_of(ConvArgs& a, int sms, bool bwd, bool fp32)
{
    const int V = 2 * (bwd ? kBwdPairs : kFwdPairs);
    a.ctiles = (a.D + LANES * V - 1) / (LANES * V);
    auto groups_of = [&](int run) {
        const long long runs = ((long long)a.T + run - 1) / run;
        a.run = run;
        a.runs = (int)(runs > 1 ? runs : 1);
        return ((long long)a.B * a.runs + RUNS - 1) / RUNS;
    };
    long long best = 0, cost = -1;
    int at = UNR;
    for (int run = UNR; run <= (fp32 && !bwd ? 32 : 128); run += run < 8 ? 4 : 8) {
        const long long sm = bwd ? (fp32 && run > 16 ? 2 : 3) : fp32 && run > 8 ? 3 : 4;
        const long long groups = groups_of(run);
        long long rounds;
        if (bwd) {
            const long long most = sm * sms / a.ctiles > 1 ? sm * sms / a.ctiles : 1;
            rounds = (groups + most - 1) / most;
        } else {
            rounds = (groups * a.ctiles + sm * sms - 1) / (sm * sms);
        }
        const long long c = rounds * (run + (bwd ? 6 : 4)) * sm;
        if (cost < 0 || c < cost) { cost = c; at = run; best = bwd ? (groups + rounds - 1) / rounds : groups; }
    }
    groups_of(at);
    return (int)best;
}

template <typename E, int W>
cudaError_t launch(ConvArgs a, int sms, bool bwd, cudaStream_t s)
{
    const unsigned g = (unsigned)((long long)grid_of(a, sms, bwd, sizeof(E) > 2) * a.ctiles);
    if (bwd && a.run > 16) gla_conv_bwd_kernel<E, W, 2 * UNR><<<g, NT, 0, s>>>(a);  // (fp32, the layer: 99 us with four)
    else if (bwd) gla_conv_bwd_kernel<E, W, UNR><<<g, NT, 0, s>>>(a);               // (3 x 777 tokens of 1040 channels: 18 us with eight, 15)
    else if (a.run > 8) gla_conv_fwd_kernel<E, W, 2 * UNR><<<g, NT, 0, s>>>(a);     // (the layer: 35 us with four)
    else gla_conv_fwd_kernel<E, W, UNR><<<g, NT, 0, s>>>(a);                        // (128 single tokens: 6.6 us with eight, 5.5)
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
    *blocks = grid_of(a, sms, true, p->dtype == GLA_FP32);
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
