// gla_qk_norm_rope: the rows of q and k of every head on their way to an attention call, in one
// pass: x -> R(pos) (w (.) x / n(x)), n the 2-norm sqrt(sum x^2 + eps) or the root mean square
// sqrt(mean x^2 + eps), R the rotation of the first `rot` values by the row's position. Backward,
// with z = R^T dy, x^ = x / n and N = 1 (2-norm) or d (root mean square):
//
//     dw = sum over rows of z (.) x^,    dx = (z (.) w - x^ (sum z (.) w (.) x^) / N) / n.
//
// Bound by HBM: every row is read once and written once (backward: x and dy read, dx written); the
// rows of 8 x 2048 tokens, 16 + 16 heads of 128 bf16 values take 47 us forward, 5.7 TB/s, 0.84 of the
// measured copy rate, caches cold, with four blocks of 64 registers a thread per SM (three of 80: 54 us).
// A row is LPR lanes of eight values (16 bytes in bf16); a thread keeps its row of the batch and
// takes that token's heads one after the other, so a token's angles are formed once per block
// (in shared memory) and four heads' loads are in flight at a time. Reads go through strides (a fused projection's
// [B,T,heads,d] slice), writes are dense [B,H,T,d].
//
// Angles: the caller's frequencies are radians per position in fp64. Each becomes a fraction of
// a turn in 2^-64 units, so position * frequency modulo one turn is one wrapping 64-bit product
// without rounding (fp32 products lose the angle beyond a few thousand positions, and fp64
// ones cost the few fp64 units this chip has); the remaining fraction goes to sincospi in fp32.
// What the fraction itself was rounded by, 2^-52 of it and half a unit, grows with the position: at
// most |pos f| 2^-52 + |pos| 2^-62 radians, below the fp32 rounding up to pos f = 2^28.
//
// The weights' gradients are summed in fp32: over a thread's rows, over the block in shared
// memory, over the blocks by a second kernel, each in a fixed order.
#include <cuda_bf16.h>
#include <cmath>
#include <cstring>
#include <utility>

#include "gla_internal.h"

namespace gla {
namespace {

constexpr int NT = 256;
constexpr int VEC = 8;        // values per lane
constexpr int UNR = 4;        // heads in flight per thread; the backward takes one at a time
constexpr long long kBlocksPerSm = 4;

struct QkArgs {
    const void* x[2]; void* y[2];                 // q, k (strided) and their results (dense)
    const void* dy[2]; void* dx[2]; float* part;  // backward: dense gradients in, strided out
    long long sx[2][3], sdx[2][3];                // strides (b, h, t) in elements
    const float* w[2];
    const double* inv_freq; const long long* positions; long long start;
    int heads[2];
    int B, T, d, rot, interleaved, norm;
    float eps;
    int hsplit;                                   // heads (q's and k's in a row) per block
};

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

// f radians per position as a fraction of a turn in units of 2^-64 (modulo one turn).
__device__ __forceinline__ unsigned long long turn_units(double f)
{
    const double x = f * 0.15915494309189533577;   // 1 / (2 pi)
    const unsigned long long bits = (unsigned long long)__double_as_longlong(x);
    const int e = (int)((bits >> 52) & 0x7ff);
    if (e == 0 || e == 0x7ff) return 0ull;          // zero, subnormal, not finite: no turn
    const unsigned long long m = (bits & 0xfffffffffffffull) | (1ull << 52);
    const int sh = e - 1075 + 64;                   // x = m 2^(e - 1075)
    unsigned long long u;
    if (sh >= 0) u = sh < 64 ? m << sh : 0ull;
    else u = sh > -54 ? (m + (1ull << (-sh - 1))) >> -sh : 0ull;
    return (bits >> 63) ? 0ull - u : u;
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}

// The rotation of this lane's eight values. Neighbouring pairs lie in the lane; halves pair value
// i with i + rot / 2, `hop` lanes on. The sines carry the sign that their place wants (and the
// transpose's), lanes past `rot` have cosine one and sine zero.
template <int LPR>
__device__ __forceinline__ void rotate(float (&x)[VEC], const float (&cs)[VEC], const float (&sn)[VEC], int from,
                                       int interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
            const float a = x[j], b = x[j + 1], s = sn[j / 2];
            x[j] = fmaf(a, cs[j / 2], -b * s);
            x[j + 1] = fmaf(b, cs[j / 2], a * s);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const float m = __shfl_sync(~0u, x[j], from, LPR);
        x[j] = fmaf(x[j], cs[j], sn[j] * m);
    }
}

// One block: NT / LPR tokens by hsplit heads. BWD: dy, x -> dx and the weights' partials.
template <typename E, int LPR, bool BWD>
__global__ void __launch_bounds__(NT, BWD ? 3 : 4) gla_qk_norm_rope_kernel(QkArgs a)
{
    constexpr int RPB = NT / LPR, U = BWD ? 1 : UNR;
    __shared__ unsigned long long turns[LPR * VEC / 2];
    // cosines and sines of the block's tokens; the weights' sums take their place at the end
    __shared__ __align__(16) float trig[2][RPB][LPR * VEC / 2];
    float* red = &trig[0][0][0];
    static_assert(!BWD || sizeof(trig) >= NT * VEC * 4, "weights' sums");
    const int l = threadIdx.x % LPR, lo = l * VEC, row = threadIdx.x / LPR;
    const long long ntok = (long long)a.B * a.T;
    const bool lane_in = lo < a.d;
    for (int i = threadIdx.x; i < a.rot / 2; i += NT) turns[i] = turn_units(a.inv_freq[i]);
    __syncthreads();

    // this block's heads of q (z = 0) and of k (z = 1)
    const int h0 = blockIdx.y * a.hsplit, h1 = min(a.heads[0] + a.heads[1], h0 + a.hsplit);
    float dw[2][VEC];
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[z][j] = 0.f;
    const float invn = a.norm == GLA_NORM_RMS ? 1.f / (float)a.d : 1.f;

    for (long long t0 = (long long)blockIdx.x * RPB; t0 < ntok; t0 += (long long)gridDim.x * RPB) {
        const long long tok = t0 + row;
        const bool on = lane_in && tok < ntok;
        const long long tk = tok < ntok ? tok : ntok - 1;
        const long long b = ntok <= 0x7fffffff ? (unsigned)tk / (unsigned)a.T : tk / a.T, t = tk - b * a.T;
        float cs[VEC], sn[VEC];
        if (a.rot) {
            // one angle per token and pair, shared by the row's lanes (a pair's halves lie in two)
            const int half = a.rot / 2;
            __syncthreads();
            for (int i = threadIdx.x; i < RPB * half; i += NT) {
                const int rr = i / half, p = i - rr * half;
                const long long tt = min(t0 + rr, ntok - 1);
                const unsigned long long pos =
                    (unsigned long long)(a.positions ? a.positions[tt] : a.start + (ntok <= 0x7fffffff ? (unsigned)tt % (unsigned)a.T : tt % a.T));
                const int top = (int)(unsigned)((pos * turns[p]) >> 32);
                sincospif((float)top * 4.6566128730773926e-10f, &trig[1][rr][p], &trig[0][rr][p]);   // 2^-31: half turns
            }
            __syncthreads();
            const bool turned = lo < a.rot, low = lo < half;
            const int first = !turned ? 0 : a.interleaved ? lo / 2 : low ? lo : lo - half;
            const float sg = (a.interleaved || !low) != BWD ? 1.f : -1.f;
#pragma unroll
            for (int j = 0; j < VEC; j += 4) {
                if (a.interleaved && j >= VEC / 2) break;
                const float4 c4 = *reinterpret_cast<const float4*>(&trig[0][row][first + j]);
                const float4 s4 = *reinterpret_cast<const float4*>(&trig[1][row][first + j]);
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    cs[j + e] = turned ? c[e] : 1.f;
                    sn[j + e] = turned ? sg * s[e] : 0.f;
                }
            }
        }
        const int hop = a.rot / (2 * VEC);
        const int from = lo < a.rot / 2 ? l + hop : lo < a.rot ? l - hop : l;   // the lane of the pairs' other halves
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int hb0 = max(0, h0 - (z ? a.heads[0] : 0)), hb1 = min(a.heads[z], h1 - (z ? a.heads[0] : 0));
            if (hb0 >= hb1) continue;
            float w[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) w[j] = a.w[z] && lane_in ? a.w[z][lo + j] : 1.f;
            const E* xp = static_cast<const E*>(a.x[z]) + b * a.sx[z][0] + hb0 * a.sx[z][1] + t * a.sx[z][2] + lo;
            const long long hstep = (long long)a.T * a.d, dense = ((b * a.heads[z] + hb0) * a.T + t) * a.d + lo;
            E* yp = BWD ? static_cast<E*>(a.dx[z]) + b * a.sdx[z][0] + hb0 * a.sdx[z][1] + t * a.sdx[z][2] + lo
                        : static_cast<E*>(a.y[z]) + dense;
            const E* gp = BWD ? static_cast<const E*>(a.dy[z]) + dense : nullptr;
            const long long xstep = a.sx[z][1], ystep = BWD ? a.sdx[z][1] : hstep;
            auto one = [&](const typename Raw<E>::type& xr, const typename Raw<E>::type& gr, E* out) {
                float x[VEC];
                unpack(xr, x);
                float inv = 1.f;
                if (a.norm != GLA_NORM_NONE) {
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) s = fmaf(x[j], x[j], s);
                    inv = rsqrtf(fmaf(row_sum<LPR>(s), invn, a.eps));
                    if (BWD && !on) inv = 0.f;      // rows past the last token hold zeros: with eps = 0, 1 / 0
                }
                if constexpr (!BWD) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[j] *= inv * w[j];
                    if (a.rot) rotate<LPR>(x, cs, sn, from, a.interleaved);
                    if (on) save8(out, x);
                } else {
                    float g[VEC];
                    unpack(gr, g);
                    if (a.rot) rotate<LPR>(g, cs, sn, from, a.interleaved);
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        x[j] *= inv;                                    // x^
                        dw[z][j] = fmaf(g[j], x[j], dw[z][j]);          // (rows past the last token: x^ = 0)
                        g[j] *= w[j];
                        s = fmaf(g[j], x[j], s);
                    }
                    if (a.norm != GLA_NORM_NONE) {
                        s = row_sum<LPR>(s) * invn;
#pragma unroll
                        for (int j = 0; j < VEC; ++j) g[j] = inv * fmaf(-x[j], s, g[j]);
                    }
                    if (on) save8(out, g);
                }
            };
            for (int hb = hb0; hb < hb1; hb += U) {
                typename Raw<E>::type xr[U], gr[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool ok = hb + u < hb1 && on;
                    xr[u] = fetch(ok ? xp + u * xstep : nullptr);
                    if constexpr (BWD) gr[u] = fetch(ok ? gp + u * hstep : nullptr);
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (hb + u < hb1) one(xr[u], gr[u], yp + u * ystep);
                xp += U * xstep;
                yp += U * ystep;
                if constexpr (BWD) gp += U * hstep;
            }
        }
    }
    if constexpr (BWD) {
        if (a.part) {
            const size_t blk = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                __syncthreads();
#pragma unroll
                for (int j = 0; j < VEC; ++j) red[row * (LPR * VEC) + lo + j] = dw[z][j];
                __syncthreads();
                for (int i = threadIdx.x; i < a.d; i += NT) {
                    float s = 0.f;
                    for (int k = 0; k < RPB; ++k) s += red[k * (LPR * VEC) + i];
                    a.part[(blk * 2 + z) * a.d + i] = s;
                }
            }
        }
    }
}

// dw[z][i]: the blocks' partials, 32 at a time per column, then over the 32.
__global__ void __launch_bounds__(1024) gla_qk_weight_sum_kernel(const float* part, int blocks, int d, float* dq, float* dk)
{
    __shared__ float red[32][33];
    const int z = blockIdx.y, i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (i < d)
        for (int b = threadIdx.y; b < blocks; b += 32) s += part[((size_t)b * 2 + z) * d + i];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    float* out = z ? dk : dq;
    if (threadIdx.y == 0 && i < d && out) {
        s = 0.f;
        for (int k = 0; k < 32; ++k) s += red[k][threadIdx.x];
        out[i] = s;
    }
}

dim3 grid_of(const QkArgs& a, int lpr, int sms, bool bwd, int* hsplit)
{
    const long long rows = NT / lpr, tg = ((long long)a.B * a.T + rows - 1) / rows;
    const int nh = a.heads[0] + a.heads[1];
    // The heads are spread over blocks (each forms the token's angles again) until every SM has its
    // four: more blocks pay the set-up more often (the layer's rows, 8 x 2048 tokens of 32 heads of 128
    // values: 47 us so, 60 with four times as many blocks).
    int split = 1;
    while (split < nh && tg * split < kBlocksPerSm * sms) split *= 2;
    if (split > nh) split = nh;
    *hsplit = (nh + split - 1) / split;
    const int gy = (nh + *hsplit - 1) / *hsplit;
    long long gx = tg;
    const long long most = bwd ? kBlocksPerSm * sms : 1LL << 30;   // backward: few blocks, few partials
    if (gx > most) gx = most;
    return dim3((unsigned)gx, gy);
}

template <typename E, bool BWD>
cudaError_t launch(QkArgs a, int sms, cudaStream_t s)
{
    const int lpr = a.d <= 64 ? 8 : a.d <= 128 ? 16 : 32;
    const dim3 g = grid_of(a, lpr, sms, BWD, &a.hsplit);
    if (lpr == 8) gla_qk_norm_rope_kernel<E, 8, BWD><<<g, NT, 0, s>>>(a);
    else if (lpr == 16) gla_qk_norm_rope_kernel<E, 16, BWD><<<g, NT, 0, s>>>(a);
    else gla_qk_norm_rope_kernel<E, 32, BWD><<<g, NT, 0, s>>>(a);
    return cudaGetLastError();
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Sizes, modes and presence shared by both directions.
gla_status check(const gla_qk_norm_params* p)
{
    if (!p || p->B <= 0 || p->T < 0 || p->H <= 0 || p->Hk < 0 || p->d <= 0) return GLA_ERR_INVALID_ARG;
    if (p->d % 16 != 0 || p->rot < 0 || p->rot % 16 != 0 || p->rot > p->d) return GLA_ERR_INVALID_ARG;
    if (p->dtype != GLA_BF16 && p->dtype != GLA_FP32) return GLA_ERR_INVALID_ARG;
    if (p->norm != GLA_NORM_NONE && p->norm != GLA_NORM_L2 && p->norm != GLA_NORM_RMS) return GLA_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return GLA_ERR_INVALID_ARG;
    if ((p->rot > 0) != (p->inv_freq != nullptr)) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!p->q || (p->Hk > 0 && !p->k))) return GLA_ERR_INVALID_ARG;
    if ((long long)p->B * p->T > (1LL << 40) || (long long)p->H + p->Hk > 65535) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4;
    for (const long long s : {p->q_stride[0], p->q_stride[1], p->q_stride[2], p->k_stride[0], p->k_stride[1], p->k_stride[2]})
        if (s * (long long)e % 16 != 0) return GLA_ERR_INVALID_ARG;   // every row starts on 16 bytes
    for (const void* x : {p->q, p->k, (const void*)p->w_q, (const void*)p->w_k})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(p->inv_freq, 8) || !aligned(p->positions, 8)) return GLA_ERR_INVALID_ARG;
    if (p->d > 256) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

// The bytes a strided [B,H,T,d] tensor spans (strides may be zero or negative).
struct Span { uintptr_t lo, hi; };
Span span(const void* p, const long long* st, int B, int H, int T, int d, size_t e)
{
    if (!p || B <= 0 || H <= 0 || T <= 0) return Span{0, 0};
    long long lo = 0, hi = d;
    const long long n[3] = {B - 1LL, H - 1LL, T - 1LL};
    for (int i = 0; i < 3; ++i) (st[i] < 0 ? lo : hi) += st[i] * n[i];
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a + (uintptr_t)(lo * (long long)e), a + (uintptr_t)(hi * (long long)e)};
}
Span flat(const void* p, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p ? Span{a, a + bytes} : Span{0, 0};
}
bool overlap(Span a, Span b) { return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi; }

// Whether the rows of a strided output are apart: dimension by dimension, from the smallest
// stride, each steps past everything that the ones before it cover.
bool apart(const long long* st, int B, int H, int T, int d)
{
    long long n[3] = {B, H, T}, s[3];
    for (int i = 0; i < 3; ++i) s[i] = st[i] < 0 ? -st[i] : st[i];
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) { std::swap(s[i], s[j]); std::swap(n[i], n[j]); }
    long long cover = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < cover) return false;
        cover += s[i] * (n[i] - 1);
    }
    return true;
}

QkArgs common(const gla_qk_norm_params* p)
{
    QkArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x[0] = p->q; a.x[1] = p->k;
    for (int i = 0; i < 3; ++i) { a.sx[0][i] = p->q_stride[i]; a.sx[1][i] = p->k_stride[i]; }
    a.w[0] = p->w_q; a.w[1] = p->w_k;
    a.inv_freq = p->inv_freq; a.positions = p->positions; a.start = p->start;
    a.heads[0] = p->H; a.heads[1] = p->Hk;
    a.B = p->B; a.T = p->T; a.d = p->d; a.rot = p->rot; a.interleaved = p->interleaved != 0; a.norm = p->norm;
    a.eps = p->eps;
    return a;
}

// Backward partials: blocks of the grid times two rows of d values.
size_t part_bytes(const gla_qk_norm_params* p, int sms, int* blocks)
{
    QkArgs a = common(p);
    int hs;
    const dim3 g = grid_of(a, p->d <= 64 ? 8 : p->d <= 128 ? 16 : 32, sms, true, &hs);
    *blocks = (int)(g.x * g.y);
    return (size_t)*blocks * 2 * p->d * 4;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

gla_status gla_qk_norm_rope(const gla_qk_norm_params* p, void* q_out, void* k_out, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (p->T > 0 && (!q_out || (p->Hk > 0 && !k_out))) return GLA_ERR_INVALID_ARG;
    if (!aligned(q_out, 16) || !aligned(k_out, 16)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, row = (size_t)p->B * p->T * p->d * e;
    const Span in[] = {span(p->q, p->q_stride, p->B, p->H, p->T, p->d, e),
                       span(p->k, p->k_stride, p->B, p->Hk, p->T, p->d, e), flat(p->w_q, p->d * 4),
                       flat(p->w_k, p->d * 4), flat(p->inv_freq, p->rot * 4),
                       flat(p->positions, (size_t)p->B * p->T * 8)};
    const Span q = flat(q_out, row * p->H), k = flat(k_out, row * p->Hk);
    for (const Span& s : in)
        if (overlap(q, s) || overlap(k, s)) return GLA_ERR_INVALID_ARG;
    if (overlap(q, k)) return GLA_ERR_INVALID_ARG;
    int sms = 0;
    st = device_ready(&sms);
    if (st != GLA_OK || p->T == 0) return st;
    QkArgs a = common(p);
    a.y[0] = q_out; a.y[1] = k_out;
    const cudaError_t r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16, false>(a, sms, stream)
                                               : launch<float, false>(a, sms, stream);
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

size_t gla_qk_norm_rope_bwd_workspace_size(const gla_qk_norm_params* p)
{
    int sms = 0, blocks;
    if (check(p) != GLA_OK || p->T == 0 || (!p->w_q && !p->w_k)) return 0;
    if (device_ready(&sms) != GLA_OK) sms = 152;
    return part_bytes(p, sms, &blocks);
}

gla_status gla_qk_norm_rope_bwd(const gla_qk_norm_params* p, const gla_qk_norm_grads* g, void* workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    gla_status st = check(p);
    if (st != GLA_OK) return st;
    if (!g) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!g->grad_q_out || !g->grad_q || (p->Hk > 0 && (!g->grad_k_out || !g->grad_k))))
        return GLA_ERR_INVALID_ARG;
    if ((g->grad_w_q && !p->w_q) || (g->grad_w_k && !p->w_k)) return GLA_ERR_INVALID_ARG;
    const size_t e = p->dtype == GLA_BF16 ? 2 : 4, row = (size_t)p->B * p->T * p->d * e;
    for (int i = 0; i < 3; ++i)
        if (g->q_stride[i] * (long long)e % 16 != 0 || g->k_stride[i] * (long long)e % 16 != 0)
            return GLA_ERR_INVALID_ARG;
    for (const void* x : {g->grad_q_out, g->grad_k_out, (const void*)g->grad_q, (const void*)g->grad_k})
        if (!aligned(x, 16)) return GLA_ERR_INVALID_ARG;
    if (!aligned(g->grad_w_q, 4) || !aligned(g->grad_w_k, 4) || !aligned(workspace, 256)) return GLA_ERR_INVALID_ARG;
    const Span in[] = {span(p->q, p->q_stride, p->B, p->H, p->T, p->d, e),
                       span(p->k, p->k_stride, p->B, p->Hk, p->T, p->d, e), flat(p->w_q, p->d * 4),
                       flat(p->w_k, p->d * 4), flat(p->inv_freq, p->rot * 4),
                       flat(p->positions, (size_t)p->B * p->T * 8), flat(g->grad_q_out, row * p->H),
                       flat(g->grad_k_out, row * p->Hk)};
    // grad_q and grad_k may be interleaved slices of one tensor (their rows apart): only equal
    // starts are refused between them
    const Span out[] = {span(g->grad_q, g->q_stride, p->B, p->H, p->T, p->d, e),
                        span(g->grad_k, g->k_stride, p->B, p->Hk, p->T, p->d, e), flat(g->grad_w_q, p->d * 4),
                        flat(g->grad_w_k, p->d * 4)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return GLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (!(i == 0 && j == 1) && overlap(out[i], out[j])) return GLA_ERR_INVALID_ARG;
    }
    if (p->T > 0 && g->grad_q == g->grad_k) return GLA_ERR_INVALID_ARG;
    if (p->T > 0 && (!apart(g->q_stride, p->B, p->H, p->T, p->d) ||
                     (p->Hk > 0 && !apart(g->k_stride, p->B, p->Hk, p->T, p->d))))
        return GLA_ERR_INVALID_ARG;
    int sms = 0, blocks = 0;
    st = device_ready(&sms);
    if (st != GLA_OK) return st;
    cudaError_t r = cudaSuccess;
    const bool dw = g->grad_w_q || g->grad_w_k;
    if (p->T == 0) {
        if (g->grad_w_q) r = cudaMemsetAsync(g->grad_w_q, 0, p->d * 4, stream);
        if (r == cudaSuccess && g->grad_w_k) r = cudaMemsetAsync(g->grad_w_k, 0, p->d * 4, stream);
        return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
    }
    const size_t need = dw ? part_bytes(p, sms, &blocks) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GLA_ERR_WORKSPACE;
    QkArgs a = common(p);
    a.dy[0] = g->grad_q_out; a.dy[1] = g->grad_k_out;
    a.dx[0] = g->grad_q; a.dx[1] = g->grad_k;
    for (int i = 0; i < 3; ++i) { a.sdx[0][i] = g->q_stride[i]; a.sdx[1][i] = g->k_stride[i]; }
    a.part = dw ? static_cast<float*>(workspace) : nullptr;
    r = p->dtype == GLA_BF16 ? launch<__nv_bfloat16, true>(a, sms, stream) : launch<float, true>(a, sms, stream);
    if (r == cudaSuccess && dw) {
        gla_qk_weight_sum_kernel<<<dim3((p->d + 31) / 32, 2), dim3(32, 32), 0, stream>>>(
            a.part, blocks, p->d, g->grad_w_q, g->grad_w_k);
        r = cudaGetLastError();
    }
    return r == cudaSuccess ? GLA_OK : GLA_ERR_CUDA;
}

}  // extern "C"
