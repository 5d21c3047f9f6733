// The selective scan: N states for each of the D channels, with a decay per channel, state and token,
//
//     delta_t = softplus(dt_t + dt_bias),   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
//     y_t = (C_t . h_t + D x_t) silu(z_t).
//
// No product of matrices is in it: per token, channel and state one exponential, two products and two fused
// multiply-adds, all fp32, the states in registers from the first token to the last.
//
// gla_ssm_walk: a thread holds eight states of a channel and walks the tokens, its products packed pairs of states. The block goes
// in tiles of 32 tokens (16 where they would take too much room): raw rows arrive by asynchronous copies one tile ahead, delta and
// delta x are formed once per channel and token into shared memory, B and C widened there, the walk leaves C . h in their places, and y
// is formed from it eight channels at a time. Bound by waits, no pipe is full: eight rows of 2048 tokens of 4096 channels of 16 states (1.07e9 of
// them, 0.54 GB) take 389 us at 7.7 warp instructions a state, with 61% of the issue slots taken (70% on the schedulers that got four warps, not
// three), 54% of the shared-memory path, 47% of the multiply-adds' pipe and 38% of the exponentials'; a tile's preparing and finishing overlap
// other blocks' walks only. The bytes would take 80, the exponentials 107. Two blocks of two warps measured better than one of four (by 3%).
//
// Few channels: the sequence is cut into segments. A first walk leaves each segment's state from zero and its sum of delta
// (the decay across the segment is exp(A sum)), gla_ssm_scan the states entering them, a second walk y (one row of 16421
// tokens: 213 + 14 + 341 us in 23 segments).
//
// gla_ssm_step: single and few tokens: a thread holds four states of a channel, of four batch rows where there are many. The next token of 128
// rows of 4096 channels takes 17 us with cold caches (4.2 TB/s) and 14 call after call, when part of the states is still in L2: bound by the
// states' latency and, with 67% of the issue slots taken, by instructions, as each of a channel's lanes forms its step and gate again.
#include "gla_ssm.cuh"

namespace gla {
namespace {

// ------------------------------------------------------------------ few tokens

template <typename E> __device__ __forceinline__ float one(const E* p) { return (float)*p; }
__device__ __forceinline__ void four(const __nv_bfloat16* p, float (&v)[4])
{
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void four(const float* p, float (&v)[4])
{
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}

constexpr int kStepNT = 128;

// ROWS batch rows of a channel's four states per thread: their loads are in flight together, A and the channel's parameters
// are read once for all.
template <typename E, int N, int ROWS>
__global__ void __launch_bounds__(kStepNT) gla_ssm_step_kernel(SsmArgs a)
{
    constexpr int LPC = N / 4, CPB = kStepNT / LPC;
    const int ctiles = (a.D + CPB - 1) / CPB;
    const int b0 = (int)(blockIdx.x / ctiles) * ROWS;
    const int c = (int)(blockIdx.x % ctiles) * CPB + threadIdx.x / LPC, l = threadIdx.x % LPC, n = l * 4;
    const bool on = c < a.D;
    const int cc = on ? c : a.D - 1, g = cc / (a.D / a.G);
    const size_t per = (size_t)a.D * N, so = (size_t)cc * N + n;
    float h[ROWS][4], A[4];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        if (a.S0 && b0 + u < a.B) four(a.S0 + (b0 + u) * per + so, h[u]);
        else h[u][0] = h[u][1] = h[u][2] = h[u][3] = 0.f;
    }
    four(a.A + so, A);
    const float bias = a.bias ? a.bias[cc] : 0.f, Dk = a.Dk ? a.Dk[cc] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] *= kLog2e;
    for (int t = 0; t < a.T; ++t) {
        float x[ROWS], d[ROWS], z[ROWS], Bv[ROWS][4], Cv[ROWS][4];
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const long long b = b0 + u < a.B ? b0 + u : b0;
            x[u] = one(static_cast<const E*>(a.x) + b * a.sx[0] + t * a.sx[1] + cc);
            d[u] = one(static_cast<const E*>(a.dt) + b * a.sdt[0] + t * a.sdt[1] + cc) + bias;
            z[u] = a.z ? one(static_cast<const E*>(a.z) + b * a.sz[0] + t * a.sz[1] + cc) : 0.f;
            four(static_cast<const E*>(a.Bm) + b * a.sB[0] + t * a.sB[1] + g * N + n, Bv[u]);
            four(static_cast<const E*>(a.Cm) + b * a.sC[0] + t * a.sC[1] + g * N + n, Cv[u]);
        }
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            if (a.softplus) d[u] = softplus(d[u]);
            const float dx = d[u] * x[u];
            float y = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[u][j] = fmaf(ex2(d[u] * A[j]), h[u][j], dx * Bv[u][j]);
                y = fmaf(h[u][j], Cv[u][j], y);
            }
            y = row_sum<LPC>(y);
            y = fmaf(Dk, x[u], y);
            if (a.z) y *= z[u] * sig(z[u]);
            if (on && l == 0 && b0 + u < a.B) static_cast<E*>(a.y)[((size_t)(b0 + u) * a.T + t) * a.D + cc] = (E)y;
        }
    }
    if (!on || !a.ST) return;
#pragma unroll
    for (int u = 0; u < ROWS; ++u)
        if (b0 + u < a.B) *reinterpret_cast<float4*>(a.ST + (b0 + u) * per + so) = make_float4(h[u][0], h[u][1], h[u][2], h[u][3]);
}

// ------------------------------------------------------------------ the walk

// Tokens per tile of loads: two of the kept states' tiles, or one where the rows of so many channels would leave an SM half its blocks
// (8 x 2048 tokens of 8192 channels of 8 states: 566 us with 32, 485 with 16, fp32 716 and 632; 4096 of 16 390 and 403, fp32 477 and
// 411; 2048 of 32 402 and 442, fp32 482 and 461 but of half the rows 257 and 293).
template <typename E, int N> constexpr int kWalkTile = N == 8 || (N == 16 && sizeof(E) == 4) ? 16 : 32;
constexpr int kS = 8;              // states of a thread: B and C are read once for them
template <int N> constexpr int kWalkWarps = N >= 64 ? 4 : 2;
template <int N> constexpr int kWalkChannels = kWalkWarps<N> * 32 * kS / N;

// A thread's states of a channel, from the first of them on: by fours N / 2 apart, so that neighbouring lanes read neighbouring 16
// bytes.
template <int N>
__device__ __forceinline__ void pick(const float* p, f2 (&r)[kS / 2])
{
#pragma unroll
    for (int i = 0; i < kS / 4; ++i) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p + i * (N / 2));
        r[2 * i] = q.x;
        r[2 * i + 1] = q.y;
    }
}
template <int N>
__device__ __forceinline__ void drop(float* p, const f2 (&r)[kS / 2])
{
#pragma unroll
    for (int i = 0; i < kS / 4; ++i) *reinterpret_cast<ulonglong2*>(p + i * (N / 2)) = make_ulonglong2(r[2 * i], r[2 * i + 1]);
}

template <typename E, int N, int MODE>
struct WalkShared {
    static constexpr int CB = kWalkChannels<N>, TT = kWalkTile<E, N>;
    static constexpr bool HAS_B = MODE != kSsmRev, HAS_C = MODE == kSsmOut || MODE == kSsmRev, HAS_Z = HAS_C;
    E raw[2][HAS_Z ? 3 : 2][TT][CB];   // x, dt, z (REV: dy, dt, z)
    E bc[2][HAS_B + HAS_C][TT][N];
    float wide[HAS_B + HAS_C][TT][N];  // B, C of the tile in fp32
    // delta, delta x (REV: dy silu(z)); a token's places take the two halves of its C . h once it has been walked
    // (rows four values further on each time, the second half 64 bytes: no store meets a bank twice)
    static constexpr int P = CB + 4;
    float work[2][TT * P + 16];
};

template <typename E, int N, int MODE>
__global__ void __launch_bounds__(kWalkWarps<N> * 32, MODE == kSsmOut ? 14 / kWalkWarps<N> : 1) gla_ssm_walk_kernel(SsmArgs a)
{
    typedef WalkShared<E, N, MODE> Shared;
    constexpr int NT = kWalkWarps<N> * 32, CB = kWalkChannels<N>, P = Shared::P, Q = N / kS, TT = kWalkTile<E, N>, SUB = kSsmTile;
    constexpr bool REV = MODE == kSsmRev, OUT = MODE == kSsmOut;
    constexpr int IC = Shared::HAS_B ? 1 : 0;      // where C lies beside B
    extern __shared__ __align__(16) char smem_raw[];
    auto& sm = *reinterpret_cast<Shared*>(smem_raw);
    const int Dg = a.D / a.G, ct = blockIdx.x % a.ctiles;
    const long long bg = blockIdx.x / a.ctiles;
    const int b = (int)(bg / a.G), g = (int)(bg % a.G);
    const int c0 = g * Dg + ct * CB, c1 = g * Dg + Dg;           // this block's channels end at c1
    const int seg = blockIdx.y + (REV ? 1 : 0), s0 = seg * a.seg, s1 = min(a.T, s0 + a.seg);
    const int tiles = (s1 - s0 + TT - 1) / TT, first = REV ? s0 + (tiles - 1) * TT : s0;

    const E* const zp = a.z && Shared::HAS_Z ? static_cast<const E*>(a.z) + b * a.sz[0] + c0 : nullptr;
    TileCopy<E, TT, CB, NT> cx, cd, cz;
    TileCopy<E, TT, N, NT> cB, cC;
    if (REV) cx.start(static_cast<const E*>(a.dy) + (size_t)b * a.T * a.D + c0, a.D, first, c1 - c0);
    else cx.start(static_cast<const E*>(a.x) + b * a.sx[0] + c0, a.sx[1], first, c1 - c0);
    cd.start(static_cast<const E*>(a.dt) + b * a.sdt[0] + c0, a.sdt[1], first, c1 - c0);
    if (zp) cz.start(zp, a.sz[1], first, c1 - c0);
    if (Shared::HAS_B) cB.start(static_cast<const E*>(a.Bm) + b * a.sB[0] + g * N, a.sB[1], first, N);
    if (Shared::HAS_C) cC.start(static_cast<const E*>(a.Cm) + b * a.sC[0] + g * N, a.sC[1], first, N);
    auto load = [&](int stage) {
        constexpr int step = REV ? -TT : TT;
        cx.go(&sm.raw[stage][0][0][0], s1, step);
        cd.go(&sm.raw[stage][1][0][0], s1, step);
        if (zp) cz.go(&sm.raw[stage][Shared::HAS_Z ? 2 : 0][0][0], s1, step);
        if (Shared::HAS_B) cB.go(&sm.bc[stage][0][0][0], s1, step);
        if (Shared::HAS_C) cC.go(&sm.bc[stage][IC][0][0], s1, step);
        copies_end();
    };
    load(0);

    // this thread's channel and eight states
    const int sg = threadIdx.x % Q, cl = threadIdx.x / Q;
    const bool on = c0 + cl < c1;
    f2 h[kS / 2], A[kS / 2];
    const size_t per = (size_t)a.D * N, so = (size_t)(on ? c0 + cl : c0) * N + sg * 4;
    const float* from = nullptr;          // this batch row's states, [D][N]
    if (REV) {
        if (seg == a.nseg - 1 && a.dST) from = a.dST + b * per;
    } else if (MODE != kSsmState || seg == 0) {
        if (seg > 0) from = a.segS + ((size_t)b * (a.nseg - 1) + seg - 1) * per;
        else if (a.S0) from = a.S0 + b * per;
    }
    pick<N>(a.A + so, A);
#pragma unroll
    for (int j = 0; j < kS / 2; ++j) {
        A[j] = mul2(A[j], both(kLog2e));
        h[j] = 0ull;
    }
    if (from) pick<N>(from + so, h);
    // the vectors of eight channels that this thread prepares and finishes: always the same channels
    constexpr int COLS = CB / VEC, VPT = TT * COLS;
    const int vc = threadIdx.x % COLS * VEC;
    const bool vin = c0 + vc < c1;
    f2 bias[4], Dk[4], sumd[4];
    params8(a.bias ? a.bias + c0 + vc : nullptr, vin, bias);
    params8(OUT && a.Dk ? a.Dk + c0 + vc : nullptr, vin, Dk);
#pragma unroll
    for (int j = 0; j < 4; ++j) sumd[j] = 0ull;

    for (int tile = 0; tile < tiles; ++tile) {
        const int stage = tile & 1, t0 = s0 + (REV ? tiles - 1 - tile : tile) * TT;
        copies_wait<0>();
        __syncthreads();
        if (tile + 1 < tiles) load(stage ^ 1);
#pragma unroll 2
        for (int i = threadIdx.x; i < (Shared::HAS_B + Shared::HAS_C) * TT * N / 4; i += NT) {
            f2 v[2];
            states<4>(&sm.bc[stage][0][0][0] + i * 4, v);
            *reinterpret_cast<ulonglong2*>(&sm.wide[0][0][0] + i * 4) = make_ulonglong2(v[0], v[1]);
        }
        for (int i = threadIdx.x; i < VPT; i += NT) {
            const int tok = i / COLS;
            f2 x[4], d[4], z[4];
            states<8>(&sm.raw[stage][0][tok][vc], x);
            states<8>(&sm.raw[stage][1][tok][vc], d);
            const bool ok = t0 + tok < s1;
            if (REV && zp) states<8>(&sm.raw[stage][Shared::HAS_Z ? 2 : 0][tok][vc], z);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = add2(d[j], bias[j]);
                if (a.softplus) d[j] = softplus(d[j]);
                if (!ok) d[j] = 0ull;
                if (MODE == kSsmState) sumd[j] = add2(sumd[j], d[j]);
                if (REV) {
                    if (zp) x[j] = mul2(x[j], mul2(z[j], sig(z[j])));
                } else {
                    x[j] = mul2(x[j], d[j]);
                }
            }
            keep8(&sm.work[0][tok * P + vc], d);
            keep8(&sm.work[1][tok * P + vc], x);
        }
        __syncthreads();
        // (a segment's last tile may hold one of the two parts)
        const int parts = t0 + SUB < s1 ? TT : SUB;
#pragma unroll 1
        for (int sub = REV ? TT - parts : 0; sub < (REV ? TT : parts); sub += SUB) {
            const int base = REV ? TT - SUB - sub : sub;
            if (MODE == kSsmKeep && on)
                drop<N>(a.keep + ((size_t)b * ((a.T + SUB - 1) / SUB) + (t0 + base) / SUB) * per + so, h);
            // At the end of these tokens the state that entered takes their whole decay at once, so that a long memory is rounded once
            // per 16 tokens, not at every one. Beside the states runs what they multiply it by, the product of the decays; where the states
            // between are not wanted, only what the tokens themselves add (from zero).
            f2 in[kS / 2], beside[kS / 2];
            float sd = 0.f;
#pragma unroll
            for (int j = 0; j < kS / 2; ++j) {
                in[j] = h[j];
                beside[j] = 0ull;
            }
            // A token in three steps, so that no wait for shared memory or an exponential is seen: its operands are fetched two
            // tokens ahead, its decays and inputs formed one ahead.
            struct Token { float d, x; f2 B[kS / 2], C[kS / 2], e[kS / 2], u[kS / 2]; };
            auto fetch = [&](int n, Token& p) {
                const int tok = base + (REV ? SUB - 1 - n : n);
                p.d = sm.work[0][tok * P + cl];
                p.x = sm.work[1][tok * P + cl];
                pick<N>(&sm.wide[0][tok][sg * 4], p.B);
                if (OUT) pick<N>(&sm.wide[IC][tok][sg * 4], p.C);
            };
            auto form = [&](Token& p) {
                sd += p.d;
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    p.e[j] = ex2_2(mul2(both(p.d), A[j]));
                    p.u[j] = mul2(both(p.x), p.B[j]);
                    if (REV) p.u[j] = mul2(p.e[j], p.u[j]);
                }
            };
            auto use = [&](int n, const Token& p) {
                f2 s = 0ull;
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    if (OUT) {
                        h[j] = fma2(p.e[j], h[j], p.u[j]);
                        beside[j] = n ? mul2(beside[j], p.e[j]) : p.e[j];
                    } else {
                        beside[j] = n ? fma2(p.e[j], beside[j], p.u[j]) : p.u[j];
                    }
                    if (OUT) s = fma2(h[j], p.C[j], s);
                }
                if (OUT) {
                    // into the places of the token's delta and delta x, which all of the channel's threads (of this warp) have read
                    float v = sum2(s);
#pragma unroll
                    for (int o = 2; o < Q; o *= 2) v += __shfl_xor_sync(~0u, v, o);
                    __syncwarp();
                    if (Q <= 2 || sg < 2) sm.work[sg & 1][(base + n) * P + cl] = v;
                }
            };
            Token p[3];
            fetch(0, p[0]);
            fetch(1, p[1]);
            form(p[0]);
#pragma unroll
            for (int n = 0; n < SUB; ++n) {
                if (n + 2 < SUB) fetch(n + 2, p[(n + 2) % 3]);
                if (n + 1 < SUB) form(p[(n + 1) % 3]);
                use(n, p[n % 3]);
            }
#pragma unroll
            for (int j = 0; j < kS / 2; ++j) {
                const f2 e = ex2_2(mul2(both(sd), A[j]));
                h[j] = OUT ? fma2(fma2(beside[j], both(-1.f), e), in[j], h[j]) : fma2(e, in[j], beside[j]);
            }
        }
        if (!OUT) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < VPT; i += NT) {
            const int tok = i / COLS;
            if (t0 + tok >= s1 || !vin) continue;
            f2 y[4], v[4], z[4];
            states<8>(&sm.raw[stage][0][tok][vc], y);
            if (zp) states<8>(&sm.raw[stage][Shared::HAS_Z ? 2 : 0][tok][vc], z);
#pragma unroll
            for (int q = 0; q < (Q < 2 ? 1 : 2); ++q) {
                f2 u[4];
                states<8>(&sm.work[q][tok * P + vc], u);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = q ? add2(v[j], u[j]) : u[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                y[j] = fma2(Dk[j], y[j], v[j]);
                if (zp) y[j] = mul2(y[j], mul2(z[j], sig(z[j])));
            }
            keep8(static_cast<E*>(a.y) + ((size_t)b * a.T + t0 + tok) * a.D + c0 + vc, y);
        }
    }

    float* to = nullptr;
    if (OUT && seg == a.nseg - 1 && a.ST) to = a.ST + b * per;
    if (MODE == kSsmState) to = a.segS + ((size_t)b * (a.nseg - 1) + seg) * per;
    if (REV) to = a.segG + ((size_t)b * (a.nseg - 1) + seg - 1) * per;
    if (to && on) drop<N>(to + so, h);
    if (MODE == kSsmState) {
        // the sums of delta over the threads that prepared the same channels, in order
        __syncthreads();
        float* sums = &sm.work[0][0];
        constexpr int ROWS = (NT < VPT ? NT : VPT) / COLS;
        if (threadIdx.x < ROWS * COLS) keep8(sums + threadIdx.x / COLS * CB + vc, sumd);
        __syncthreads();
        for (int c = threadIdx.x; c < CB; c += NT) {
            float s = 0.f;
            for (int r = 0; r < ROWS; ++r) s += sums[r * CB + c];
            if (c0 + c < c1) a.sumd[((size_t)b * (a.nseg - 1) + seg) * a.D + c0 + c] = s;
        }
    }
}

// 2^p x + o for large p, that of a long segment of states that grow: in two steps, as 2^p may be no fp32 number where 2^p x is
// one. No state stays none.
__device__ __forceinline__ float grow(float p, float x, float o)
{
    const float e = ex2(0.5f * p);
    return x == 0.f ? o : fmaf(e, e * x, o);
}

// The states entering segments 1 .., in place of the segments' own: the first's own starts from S0, X_{s+1} = exp(A sum_s) X_s
// + own_s. rev: the gradients of the states after segments .. nseg - 2, in place of what each next segment leaves of its
// own (the last one's starts from dST).
__global__ void gla_ssm_scan_kernel(SsmArgs a, int rev)
{
    const long long per = (long long)a.D * a.N, all = (long long)a.B * per;
    const int m = a.nseg - 1;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (long long)gridDim.x * blockDim.x) {
        const long long b = i / per, o = i - b * per;
        const float A = a.A[o] * kLog2e;
        const float* sd = a.sumd + b * m * a.D + o / a.N;
        float* s = (rev ? a.segG : a.segS) + b * m * per + o;
        float X = s[rev ? (m - 1) * per : 0];
        // (a step's sum and state are read before the one before it is stored, whose place the compiler cannot tell apart)
        auto at = [&](int k) { return rev ? m - 1 - k : k; };
        float p = 0.f, own = 0.f;
        auto read = [&](int k) {
            p = A * sd[(long long)(rev ? at(k) + 1 : at(k)) * a.D];
            own = s[at(k) * per];
        };
        if (m > 1) read(1);
        for (int k = 1; k < m; ++k) {
            X = p < 64.f ? fmaf(ex2(p), X, own) : grow(p, X, own);
            if (k + 1 < m) read(k + 1);
            s[at(k) * per] = X;
        }
    }
}

template <typename E, int N, int MODE>
cudaError_t walk(const SsmArgs& a0, cudaStream_t s)
{
    SsmArgs a = a0;
    constexpr int CB = kWalkChannels<N>;
    a.ctiles = (a.D / a.G + CB - 1) / CB;
    const int n = (int)sizeof(WalkShared<E, N, MODE>);
    const cudaError_t r = cudaFuncSetAttribute(gla_ssm_walk_kernel<E, N, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    if (r != cudaSuccess) return r;
    const dim3 g((unsigned)((long long)a.B * a.G * a.ctiles), MODE == kSsmState || MODE == kSsmRev ? a.nseg - 1 : a.nseg);
    gla_ssm_walk_kernel<E, N, MODE><<<g, kWalkWarps<N> * 32, n, s>>>(a);
    return cudaGetLastError();
}
template <typename E, int N>
cudaError_t walk(const SsmArgs& a, int mode, cudaStream_t s)
{
    return mode == kSsmOut ? walk<E, N, kSsmOut>(a, s) : mode == kSsmState ? walk<E, N, kSsmState>(a, s)
           : mode == kSsmKeep ? walk<E, N, kSsmKeep>(a, s) : walk<E, N, kSsmRev>(a, s);
}
template <typename E>
cudaError_t walk(const SsmArgs& a, int mode, cudaStream_t s)
{
    return a.N == 8 ? walk<E, 8>(a, mode, s) : a.N == 16 ? walk<E, 16>(a, mode, s)
           : a.N == 32 ? walk<E, 32>(a, mode, s) : walk<E, 64>(a, mode, s);
}

template <typename E, int ROWS>
cudaError_t step(const SsmArgs& a, cudaStream_t s)
{
    const int cpb = kStepNT / (a.N / 4);
    const unsigned g = (unsigned)((long long)((a.B + ROWS - 1) / ROWS) * ((a.D + cpb - 1) / cpb));
    if (a.N == 8) gla_ssm_step_kernel<E, 8, ROWS><<<g, kStepNT, 0, s>>>(a);
    else if (a.N == 16) gla_ssm_step_kernel<E, 16, ROWS><<<g, kStepNT, 0, s>>>(a);
    else if (a.N == 32) gla_ssm_step_kernel<E, 32, ROWS><<<g, kStepNT, 0, s>>>(a);
    else gla_ssm_step_kernel<E, 64, ROWS><<<g, kStepNT, 0, s>>>(a);
    return cudaGetLastError();
}
// Four rows to a thread once that leaves every SM 1024 threads (128 rows of 4096 channels of 16 states, call after call: 22 us singly, 14 so).
template <typename E>
cudaError_t step(const SsmArgs& a, int sms, cudaStream_t s)
{
    return (long long)a.B * a.D * a.N >= 4LL * 4 * 1024 * sms ? step<E, 4>(a, s) : step<E, 1>(a, s);
}

}  // namespace

int ssm_walk_warps(int N) { return N >= 64 ? kWalkWarps<64> : kWalkWarps<8>; }
int ssm_walk_channels(int N) { return kWalkChannels<8> * 8 / N * (N >= 64 ? 2 : 1); }

cudaError_t launch_ssm_step(const SsmArgs& a, gla_dtype dtype, int sms, cudaStream_t s)
{
    return dtype == GLA_BF16 ? step<__nv_bfloat16>(a, sms, s) : step<float>(a, sms, s);
}
cudaError_t launch_ssm_walk(const SsmArgs& a, int mode, gla_dtype dtype, cudaStream_t s)
{
    return dtype == GLA_BF16 ? walk<__nv_bfloat16>(a, mode, s) : walk<float>(a, mode, s);
}
cudaError_t launch_ssm_scan(const SsmArgs& a, bool rev, int sms, cudaStream_t s)
{
    const long long n = ((long long)a.B * a.D * a.N + 255) / 256;
    gla_ssm_scan_kernel<<<(unsigned)(n < 8LL * sms ? n : 8LL * sms), 256, 0, s>>>(a, rev);
    return cudaGetLastError();
}

}  // namespace gla
