// The selective scan's gradients. With r_t = dy_t silu(z_t), a_t = exp(delta_t A) and G_t = dL/dh_t,
//
//     G_t = r_t C_t + a_{t+1} G_{t+1}   (G_T from dS_T),
//     dC_t = sum over channels of r_t h_t,   dB_t = sum over channels of delta_t x_t G_t,
//     p_t = G_t . B_t,   e_t = sum over states of G_t a_t h_{t-1} A,   dA = sum over tokens of delta_t G_t a_t h_{t-1},
//     dx_t = delta_t p_t + D r_t,   ddelta_t = x_t p_t + e_t,   ddt_t = ddelta_t softplus'(dt_t + dt_bias),
//     dz_t = dy_t (C_t . h_t + D x_t) silu'(z_t),   dD = sum r_t x_t,   ddt_bias = sum ddt_t,   dS0 = a_1 G_1.
//
// A walk over the tokens has left the state entering every tile of 16 (gla_ssm_walk). gla_ssm_bwd takes the tiles from
// the last: a thread holds two channels by four states of h, a and G; the tile's two halves of eight tokens are
// formed again with h and a in registers, then walked back. Products a h_{t-1} are formed as such: as h_t - delta x B they would
// lose their digits where a decay is steep. Sums over states end in shared memory per channel and token, sums over channels
// per token over the warp by halving exchanges, then over the block's warps; a block leaves them as partials per channel tile,
// added in a fixed order by gla_ssm_bc_sum. No atomics: results are equal bit for bit from call to call.
//
// Bound by issue: per token, channel and state 9 products or multiply-adds back, 4 for h again and 4.5 for the states kept,
// with 2.5 exponentials.
#include "gla_rows.cuh"
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kS = 4, kC = 2;             // states and channels of a thread
constexpr int kWarps = 4, NT = kWarps * 32;
constexpr int TT = kSsmTile, HALF = TT / 2;

template <int N> constexpr int kBwdChannels = NT * kS * kC / N;

template <typename E, int N>
struct BwdShared {
    static constexpr int CB = kBwdChannels<N>;
    E raw[2][4][TT][CB];                  // x, dt, z, dy
    E bc[2][2][TT][N];
    float delta[TT][CB], dx[TT][CB], r[TT][CB];
    float y[TT][CB], p[TT][CB], e[TT][CB];
    float red[kWarps][TT][2 * N];         // dB, dC over each warp's channels
};

// V values in each of the lanes that differ in bits FROM, 2 FROM .. of the lane, CNT lanes in all: halves are exchanged
// until one value is left (lane bit i choosing the half) or the lanes are done; further lanes add up.
template <int V, int FROM, int CNT>
__device__ __forceinline__ void halve(float (&v)[V])
{
    if constexpr (CNT > 1) {
        if constexpr (V > 1) {
            const bool upper = threadIdx.x & FROM;
            float w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float give = upper ? v[i] : v[V / 2 + i], own = upper ? v[V / 2 + i] : v[i];
                w[i] = own + __shfl_xor_sync(~0u, give, FROM);
            }
            halve<V / 2, FROM * 2, CNT / 2>(w);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) v[i] = w[i];
        } else {
            v[0] += __shfl_xor_sync(~0u, v[0], FROM);
            halve<1, FROM * 2, CNT / 2>(v);
        }
    }
}
constexpr int log2i(int n) { return n <= 1 ? 0 : 1 + log2i(n / 2); }

template <typename E, int N>
__global__ void __launch_bounds__(NT, 2) gla_ssm_bwd_kernel(SsmArgs a)
{
    constexpr int CB = kBwdChannels<N>, Q = N / kS, GROUPS = 32 / Q;
    extern __shared__ __align__(16) char smem_raw[];
    auto& sm = *reinterpret_cast<BwdShared<E, N>*>(smem_raw);
    const int Dg = a.D / a.G, ct = blockIdx.x % a.ctiles;
    const long long bg = blockIdx.x / a.ctiles;
    const int b = (int)(bg / a.G), g = (int)(bg % a.G);
    const int c0 = g * Dg + ct * CB, c1 = g * Dg + Dg;
    const int seg = blockIdx.y, s0 = seg * a.seg, s1 = min(a.T, s0 + a.seg);
    const int tiles = (s1 - s0 + TT - 1) / TT, alltiles = (a.T + TT - 1) / TT;
    const size_t per = (size_t)a.D * N;

    const E* xp = static_cast<const E*>(a.x) + b * a.sx[0];
    const E* dtp = static_cast<const E*>(a.dt) + b * a.sdt[0];
    const E* zp = a.z ? static_cast<const E*>(a.z) + b * a.sz[0] : nullptr;
    const E* dyp = static_cast<const E*>(a.dy) + (size_t)b * a.T * a.D;
    const E* Bp = static_cast<const E*>(a.Bm) + b * a.sB[0] + g * N;
    const E* Cp = static_cast<const E*>(a.Cm) + b * a.sC[0] + g * N;
    auto load = [&](int tile) {                      // tiles from the last, stages in turn
        const int stage = tile & 1, t0 = s0 + tile * TT;
        copy_rows<E, CB, NT>(&sm.raw[stage][0][0][0], xp, a.sx[1], t0, s1, c0, c1);
        copy_rows<E, CB, NT>(&sm.raw[stage][1][0][0], dtp, a.sdt[1], t0, s1, c0, c1);
        if (zp) copy_rows<E, CB, NT>(&sm.raw[stage][2][0][0], zp, a.sz[1], t0, s1, c0, c1);
        copy_rows<E, CB, NT>(&sm.raw[stage][3][0][0], dyp, a.D, t0, s1, c0, c1);
        copy_states<E, N, NT>(&sm.bc[stage][0][0][0], Bp, a.sB[1], t0, s1);
        copy_states<E, N, NT>(&sm.bc[stage][1][0][0], Cp, a.sC[1], t0, s1);
        copies_end();
    };
    if (tiles > 0) load(tiles - 1);

    const int sg = threadIdx.x % Q, cl = threadIdx.x / Q * kC, warp = threadIdx.x / 32;
    const bool on = c0 + cl < c1;
    const size_t so = (size_t)(on ? c0 + cl : c0) * N + sg * kS;
    f2 A[kC][kS / 2], G[kC][kS / 2], dA[kC][kS / 2];
    const float* gfrom = seg < a.nseg - 1 ? a.segG + ((size_t)b * (a.nseg - 1) + seg) * per : a.dST ? a.dST + b * per : nullptr;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        states<kS>(a.A + so + (on ? i * N : 0), A[i]);
#pragma unroll
        for (int j = 0; j < kS / 2; ++j) {
            A[i][j] = mul2(A[i][j], pk(kLog2e, kLog2e));
            G[i][j] = dA[i][j] = pk(0.f, 0.f);
        }
        if (gfrom && on) states<kS>(gfrom + so + i * N, G[i]);
    }
    constexpr int COLS = CB / VEC, VPT = TT * COLS;
    const int vc = threadIdx.x % COLS * VEC;
    float bias[VEC], Dk[VEC], dD[VEC], db[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const bool in = c0 + vc < c1;
        bias[j] = a.bias && in ? a.bias[c0 + vc + j] : 0.f;
        Dk[j] = a.Dk && in ? a.Dk[c0 + vc + j] : 0.f;
        dD[j] = db[j] = 0.f;
    }
    auto vec = [&](const E* p, float (&f)[VEC]) { unpack(*reinterpret_cast<const typename Raw<E>::type*>(p), f); };
    auto put = [&](float* p, const float (&f)[VEC]) { save8(p, f); };

    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int stage = tile & 1, t0 = s0 + tile * TT;
        // the state entering the tile; its loads are in flight during the preparation
        f2 H[kC][kS / 2];
#pragma unroll
        for (int i = 0; i < kC; ++i)
            states<kS>(a.keep + ((size_t)b * alltiles + t0 / TT) * per + so + (on ? i * N : 0), H[i]);
        copies_wait<0>();
        __syncthreads();
        if (tile > 0) load(tile - 1);
        for (int i = threadIdx.x; i < VPT; i += NT) {
            const int tok = i / COLS;
            float x[VEC], d[VEC], r[VEC];
            vec(&sm.raw[stage][0][tok][vc], x);
            vec(&sm.raw[stage][1][tok][vc], d);
            vec(&sm.raw[stage][3][tok][vc], r);
            if (zp) {
                float z[VEC];
                vec(&sm.raw[stage][2][tok][vc], z);
#pragma unroll
                for (int j = 0; j < VEC; ++j) r[j] *= z[j] * sigmoid(z[j]);
            }
            const bool ok = t0 + tok < s1;
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                d[j] += bias[j];
                if (a.softplus) d[j] = softplus(d[j]);
                if (!ok) d[j] = 0.f;
                x[j] *= d[j];
            }
            put(&sm.delta[tok][vc], d);
            put(&sm.dx[tok][vc], x);
            put(&sm.r[tok][vc], r);
        }
        __syncthreads();

        // h and a of a half from the state entering it
        f2 h[HALF][kC][kS / 2], ea[HALF][kC][kS / 2];
        auto ahead = [&](int tok, f2 (&hn)[kC][kS / 2], f2 (&an)[kC][kS / 2], const f2 (&hp)[kC][kS / 2]) {
            const float2 d = *reinterpret_cast<const float2*>(&sm.delta[tok][cl]), x = *reinterpret_cast<const float2*>(&sm.dx[tok][cl]);
            f2 Bv[kS / 2];
            states<kS>(&sm.bc[stage][0][tok][sg * kS], Bv);
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const float di = i ? d.y : d.x, xi = i ? x.y : x.x;
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    an[i][j] = ex2_2(mul2(pk(di, di), A[i][j]));
                    hn[i][j] = fma2(an[i][j], hp[i][j], mul2(pk(xi, xi), Bv[j]));
                }
            }
        };
        f2 M[kC][kS / 2], unused[kC][kS / 2];         // the state entering the second half
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
            for (int j = 0; j < kS / 2; ++j) M[i][j] = H[i][j];
#pragma unroll
        for (int n = 0; n < HALF; ++n) ahead(n, M, unused, M);

#pragma unroll 1
        for (int half = 1; half >= 0; --half) {
            f2 in[kC][kS / 2];
#pragma unroll
            for (int i = 0; i < kC; ++i)
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) in[i][j] = half ? M[i][j] : H[i][j];
            const int tb = half * HALF;
#pragma unroll
            for (int n = 0; n < HALF; ++n) ahead(tb + n, h[n], ea[n], n ? h[n - 1] : in);
#pragma unroll
            for (int n = HALF - 1; n >= 0; --n) {
                const int tok = tb + n;
                const float2 d = *reinterpret_cast<const float2*>(&sm.delta[tok][cl]), x = *reinterpret_cast<const float2*>(&sm.dx[tok][cl]),
                             r = *reinterpret_cast<const float2*>(&sm.r[tok][cl]);
                f2 Bv[kS / 2], Cv[kS / 2], dB[kS / 2], dC[kS / 2];
                states<kS>(&sm.bc[stage][0][tok][sg * kS], Bv);
                states<kS>(&sm.bc[stage][1][tok][sg * kS], Cv);
                float per_c[3][kC];                   // y, p, e of the two channels
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    const f2 d2 = i ? pk(d.y, d.y) : pk(d.x, d.x), x2 = i ? pk(x.y, x.y) : pk(x.x, x.x), r2 = i ? pk(r.y, r.y) : pk(r.x, r.x);
                    f2 ys = pk(0.f, 0.f), ps = ys, es = ys;
#pragma unroll
                    for (int j = 0; j < kS / 2; ++j) {
                        const f2 hp = n ? h[n - 1][i][j] : in[i][j];
                        ys = fma2(h[n][i][j], Cv[j], ys);
                        dC[j] = i ? fma2(r2, h[n][i][j], dC[j]) : mul2(r2, h[n][i][j]);
                        f2 gg = fma2(r2, Cv[j], G[i][j]);
                        dB[j] = i ? fma2(x2, gg, dB[j]) : mul2(x2, gg);
                        ps = fma2(gg, Bv[j], ps);
                        gg = mul2(ea[n][i][j], gg);           // a G: what goes on to the token before
                        G[i][j] = gg;
                        const f2 q = mul2(gg, hp);
                        es = fma2(q, A[i][j], es);
                        dA[i][j] = fma2(q, d2, dA[i][j]);
                    }
                    float u, v;
                    up(ys, u, v); per_c[0][i] = u + v;
                    up(ps, u, v); per_c[1][i] = u + v;
                    up(es, u, v); per_c[2][i] = u + v;
                }
                // over the channel's Q threads: one channel each, then alike
                float* out[3] = {&sm.y[tok][cl], &sm.p[tok][cl], &sm.e[tok][cl]};
                const bool odd = sg & 1;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    float v = (odd ? per_c[k][1] : per_c[k][0]) + __shfl_xor_sync(~0u, odd ? per_c[k][0] : per_c[k][1], 1);
#pragma unroll
                    for (int o = 2; o < Q; o *= 2) v += __shfl_xor_sync(~0u, v, o);
                    if (sg < 2) out[k][sg] = v;
                }
                // over the warp's channels: eight sums, halved over the lanes
                float s[2 * kS];
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    up(dB[j], s[2 * j], s[2 * j + 1]);
                    up(dC[j], s[kS + 2 * j], s[kS + 2 * j + 1]);
                }
                halve<2 * kS, Q, GROUPS>(s);
                constexpr int STEPS = log2i(GROUPS) < 3 ? log2i(GROUPS) : 3, LEFT = 8 >> STEPS;
                const int lane = threadIdx.x % 32, gi = lane / Q;     // bit 0 of gi chose half of eight, bit 1 of four, ..
                int at = 0;
#pragma unroll
                for (int k = 0; k < STEPS; ++k) at += (gi >> k & 1) * (4 >> k);
                if (gi < 1 << STEPS)
#pragma unroll
                    for (int k = 0; k < LEFT; ++k) {
                        const int which = at + k;                    // 0..3 dB, 4..7 dC
                        sm.red[warp][tok][(which / kS) * N + sg * kS + which % kS] = s[k];
                    }
            }
        }
        __syncthreads();
        // rows beyond the channels' end have r = 0, delta = 0 and delta x = 0: they add nothing
        for (int i = threadIdx.x; i < TT * 2 * N; i += NT) {
            const int tok = i / (2 * N), k = i % (2 * N);
            if (t0 + tok >= s1) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += sm.red[w][tok][k];
            a.part_bc[((((size_t)ct * a.B + b) * a.T + t0 + tok) * a.G + g) * (2 * N) + k] = s;
        }
        for (int i = threadIdx.x; i < VPT; i += NT) {
            const int tok = i / COLS;
            if (t0 + tok >= s1 || c0 + vc >= c1) continue;
            float x[VEC], dt[VEC], dy[VEC], d[VEC], r[VEC], y[VEC], p[VEC], e[VEC];
            vec(&sm.raw[stage][0][tok][vc], x);
            vec(&sm.raw[stage][1][tok][vc], dt);
            vec(&sm.raw[stage][3][tok][vc], dy);
            auto get = [&](const float* q, float (&f)[VEC]) {
                unpack(*reinterpret_cast<const Raw<float>::type*>(q), f);
            };
            get(&sm.delta[tok][vc], d);
            get(&sm.r[tok][vc], r);
            get(&sm.y[tok][vc], y);
            get(&sm.p[tok][vc], p);
            get(&sm.e[tok][vc], e);
            const size_t o = ((size_t)b * a.T + t0 + tok) * a.D + c0 + vc;
            if (zp) {
                float z[VEC];
                vec(&sm.raw[stage][2][tok][vc], z);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float s = sigmoid(z[j]);
                    z[j] = dy[j] * fmaf(Dk[j], x[j], y[j]) * fmaf(z[j] * s, 1.f - s, s);
                }
                save8(static_cast<E*>(a.dz) + o, z);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                dD[j] = fmaf(r[j], x[j], dD[j]);
                float ddt = fmaf(x[j], p[j], e[j] * kLn2);
                if (a.softplus) ddt *= softplus_slope(dt[j] + bias[j]);
                db[j] += ddt;
                dt[j] = ddt;
                x[j] = fmaf(d[j], p[j], Dk[j] * r[j]);
            }
            save8(static_cast<E*>(a.dx) + o, x);
            save8(static_cast<E*>(a.ddt) + o, dt);
        }
    }

    if (on && seg == 0 && a.dS0) {
#pragma unroll
        for (int i = 0; i < kC; ++i)
            *reinterpret_cast<ulonglong2*>(a.dS0 + b * per + so + i * N) = make_ulonglong2(G[i][0], G[i][1]);
    }
    float* part = a.part_p + ((size_t)b * a.nseg + seg) * (per + 2 * (size_t)a.D);
    if (on) {
#pragma unroll
        for (int i = 0; i < kC; ++i)
            *reinterpret_cast<ulonglong2*>(part + so + i * N) = make_ulonglong2(dA[i][0], dA[i][1]);
    }
    // dD and ddt_bias over the threads that finished the same channels, in order
    __syncthreads();
    constexpr int ROWS = (NT < VPT ? NT : VPT) / COLS;
    if (threadIdx.x < ROWS * COLS) {
        put(&sm.delta[0][0] + threadIdx.x / COLS * CB + vc, dD);
        put(&sm.y[0][0] + threadIdx.x / COLS * CB + vc, db);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < CB; c += NT) {
        if (c0 + c >= c1) continue;
        float s = 0.f, q = 0.f;
        for (int k = 0; k < ROWS; ++k) {
            s += (&sm.delta[0][0])[k * CB + c];
            q += (&sm.y[0][0])[k * CB + c];
        }
        part[per + c0 + c] = s;
        part[per + a.D + c0 + c] = q;
    }
}

// dB and dC: the channel tiles' partials, in order, four values per thread.
template <typename E>
__global__ void gla_ssm_bc_sum_kernel(const float* part, long long rows, int N, int ctiles, E* dB, E* dC)
{
    const int q = N / 2;                              // groups of four values per row of 2 N
    const long long all = rows * q;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += (long long)gridDim.x * blockDim.x) {
        const long long row = i / q;
        const int k = (int)(i - row * q) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < ctiles; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((size_t)c * rows + row) * (2 * N) + k);
            s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
        }
        E* to = k < N ? dB + row * N + k : dC + row * N + k - N;
        to[0] = (E)s.x; to[1] = (E)s.y; to[2] = (E)s.z; to[3] = (E)s.w;
    }
}

template <typename E, int N>
cudaError_t bwd(const SsmArgs& a0, cudaStream_t s)
{
    SsmArgs a = a0;
    constexpr int CB = kBwdChannels<N>;
    a.ctiles = (a.D / a.G + CB - 1) / CB;
    const int n = (int)sizeof(BwdShared<E, N>);
    const cudaError_t r = cudaFuncSetAttribute(gla_ssm_bwd_kernel<E, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    if (r != cudaSuccess) return r;
    gla_ssm_bwd_kernel<E, N><<<dim3((unsigned)((long long)a.B * a.G * a.ctiles), a.nseg), NT, n, s>>>(a);
    return cudaGetLastError();
}
template <typename E>
cudaError_t bwd(const SsmArgs& a, cudaStream_t s)
{
    return a.N == 8 ? bwd<E, 8>(a, s) : a.N == 16 ? bwd<E, 16>(a, s) : a.N == 32 ? bwd<E, 32>(a, s) : bwd<E, 64>(a, s);
}

}  // namespace

int ssm_bwd_channels(int N) { return NT * kS * kC / N; }

cudaError_t launch_ssm_bwd(const SsmArgs& a, gla_dtype dtype, cudaStream_t s)
{
    return dtype == GLA_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}

cudaError_t launch_ssm_bc_sum(const SsmArgs& a, void* dB, void* dC, gla_dtype dtype, int sms, cudaStream_t s)
{
    const long long rows = (long long)a.B * a.T * a.G, n = (rows * (a.N / 2) + 255) / 256;
    const int CB = ssm_bwd_channels(a.N), ct = (a.D / a.G + CB - 1) / CB;
    const unsigned g = (unsigned)(n < 16LL * sms ? n : 16LL * sms);
    if (dtype == GLA_BF16)
        gla_ssm_bc_sum_kernel<<<g, 256, 0, s>>>(a.part_bc, rows, a.N, ct, static_cast<__nv_bfloat16*>(dB), static_cast<__nv_bfloat16*>(dC));
    else
        gla_ssm_bc_sum_kernel<<<g, 256, 0, s>>>(a.part_bc, rows, a.N, ct, static_cast<float*>(dB), static_cast<float*>(dC));
    return cudaGetLastError();
}

}  // namespace gla
