// The selective scan's gradients. With r_t = dy_t silu(z_t), a_t = exp(delta_t A) and G_t = dL/dh_t,
//
//     G_t = r_t C_t + a_{t+1} G_{t+1}   (G_T from dS_T),
//     dC_t = sum over channels of r_t h_t,   dB_t = sum over channels of delta_t x_t G_t,
//     p_t = G_t . B_t,   e_t = sum over states of G_t a_t h_{t-1} A,   dA = sum over tokens of delta_t G_t a_t h_{t-1},
//     dx_t = delta_t p_t + D r_t,   ddelta_t = x_t p_t + e_t,   ddt_t = ddelta_t softplus'(dt_t + dt_bias),
//     dz_t = dy_t (C_t . h_t + D x_t) silu'(z_t),   dD = sum r_t x_t,   ddt_bias = sum ddt_t,   dS0 = a_1 G_1.
//
// A walk over the tokens has left the state entering every tile of 16 (gla_ssm_walk). gla_ssm_bwd takes the tiles from
// the last: a thread holds two channels by four states of A, G and dA. It walks the tile's states once from the kept one, leaving those
// that enter its parts of four tokens, then takes the parts from the last: h and a of the four again, in registers, and back.
// Products a h_{t-1} are formed as such: as h_t - delta x B they would lose their digits where a decay is steep. Sums over
// states end in shared memory per channel and token, sums over channels per token over the warp by halving exchanges, then over the
// block's warps; a block leaves them as partials per channel tile, added in a fixed order by gla_ssm_bc_sum. No atomics: results are
// equal bit for bit from call to call.
//
// Bound by the multiply-adds' register reads (a packed one of three different pairs takes 3.75 cycles) and by waits that two warps
// a scheduler cannot hide (228 registers, 111 KB a block): four rows of 2048 tokens of 4096 channels of 16 states take 703 us, 22 warp
// instructions a state at 47% of the issue slots; per token, channel and state 10 products or multiply-adds back, 4 for h and a again, 3 for
// the tile's first walk. Preparing and finishing the tiles is 0.2 of it. One channel a thread (twice the warps) took 1.25 times as long.
#include "gla_ssm.cuh"

namespace gla {
namespace {

constexpr int kS = 4, kC = 2;             // states and channels of a thread
constexpr int kWarps = 4, NT = kWarps * 32;
constexpr int TT = kSsmTile, PART = 4;    // tokens per tile, and per part of it whose states are in registers at a time

template <int N> constexpr int kBwdChannels = NT * kS * kC / N;

// A thread's four states of a channel are taken in the order n ^ m, m from its lane: then what the lanes exchange when they
// sum over the warp's channels lies at the same place in all of them. B and C of a tile lie in shared memory once in each order,
// 64 bytes (of 8 states 32) further on each time, so that the orders' reads meet no bank twice.
template <int N> constexpr int kOrders = N >= 64 ? 2 : 4;      // (with two groups of lanes only pairs are exchanged)

// Sums over states are left in shared memory by each of a channel's N / kS threads. Where two blocks would not fit an SM so, they are
// halved first, once or twice, by exchanges between neighbouring lanes (fp32, 3 x 777 tokens of 1040 channels of 32 states: 174 us with
// one block an SM, 111 so; of 8 fp32 states nothing more can be halved: one block).
template <typename E, int N> constexpr int kHalvings = N >= 64 ? 2 : N == 16 && sizeof(E) == 2 ? 0 : 1;

template <typename E, int N>
struct BwdShared {
    static constexpr int CB = kBwdChannels<N>, Q = N / kS, PQ = Q >> kHalvings<E, N>;
    E raw[2][4][TT][CB];                      // x, dt, z, dy
    E bc[2][2][TT][N];
    float wide[2][kOrders<N>][TT * N + (N == 8 ? 8 : 16)];   // B, C
    // the states entering the tile (two tiles' in turn), and its parts but the first and the last, as each thread reads them
    float keep[2][kC][NT * 4], mid[TT / PART - 2][kC][NT * 4];
    // Rows of a value per channel: the first four of every eight channels, then the other four, with the eights 0 - 3 and 4 - 7
    // exchanged. So a thread's eight channels are two reads of 16 bytes beside its neighbours', and a warp's channels, two
    // neighbouring eights, still meet every bank once.
    static constexpr int HALF = CB / 2, TURN = CB >= 64 ? 4 : 0;
    float delta[TT][CB], dx[TT][CB], r[TT][CB];
    float part[3][PQ][TT * CB + (kHalvings<E, N> == 0 || N > 32 ? 4 : 128 / N)];     // y, p, e over states, rows so far apart that a warp's stores meet no bank twice
    float red[kWarps][TT][2 * N];             // dB, dC over each warp's channels
};

// Four values in the order n ^ m (which is its own inverse).
__device__ __forceinline__ void reorder(float (&v)[4], int m)
{
    const bool far = m & 2, near = m & 1;
    const float a = far ? v[2] : v[0], b = far ? v[3] : v[1], c = far ? v[0] : v[2], d = far ? v[1] : v[3];
    v[0] = near ? b : a; v[1] = near ? a : b; v[2] = near ? d : c; v[3] = near ? c : d;
}
__device__ __forceinline__ void load4(const float* p, int m, f2 (&r)[2])
{
    const float4 q = *reinterpret_cast<const float4*>(p);
    float v[4] = {q.x, q.y, q.z, q.w};
    reorder(v, m);
    r[0] = pk(v[0], v[1]); r[1] = pk(v[2], v[3]);
}
__device__ __forceinline__ void store4(float* p, int m, const f2 (&r)[2])
{
    float v[4];
    up(r[0], v[0], v[1]); up(r[1], v[2], v[3]);
    reorder(v, m);
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

template <typename E, int N>
__global__ void __launch_bounds__(NT, 2) gla_ssm_bwd_kernel(SsmArgs a)
{
    typedef BwdShared<E, N> Shared;
    constexpr int CB = kBwdChannels<N>, Q = N / kS, GROUPS = 32 / Q, HALF = Shared::HALF, TURN = Shared::TURN, PQ = Shared::PQ,
                  HALVINGS = kHalvings<E, N>;
    extern __shared__ __align__(16) char smem_raw[];
    auto& sm = *reinterpret_cast<Shared*>(smem_raw);
    const int Dg = a.D / a.G, ct = blockIdx.x % a.ctiles;
    const long long bg = blockIdx.x / a.ctiles;
    const int b = (int)(bg / a.G), g = (int)(bg % a.G);
    const int c0 = g * Dg + ct * CB, c1 = g * Dg + Dg;
    const int seg = blockIdx.y, s0 = seg * a.seg, s1 = min(a.T, s0 + a.seg);
    const int tiles = (s1 - s0 + TT - 1) / TT, alltiles = (a.T + TT - 1) / TT;
    const size_t per = (size_t)a.D * N;

    const int sg = threadIdx.x % Q, cl = threadIdx.x / Q * kC, warp = threadIdx.x / 32;
    const int gi = threadIdx.x % 32 / Q;             // the lane's place among those with the same states
    const int m = (gi & 1) * 2 + (GROUPS > 2 ? gi >> 1 & 1 : 0);
    const bool on = c0 + cl < c1;
    const size_t so = (size_t)(on ? c0 + cl : c0) * N + sg * kS;
    const E* const zp = a.z ? static_cast<const E*>(a.z) + b * a.sz[0] + c0 : nullptr;
    const int last = s0 + (tiles - 1) * TT;
    TileCopy<E, TT, CB, NT> cx, cd, cz, cy;
    TileCopy<E, TT, N, NT> cB, cC;
    cx.start(static_cast<const E*>(a.x) + b * a.sx[0] + c0, a.sx[1], last, c1 - c0);
    cd.start(static_cast<const E*>(a.dt) + b * a.sdt[0] + c0, a.sdt[1], last, c1 - c0);
    if (zp) cz.start(zp, a.sz[1], last, c1 - c0);
    cy.start(static_cast<const E*>(a.dy) + (size_t)b * a.T * a.D + c0, a.D, last, c1 - c0);
    cB.start(static_cast<const E*>(a.Bm) + b * a.sB[0] + g * N, a.sB[1], last, N);
    cC.start(static_cast<const E*>(a.Cm) + b * a.sC[0] + g * N, a.sC[1], last, N);
    auto load = [&](int tile) {                      // tiles from the last, stages in turn
        const int stage = tile & 1;
        cx.go(&sm.raw[stage][0][0][0], s1, -TT);
        cd.go(&sm.raw[stage][1][0][0], s1, -TT);
        if (zp) cz.go(&sm.raw[stage][2][0][0], s1, -TT);
        cy.go(&sm.raw[stage][3][0][0], s1, -TT);
        cB.go(&sm.bc[stage][0][0][0], s1, -TT);
        cC.go(&sm.bc[stage][1][0][0], s1, -TT);
        // (each thread copies the states that it reads itself)
#pragma unroll
        for (int i = 0; i < kC; ++i)
            copy16(&sm.keep[stage][i][threadIdx.x * 4], a.keep + ((size_t)b * alltiles + s0 / TT + tile) * per + so + (on ? i * N : 0), true);
        copies_end();
    };
    if (tiles > 0) load(tiles - 1);

    f2 A[kC][kS / 2], G[kC][kS / 2], dA[kC][kS / 2];
    const float* gfrom = seg < a.nseg - 1 ? a.segG + ((size_t)b * (a.nseg - 1) + seg) * per : a.dST ? a.dST + b * per : nullptr;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
        load4(a.A + so + (on ? i * N : 0), m, A[i]);
#pragma unroll
        for (int j = 0; j < kS / 2; ++j) {
            A[i][j] = mul2(A[i][j], pk(kLog2e, kLog2e));
            G[i][j] = dA[i][j] = pk(0.f, 0.f);
        }
        if (gfrom && on) load4(gfrom + so + i * N, m, G[i]);
    }
    constexpr int COLS = CB / VEC, VPT = TT * COLS;
    const int vc = threadIdx.x % COLS * VEC;
    f2 dD[4], db[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) dD[j] = db[j] = 0ull;
    // this block's sums of dA, dD and ddt_bias
    float* const part_p = a.part_p + ((size_t)b * a.nseg + seg) * (per + 2 * (size_t)a.D);
    const bool vin = c0 + vc < c1;
    // a thread's eight channels of a row, and its pair's place
    auto put8 = [&](float* row, const f2 (&v)[4]) {
        *reinterpret_cast<ulonglong2*>(row + vc / 2) = make_ulonglong2(v[0], v[1]);
        *reinterpret_cast<ulonglong2*>(row + HALF + (vc / 2 ^ 4 * TURN)) = make_ulonglong2(v[2], v[3]);
    };
    auto get8 = [&](const float* row, f2 (&v)[4]) {
        const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(row + vc / 2), q = *reinterpret_cast<const ulonglong2*>(row + HALF + (vc / 2 ^ 4 * TURN));
        v[0] = p.x; v[1] = p.y; v[2] = q.x; v[3] = q.y;
    };
    const int cp = cl & 4 ? HALF + ((cl >> 3 ^ TURN) * 4) + (cl & 3) : (cl >> 3) * 4 + (cl & 3);
    f2 bias[4], Dk[4];
    params8(a.bias ? a.bias + c0 + vc : nullptr, vin, bias);
    params8(a.Dk ? a.Dk + c0 + vc : nullptr, vin, Dk);

    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int stage = tile & 1, t0 = s0 + tile * TT;
        copies_wait<0>();
        __syncthreads();
        if (tile > 0) load(tile - 1);
        for (int i = threadIdx.x; i < 2 * TT * N / 4; i += NT) {
            const int which = i / (TT * N / 4), at = i % (TT * N / 4) * 4;
            f2 q[2];
            states<4>(&sm.bc[stage][which][0][0] + at, q);
            float v[4];
            up(q[0], v[0], v[1]); up(q[1], v[2], v[3]);
            *reinterpret_cast<float4*>(&sm.wide[which][0][at]) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(&sm.wide[which][1][at]) = make_float4(v[2], v[3], v[0], v[1]);
            if constexpr (kOrders<N> > 2) {
                *reinterpret_cast<float4*>(&sm.wide[which][2][at]) = make_float4(v[1], v[0], v[3], v[2]);
                *reinterpret_cast<float4*>(&sm.wide[which][3][at]) = make_float4(v[3], v[2], v[1], v[0]);
            }
        }
        for (int i = threadIdx.x; i < VPT; i += NT) {
            const int tok = i / COLS;
            f2 x[4], d[4], r[4];
            states<8>(&sm.raw[stage][0][tok][vc], x);
            states<8>(&sm.raw[stage][1][tok][vc], d);
            states<8>(&sm.raw[stage][3][tok][vc], r);
            if (zp) {
                f2 z[4];
                states<8>(&sm.raw[stage][2][tok][vc], z);
#pragma unroll
                for (int j = 0; j < 4; ++j) r[j] = mul2(r[j], mul2(z[j], sig(z[j])));
            }
            const bool ok = t0 + tok < s1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                d[j] = add2(d[j], bias[j]);
                if (a.softplus) d[j] = softplus(d[j]);
                if (!ok) d[j] = 0ull;
                x[j] = mul2(x[j], d[j]);
            }
            put8(sm.delta[tok], d);
            put8(sm.dx[tok], x);
            put8(sm.r[tok], r);
        }
        __syncthreads();

        // h and a of a token from the state before it
        f2 h[PART][kC][kS / 2], ea[PART][kC][kS / 2];
        const int slot = (m & 1) * 2 + (m >> 1);      // (neighbouring lanes read neighbouring places)
        const float* Bw = &sm.wide[0][slot][sg * kS];
        const float* Cw = &sm.wide[1][slot][sg * kS];
        auto ahead = [&](int tok, f2 (&hn)[kC][kS / 2], f2 (&an)[kC][kS / 2], const f2 (&hp)[kC][kS / 2]) {
            const float2 d = *reinterpret_cast<const float2*>(&sm.delta[tok][cp]), x = *reinterpret_cast<const float2*>(&sm.dx[tok][cp]);
            f2 Bv[kS / 2];
            states<kS>(Bw + tok * N, Bv);
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                const float di = i ? d.y : d.x, xi = i ? x.y : x.x;
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    an[i][j] = ex2_2(mul2(both(di), A[i][j]));
                    hn[i][j] = fma2(an[i][j], hp[i][j], mul2(both(xi), Bv[j]));
                }
            }
        };
        // the states entering the tile's parts; the first of them is the one that was kept, the last stays in registers
        f2 in[kC][kS / 2];
#pragma unroll
        for (int i = 0; i < kC; ++i) load4(&sm.keep[stage][i][threadIdx.x * 4], m, in[i]);
#pragma unroll 1
        for (int part = 0; part < TT / PART - 1; ++part) {
            if (part > 0)
#pragma unroll
                for (int i = 0; i < kC; ++i) *reinterpret_cast<ulonglong2*>(&sm.mid[part - 1][i][threadIdx.x * 4]) = make_ulonglong2(in[i][0], in[i][1]);
#pragma unroll
            for (int n = 0; n < PART; ++n) ahead(part * PART + n, in, ea[0], in);
        }

        // As the states in the walk, G takes the tile's decay at once in the end: the product of the decays runs beside it.
        f2 Gin[kC][kS / 2], run[kC][kS / 2];
        float sd[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            sd[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kS / 2; ++j) {
                Gin[i][j] = G[i][j];
                run[i][j] = both(1.f);
            }
        }
        // dB, dC of a token over the warp's channels: the lanes with the same states (GROUPS of them) halve what they hold, giving
        // away the second half of it: first pairs, then values, then B or C; lanes beyond that add up. It is done in three steps
        // among the next token's products, whose waits they fill.
        float vB[4], vC[4];
        auto sum_begin = [&](const f2 (&dB)[kS / 2], const f2 (&dC)[kS / 2]) {
            up(dB[0], vB[0], vB[1]); up(dB[1], vB[2], vB[3]);
            up(dC[0], vC[0], vC[1]); up(dC[1], vC[2], vC[3]);
            vB[2] = __shfl_xor_sync(~0u, vB[2], Q); vB[3] = __shfl_xor_sync(~0u, vB[3], Q);
            vC[2] = __shfl_xor_sync(~0u, vC[2], Q); vC[3] = __shfl_xor_sync(~0u, vC[3], Q);
        };
        auto sum_middle = [&] {
            vB[0] += vB[2]; vB[1] += vB[3]; vC[0] += vC[2]; vC[1] += vC[3];
            if constexpr (GROUPS > 2) {
                vB[1] = __shfl_xor_sync(~0u, vB[1], 2 * Q);
                vC[1] = __shfl_xor_sync(~0u, vC[1], 2 * Q);
            }
        };
        const bool isC = gi & 4;
        auto sum_last = [&] {
            if constexpr (GROUPS > 2) {
                vB[0] += vB[1];
                vC[0] += vC[1];
                if constexpr (GROUPS > 4) vB[1] = __shfl_xor_sync(~0u, isC ? vB[0] : vC[0], 4 * Q);
            }
        };
        auto sum_end = [&](int tok) {
            float* red = &sm.red[warp][tok][sg * kS];
            if constexpr (GROUPS == 2) {
                red[m] = vB[0]; red[m ^ 1] = vB[1]; red[N + m] = vC[0]; red[N + (m ^ 1)] = vC[1];
            } else if constexpr (GROUPS == 4) {
                red[m] = vB[0]; red[N + m] = vC[0];
            } else {
                float v = (isC ? vC[0] : vB[0]) + vB[1];
                if constexpr (GROUPS == 16) v += __shfl_xor_sync(~0u, v, 8 * Q);
                if (GROUPS == 8 || gi < 8) red[(isC ? N : 0) + m] = v;
            }
        };
        struct Token { float2 d, x, r; f2 B[kS / 2], C[kS / 2]; };
        auto fetch = [&](int tok, Token& p) {
            p.d = *reinterpret_cast<const float2*>(&sm.delta[tok][cp]);
            p.x = *reinterpret_cast<const float2*>(&sm.dx[tok][cp]);
            p.r = *reinterpret_cast<const float2*>(&sm.r[tok][cp]);
            states<kS>(Bw + tok * N, p.B);
            states<kS>(Cw + tok * N, p.C);
        };
        f2 dB[kS / 2], dC[kS / 2];
#pragma unroll 1
        for (int part = TT / PART - 1; part >= 0; --part) {
            const int tb = part * PART;
            if (part == 0) {
#pragma unroll
                for (int i = 0; i < kC; ++i) load4(&sm.keep[stage][i][threadIdx.x * 4], m, in[i]);
            } else if (part < TT / PART - 1) {
#pragma unroll
                for (int i = 0; i < kC; ++i) states<kS>(&sm.mid[part - 1][i][threadIdx.x * 4], in[i]);
            }
#pragma unroll
            for (int n = 0; n < PART; ++n) ahead(tb + n, h[n], ea[n], n ? h[n - 1] : in);
            Token p[2];
            fetch(tb + PART - 1, p[(PART - 1) % 2]);
#pragma unroll
            for (int n = PART - 1; n >= 0; --n) {
                const int tok = tb + n;
                const Token& t = p[n % 2];
                if (n > 0) fetch(tok - 1, p[(n - 1) % 2]);
                const bool before = n < PART - 1;              // the token after this one is of this part: its sums are due
                if (before) sum_begin(dB, dC);
                float of[3][kC];
#pragma unroll
                for (int i = 0; i < kC; ++i) {
                    const float di = i ? t.d.y : t.d.x;
                    const f2 d2 = both(di), x2 = both(i ? t.x.y : t.x.x), r2 = both(i ? t.r.y : t.r.x);
                    f2 ys = 0ull, ps = 0ull, es = 0ull;
                    sd[i] += di;
#pragma unroll
                    for (int j = 0; j < kS / 2; ++j) {
                        // (multiply-adds with a common first operand side by side: it is read from the registers once)
                        const f2 hp = n ? h[n - 1][i][j] : in[i][j];
                        ys = fma2(h[n][i][j], t.C[j], ys);
                        dC[j] = i ? fma2(h[n][i][j], r2, dC[j]) : mul2(h[n][i][j], r2);
                        const f2 gg = fma2(r2, t.C[j], G[i][j]);
                        ps = fma2(gg, t.B[j], ps);
                        dB[j] = i ? fma2(gg, x2, dB[j]) : mul2(gg, x2);
                        G[i][j] = mul2(ea[n][i][j], gg);      // what goes on to the token before
                        run[i][j] = mul2(ea[n][i][j], run[i][j]);
                        const f2 q = mul2(G[i][j], hp);
                        es = fma2(q, A[i][j], es);
                        dA[i][j] = fma2(q, d2, dA[i][j]);
                    }
                    if (before) {
                        if (i == 0) sum_middle();
                        else sum_last();
                    }
                    // y, p, e of the channel over this thread's states
                    const float sums[3] = {sum2(ys), sum2(ps), sum2(es)};
#pragma unroll
                    for (int k = 0; k < 3; ++k) of[k][i] = sums[k];
                }
                if constexpr (HALVINGS == 0) {
#pragma unroll
                    for (int k = 0; k < 3; ++k) *reinterpret_cast<float2*>(&sm.part[k][sg][tok * CB + cp]) = make_float2(of[k][0], of[k][1]);
                } else {
                    const bool odd = sg & 1;               // a pair of lanes keeps one channel each
#pragma unroll
                    for (int k = 0; k < 3; ++k) {
                        float v = (odd ? of[k][1] : of[k][0]) + __shfl_xor_sync(~0u, odd ? of[k][0] : of[k][1], 1);
                        if constexpr (HALVINGS > 1) v += __shfl_xor_sync(~0u, v, 2);
                        if (HALVINGS < 2 || !(sg & 2)) sm.part[k][sg >> HALVINGS][tok * CB + cp + (sg & 1)] = v;
                    }
                }
                if (before) sum_end(tok + 1);
            }
            sum_begin(dB, dC);
            sum_middle();
            sum_last();
            sum_end(tb);
        }
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
            for (int j = 0; j < kS / 2; ++j) G[i][j] = fma2(fma2(run[i][j], both(-1.f), ex2_2(mul2(both(sd[i]), A[i][j]))), Gin[i][j], G[i][j]);
        // dA of four tiles at a time into the sum of all: a sum of few terms is added to one of many
        if (on && tile % 4 == 0) {
            const bool begun = tile / 4 != (tiles - 1) / 4;
#pragma unroll
            for (int i = 0; i < kC; ++i) {
                f2 sum[kS / 2] = {0ull, 0ull};
                if (begun) load4(part_p + so + i * N, m, sum);
#pragma unroll
                for (int j = 0; j < kS / 2; ++j) {
                    sum[j] = add2(sum[j], dA[i][j]);
                    dA[i][j] = 0ull;
                }
                store4(part_p + so + i * N, m, sum);
            }
        }
        __syncthreads();
        // (channels beyond the group's end have r = 0 and delta x = 0: they add nothing)
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
            if (t0 + tok >= s1 || !vin) continue;
            f2 x[4], dt[4], d[4], r[4], o[3][4];
            states<8>(&sm.raw[stage][0][tok][vc], x);
            states<8>(&sm.raw[stage][1][tok][vc], dt);
            get8(sm.delta[tok], d);
            get8(sm.r[tok], r);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                get8(&sm.part[k][0][tok * CB], o[k]);
#pragma unroll
                for (int q = 1; q < PQ; ++q) {
                    f2 f[4];
                    get8(&sm.part[k][q][tok * CB], f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[k][j] = add2(o[k][j], f[j]);
                }
            }
            const size_t at = ((size_t)b * a.T + t0 + tok) * a.D + c0 + vc;
            if (zp) {
                f2 z[4], dy[4];
                states<8>(&sm.raw[stage][2][tok][vc], z);
                states<8>(&sm.raw[stage][3][tok][vc], dy);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const f2 s = sig(z[j]), left = fma2(s, both(-1.f), both(1.f));
                    z[j] = mul2(mul2(dy[j], fma2(Dk[j], x[j], o[0][j])), fma2(mul2(z[j], s), left, s));
                }
                keep8(static_cast<E*>(a.dz) + at, z);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                dD[j] = fma2(r[j], x[j], dD[j]);
                f2 g = fma2(x[j], o[1][j], mul2(o[2][j], both(kLn2)));
                if (a.softplus) g = mul2(g, sig(add2(dt[j], bias[j])));
                db[j] = add2(db[j], g);
                dt[j] = g;
                x[j] = fma2(d[j], o[1][j], mul2(Dk[j], r[j]));
            }
            keep8(static_cast<E*>(a.dx) + at, x);
            keep8(static_cast<E*>(a.ddt) + at, dt);
        }
    }

    if (on && seg == 0 && a.dS0) {
#pragma unroll
        for (int i = 0; i < kC; ++i) store4(a.dS0 + b * per + so + i * N, m, G[i]);
    }
    // dD and ddt_bias over the threads that finished the same channels, in order
    __syncthreads();
    constexpr int ROWS = (NT < VPT ? NT : VPT) / COLS;
    if (threadIdx.x < ROWS * COLS) {
        keep8(&sm.delta[0][0] + threadIdx.x / COLS * CB + vc, dD);
        keep8(&sm.dx[0][0] + threadIdx.x / COLS * CB + vc, db);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < CB; c += NT) {
        if (c0 + c >= c1) continue;
        float s = 0.f, q = 0.f;
        for (int k = 0; k < ROWS; ++k) {
            s += (&sm.delta[0][0])[k * CB + c];
            q += (&sm.dx[0][0])[k * CB + c];
        }
        part_p[per + c0 + c] = s;
        part_p[per + a.D + c0 + c] = q;
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
#pragma unroll 8
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
