// gla_delta_chain: the serial pass of the chunk form of the gated delta rule. For each 64-token
// chunk, with the state S entering it, the prep's T, P and gates (e = exp(G), l = exp(G_end - G)):
//
//     R = -e K S,   U = T V + T R,   O = scale e (Q S) + P U,   S <- exp(G_end) S + K^T (l U).
//
// A CTA owns 128 columns of dv of one head. Everything is kept transposed, dv along the 128
// tensor-memory lanes, so that the state, R and U are A operands read from tensor memory and a
// thread owns one column of dv: no operand of the chain passes through shared memory. The state
// itself stays in fp32 registers (64 keys a thread at dk = 128); the tensor cores only form the
// chunk's increment. Per chunk the chain is four products with a register step between each:
//
//     S -> bf16 parts | K S | R -> parts | T R | l U -> parts | K^T (l U) | S
//
// Every operand that is not an input (S, R, U, T, P) goes into the products in two bf16 parts,
// hi + lo, good to 2^-17; K, V and Q are exact: two products for K S, K^T U, Q S and T V, three for
// T R and P U. So the fp32 state is good to 3e-6, and O to its last rounding: with one part of P
// and U it was not (keys that repeat make P U a sum of cancelling terms: 7.5e-3 where all keys
// are the same). Q S, T V and P U run off the chain, and so does the drain of O on four other warps.
//
// Bound by the chain's latency (the products are 0.4 us of it per chunk at dk = dv = 128).
//
// Warps: 0 TMA producer, 1 MMA issuer and tensor-memory owner, 4-11 the chain's register steps
// (two groups of four warps; a group owns half of the keys and half of the tokens), 12-15 drain.
#include "gla_delta_dev.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 512;
constexpr int NST = 2;            // chunks in flight
constexpr int DVT = 128;          // dv columns per CTA

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

enum { ERR_TMA = 0x611, ERR_MMA = 0x612, ERR_EPI = 0x613, ERR_DRAIN = 0x614 };

template <int DK>
struct CL {
    static constexpr int KB = (DK / 64) * SLAB;
    static constexpr int K_OFF = 0, Q_OFF = KB, V_OFF = 2 * KB, TH_OFF = V_OFF + 2 * SLAB, TL_OFF = TH_OFF + SLAB,
                         P_OFF = TL_OFF + SLAB, PL_OFF = P_OFF + SLAB, G_OFF = PL_OFF + SLAB;
    static constexpr int STAGE = G_OFF + 1024;
    static constexpr int BYTES = G_OFF + 4 * C * 4;       // of one stage's loads, all of dv present
    static constexpr int O_OFF = NST * STAGE;             // [2 halves of dv][64 tokens][64] bf16
    static constexpr int BAR_OFF = O_OFF + 2 * SLAB;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    // tensor memory columns
    static constexpr int tD = 0;                          // the state's increment, [dv][DK]
    static constexpr int tSh = DK, tSl = tSh + DK / 2;    // the state's parts
    static constexpr int tKs = 0;                         // K S, before the increment takes its place
    static constexpr int tX = 2 * DK;                     // U; then its high part
    static constexpr int tRh = tX + 64, tRl = tRh + 32;   // R's parts, then l U's
    static constexpr int tOq = tRl + 32, tOp = tOq + 64;  // Q S, P U
    static constexpr int TCOLS = 512;
    static_assert(tOp + 64 <= TCOLS, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int DK>
__global__ void __launch_bounds__(NT, 1)
gla_delta_chain_kernel(DeltaChain a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmTh,
                       const __grid_constant__ CUtensorMap tmTl, const __grid_constant__ CUtensorMap tmP,
                       const __grid_constant__ CUtensorMap tmPl,
                       const __grid_constant__ CUtensorMap tmO, int* status)
{
    using L = CL<DK>;
    constexpr int HC = DK / 2;        // keys per group
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* full = bar;             // [NST] stage loaded
    uint64_t* empty = bar + NST;      // [NST] stage consumed: the products' commit and four drain warps
    uint64_t* s_ready = bar + 2 * NST;      // state parts written (8 warps)
    uint64_t* ks_full = s_ready + 1;        // K S formed
    uint64_t* r_ready = s_ready + 2;        // R's parts written (8 warps)
    uint64_t* u_full = s_ready + 3;         // T R formed
    uint64_t* u_ready = s_ready + 4;        // U's parts written (8 warps)
    uint64_t* d_full = s_ready + 5;         // the increment formed
    uint64_t* o_full = s_ready + 6;         // Q S and P U formed
    uint64_t* o_empty = s_ready + 7;        // O read out (4 warps)
    uint64_t* p_ready = s_ready + 8;        // U's own parts written, for P U (8 warps)
    uint64_t* fin = s_ready + 9;
    uint32_t* holder = reinterpret_cast<uint32_t*>(s_ready + 10);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(s_ready + 11);

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32, wg = warp / 4;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int dv0 = blockIdx.x * DVT;
    const bool wide = dv0 + 64 < a.dv;      // the tile's second half is inside dv
    const int n = a.nch;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 5);
        }
        for (int i = 0; i < 10; ++i) mbar_init(&s_ready[i], (i == 0 || i == 2 || i == 4 || i == 8) ? 8 : i == 7 ? 4 : 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, L::TCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *holder;

    if (wg == 0) {
        regs_dec<56>();
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------ TMA producer
            prefetch_tmap(&tmK); prefetch_tmap(&tmQ); prefetch_tmap(&tmV);
            prefetch_tmap(&tmTh); prefetch_tmap(&tmTl); prefetch_tmap(&tmP); prefetch_tmap(&tmO);
            int issued = 0;
            for (int m = 0; m < n && !*abort_flag; ++m, ++issued) {
                const int st = m % NST, t0 = m * C, at = bh * n + m;
                if (m >= NST) wait(&empty[st], ((m / NST) - 1) & 1, abort_flag, status, ERR_TMA);
                uint8_t* sb = sm + st * L::STAGE;
                mbar_arrive_expect_tx(&full[st], L::BYTES - (wide ? 0 : SLAB));
#pragma unroll
                for (int i = 0; i < DK / 64; ++i) tma_load_3d(sb + L::K_OFF + i * SLAB, &tmK, &full[st], 64 * i, t0, bk);
                tma_load_3d(sb + L::V_OFF, &tmV, &full[st], dv0, t0, bh);
                if (wide) tma_load_3d(sb + L::V_OFF + SLAB, &tmV, &full[st], dv0 + 64, t0, bh);
                bulk_load(sb + L::G_OFF, a.gates + (size_t)at * 4 * C, 4 * C * 4, &full[st]);
                tma_load_3d(sb + L::TH_OFF, &tmTh, &full[st], 0, 0, at);
                tma_load_3d(sb + L::TL_OFF, &tmTl, &full[st], 0, 0, at);
#pragma unroll
                for (int i = 0; i < DK / 64; ++i) tma_load_3d(sb + L::Q_OFF + i * SLAB, &tmQ, &full[st], 64 * i, t0, bk);
                tma_load_3d(sb + L::P_OFF, &tmP, &full[st], 0, 0, at);
                tma_load_3d(sb + L::PL_OFF, &tmPl, &full[st], 0, 0, at);
                if (m + NST < n) {
                    // the next stages' tiles on their way into L2
                    const int t1 = t0 + NST * C, a1 = at + NST;
                    prefetch_l2_tile_3d(&tmV, dv0, t1, bh);
                    if (wide) prefetch_l2_tile_3d(&tmV, dv0 + 64, t1, bh);
                    if (blockIdx.x == 0) {
#pragma unroll
                        for (int i = 0; i < DK / 64; ++i) {
                            prefetch_l2_tile_3d(&tmK, 64 * i, t1, bk);
                            prefetch_l2_tile_3d(&tmQ, 64 * i, t1, bk);
                        }
                        prefetch_l2_tile_3d(&tmTh, 0, 0, a1);
                        prefetch_l2_tile_3d(&tmTl, 0, 0, a1);
                        prefetch_l2_tile_3d(&tmP, 0, 0, a1);
                        prefetch_l2_tile_3d(&tmPl, 0, 0, a1);
                    }
                }
            }
            for (int m = max(0, issued - NST); m < issued; ++m) wait(&full[m % NST], (m / NST) & 1, abort_flag, status, ERR_TMA);
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            // The whole warp walks the loop and one elected lane issues, so that descriptors stay
            // in uniform registers (issued from a divergent lane each product took about 60 to 100
            // cycles of moves, twice its time on the tensor cores).
            const uint32_t id64 = idesc_bf16(128, 64, false, false), idS = idesc_bf16(128, DK, false, true);
            const uint32_t idV = idesc_bf16(128, 64, true, false);
            const uint32_t s0 = smem_u32(sm);
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NST;
                const uint32_t sb = s0 + st * L::STAGE, ph = m & 1;
                const uint64_t dK = sdesc(sb + L::K_OFF, 16, 1024, kSwizzle128);
                const uint64_t dQ = sdesc(sb + L::Q_OFF, 16, 1024, kSwizzle128);
                const uint64_t dTh = sdesc(sb + L::TH_OFF, 16, 1024, kSwizzle128);
                const uint64_t dTl = sdesc(sb + L::TL_OFF, 16, 1024, kSwizzle128);
                const uint64_t dP = sdesc(sb + L::P_OFF, 16, 1024, kSwizzle128);
                const uint64_t dPl = sdesc(sb + L::PL_OFF, 16, 1024, kSwizzle128);
                const uint64_t dKn = sdesc(sb + L::K_OFF, SLAB, 1024, kSwizzle128);   // keys along N
                const uint64_t dV = sdesc(sb + L::V_OFF, SLAB, 1024, kSwizzle128);    // dv along M
                wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_MMA);
                __syncwarp();
                if (elect_one()) {
                    // V^T T^T, both from shared memory, while the state's parts are still written
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint64_t o = (kk * 32) >> 4, v = (kk * 2048) >> 4;
                        mma_ss(tm + L::tX, dV + v, dTh + o, idV, kk > 0);
                        mma_ss(tm + L::tX, dV + v, dTl + o, idV, 1);
                    }
                }
                wait(s_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // (K S)^T: A the state's parts, B = K (64 tokens by keys, K-major)
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * SLAB + (kk & 3) * 32) >> 4;
                        mma_ts(tm + L::tKs, tm + L::tSh + kk * 8, dK + o, id64, kk > 0);
                        mma_ts(tm + L::tKs, tm + L::tSl + kk * 8, dK + o, id64, 1);
                    }
                    mma_commit(ks_full);
                }
                if (m > 0) wait(o_empty, (m - 1) & 1, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * SLAB + (kk & 3) * 32) >> 4;
                        mma_ts(tm + L::tOq, tm + L::tSh + kk * 8, dQ + o, id64, kk > 0);
                        mma_ts(tm + L::tOq, tm + L::tSl + kk * 8, dQ + o, id64, 1);
                    }
                }
                wait(r_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // U^T = R^T T^T: B = T (rows i, columns j: K-major)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint64_t o = (kk * 32) >> 4;
                        mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTh + o, id64, 1);
                        mma_ts(tm + L::tX, tm + L::tRl + kk * 8, dTh + o, id64, 1);
                        mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTl + o, id64, 1);
                    }
                    mma_commit(u_full);
                }
                wait(u_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // the increment (l U)^T K: B = K with the keys along N (MN-major)
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint64_t o = (kk * 2048) >> 4;
                        mma_ts(tm + L::tD, tm + L::tRh + kk * 8, dKn + o, idS, kk > 0);
                        mma_ts(tm + L::tD, tm + L::tRl + kk * 8, dKn + o, idS, 1);
                    }
                    mma_commit(d_full);
                }
                wait(p_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // (P U)^T: U's parts lie in X, 16 columns of 32 tokens each
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint32_t u = tm + L::tX + (kk >> 1) * 32 + (kk & 1) * 8;
                        mma_ts(tm + L::tOp, u, dP + ((kk * 32) >> 4), id64, kk > 0);
                        mma_ts(tm + L::tOp, u + 16, dP + ((kk * 32) >> 4), id64, 1);
                        mma_ts(tm + L::tOp, u, dPl + ((kk * 32) >> 4), id64, 1);
                    }
                    mma_commit(o_full);
                    mma_commit(&empty[st]);
                }
                __syncwarp();
            }
            // no product may still run when the tensor memory is freed
            if (elect_one()) mma_commit(fin);
            __syncwarp();
            mbar_wait(fin, 0, kTimeoutNs);
        }
    } else if (wg < 3) {
        // ---------------------------------------------------------- the chain's register steps
        regs_inc<184>();
        const int grp = wg - 1, d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const int k0 = grp * HC, i0 = grp * 32;       // this group's keys and tokens
        const bool in = dv0 + d < a.dv;
        const size_t sbase = (size_t)bh * DK * a.dv + (size_t)k0 * a.dv + dv0 + d;
        float2 s[HC / 2];
#pragma unroll
        for (int i = 0; i < HC / 2; ++i) {
            s[i].x = a.S0 && in ? a.S0[sbase + (size_t)(2 * i) * a.dv] : 0.f;
            s[i].y = a.S0 && in ? a.S0[sbase + (size_t)(2 * i + 1) * a.dv] : 0.f;
        }
        auto put_state = [&]() {
#pragma unroll
            for (int c = 0; c < HC; c += 32) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(s[c / 2 + i], hi[i], lo[i]);
                tmem_st16(tm + lb + L::tSh + (k0 + c) / 2, hi);
                tmem_st16(tm + lb + L::tSl + (k0 + c) / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_ready);
        };
        if (n > 0) put_state();
        for (int m = 0; m < n; ++m) {
            const int st = m % NST;
            const uint32_t ph = m & 1;
            const uint32_t gt = smem_u32(sm) + st * L::STAGE + L::G_OFF;
            wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_EPI);
            const float gend = lds1(gt + (2 * C - 1) * 4);
            uint32_t hi[16], lo[16];
            {
                float4 g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = lds4(gt + (3 * C + i0 + 4 * i) * 4);   // -e
                wait(ks_full, ph, abort_flag, status, ERR_EPI);
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(tm + lb + L::tKs + i0, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    split2(mul2(make_float2(g[i].x, g[i].y), f2(x[4 * i], x[4 * i + 1])), hi[2 * i], lo[2 * i]);
                    split2(mul2(make_float2(g[i].z, g[i].w), f2(x[4 * i + 2], x[4 * i + 3])), hi[2 * i + 1], lo[2 * i + 1]);
                }
                tmem_st16(tm + lb + L::tRh + i0 / 2, hi);
                tmem_st16(tm + lb + L::tRl + i0 / 2, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(r_ready);
            }
            {
                float4 g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = lds4(gt + (2 * C + i0 + 4 * i) * 4);   // l
                wait(u_full, ph, abort_flag, status, ERR_EPI);
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(tm + lb + L::tX + i0, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    split2(mul2(make_float2(g[i].x, g[i].y), f2(x[4 * i], x[4 * i + 1])), hi[2 * i], lo[2 * i]);
                    split2(mul2(make_float2(g[i].z, g[i].w), f2(x[4 * i + 2], x[4 * i + 3])), hi[2 * i + 1], lo[2 * i + 1]);
                }
                tmem_st16(tm + lb + L::tRh + i0 / 2, hi);
                tmem_st16(tm + lb + L::tRl + i0 / 2, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(u_ready);
                // U's own parts, off the chain: the increment's products run meanwhile
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(f2(x[2 * i], x[2 * i + 1]), hi[i], lo[i]);
                tmem_st16(tm + lb + L::tX + i0, hi);
                tmem_st16(tm + lb + L::tX + i0 + 16, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready);
            }
            wait(d_full, ph, abort_flag, status, ERR_EPI);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HC; c += 32) {
                uint32_t x[32];
                tmem_ld32(tm + lb + L::tD + k0 + c, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[c / 2 + i] = fma2(make_float2(gend, gend), s[c / 2 + i], f2(x[2 * i], x[2 * i + 1]));
            }
            if (m + 1 < n) put_state();
        }
        if (a.ST && in) {
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) {
                a.ST[sbase + (size_t)(2 * i) * a.dv] = s[i].x;
                a.ST[sbase + (size_t)(2 * i + 1) * a.dv] = s[i].y;
            }
        }
    } else {
        // ---------------------------------------------------------- drain of O
        regs_dec<88>();
        const int d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ob = smem_u32(sm) + L::O_OFF + (d >> 6) * SLAB + (d & 63) * 2;
        for (int m = 0; m < n; ++m) {
            const int st = m % NST;
            const uint32_t ph = m & 1;
            const uint32_t gt = smem_u32(sm) + st * L::STAGE + L::G_OFF + C * 4;   // e
            wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_DRAIN);
            wait(o_full, ph, abort_flag, status, ERR_DRAIN);
            tc_fence_after();
            // the tile's last store must have read it
            if (threadIdx.x == NT - 128) bulk_wait_read0();
            named_bar_sync(1, 128);
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                uint32_t x[16], y[16];
                float4 g[4];
                tmem_ld16(tm + lb + L::tOq + c, x);
                tmem_ld16(tm + lb + L::tOp + c, y);
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = lds4(gt + (c + 4 * i) * 4);
                tmem_wait_ld();
                auto put = [&](int i, float e) {
                    sts_bf16(ob + (c + i) * 128, fmaf(a.scale * e, __uint_as_float(x[i]), __uint_as_float(y[i])));
                };
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    put(4 * i, g[i].x); put(4 * i + 1, g[i].y); put(4 * i + 2, g[i].z); put(4 * i + 3, g[i].w);
                }
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_empty);
                mbar_arrive(&empty[st]);
            }
            named_bar_sync(1, 128);
            if (threadIdx.x == NT - 128) {
                tma_store_3d(&tmO, sm + L::O_OFF, dv0, m * C, bh);
                if (wide) tma_store_3d(&tmO, sm + L::O_OFF + SLAB, dv0 + 64, m * C, bh);
                bulk_commit();
            }
        }
        if (threadIdx.x == NT - 128) bulk_wait0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, L::TCOLS);
    }
}

template <int DK>
cudaError_t launch_dk(const DeltaChain& a, const CUtensorMap (&m)[8], int* status, cudaStream_t s)
{
    using L = CL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_chain_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const dim3 g((a.dv + DVT - 1) / DVT, (unsigned)(a.B * a.H));
    gla_delta_chain_kernel<DK><<<g, NT, L::SMEM, s>>>(a, m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaChain& a, int* status, cudaStream_t s)
{
    const uint64_t bk = (uint64_t)a.B * a.Hk, bh = (uint64_t)a.B * a.H, nc = bh * a.nch;
    CUtensorMap m[8];
    if (!map_rows(&m[0], a.k, a.dk, a.T, bk) || !map_rows(&m[1], a.q, a.dk, a.T, bk) ||
        !map_rows(&m[2], a.v, a.dv, a.T, bh) || !map_rows(&m[3], a.t_hi, C, C, nc) ||
        !map_rows(&m[4], a.t_lo, C, C, nc) || !map_rows(&m[5], a.p_hi, C, C, nc) ||
        !map_rows(&m[6], a.p_lo, C, C, nc))
        return cudaErrorInvalidValue;
    {   // O: staged without a swizzle
        const uint64_t dims[3] = {(uint64_t)a.dv, (uint64_t)a.T, bh}, str[2] = {(uint64_t)a.dv * 2, (uint64_t)a.dv * a.T * 2};
        const uint32_t box[3] = {64, C, 1};
        if (!make_tmap(&m[7], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.O, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    }
    return a.dk == 64 ? launch_dk<64>(a, m, status, s) : launch_dk<128>(a, m, status, s);
}

}  // namespace gla
