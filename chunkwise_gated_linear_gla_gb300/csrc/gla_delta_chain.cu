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
constexpr int NG = 4;             // their gates, which the drain reads for longer
constexpr int DVT = 128;          // dv columns per CTA
constexpr int PF = 2;             // chunks between a tile's prefetch into L2 and its load

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

enum { ERR_TMA = 0x611, ERR_MMA = 0x612, ERR_EPI = 0x613, ERR_DRAIN = 0x614 };

template <int DK>
struct CL {
    static constexpr int KB = (DK / 64) * SLAB;
    static constexpr int K_OFF = 0, Q_OFF = KB, V_OFF = 2 * KB, T_OFF = V_OFF + 2 * SLAB, P_OFF = T_OFF + 2 * SLAB;
    static constexpr int STAGE = P_OFF + 2 * SLAB;
    static constexpr int GB = 4 * C * 4;                  // gates of one chunk
    static constexpr int BYTES = STAGE + GB;              // of one chunk's loads
    static constexpr int O_OFF = NST * STAGE;             // [2 halves of dv][64 tokens][64] bf16
    static constexpr int G_OFF = O_OFF + 2 * SLAB;
    static constexpr int BAR_OFF = G_OFF + NG * GB;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    // tensor memory columns
    static constexpr int tD = 0;                          // the state's increment, [dv][DK]
    static constexpr int tSh = DK, tSl = tSh + DK / 2;    // the state's parts
    static constexpr int tX = 2 * DK;                     // U; then its high part
    static constexpr int tRh = tX + 64, tRl = tRh + 32;   // R's parts, then l U's
    static constexpr int tOq = tRl + 32, tOp = tOq + 64;  // Q S, P U
    // K S: over the increment's first half of the keys, read by then (no room else at dk = 128)
    static constexpr int tKs = DK == 128 ? tD : tOp + 64;
    static constexpr int TCOLS = 512;
    static_assert(tOp + 64 <= TCOLS && tKs + 64 <= TCOLS, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <int DK>
__global__ void __launch_bounds__(NT, 1)
gla_delta_chain_kernel(DeltaChain a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmT,
                       const __grid_constant__ CUtensorMap tmP,
                       const __grid_constant__ CUtensorMap tmO, int* status)
{
    using L = CL<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* full = bar;             // [NST] stage loaded
    uint64_t* empty = bar + NST;      // [NST] stage consumed
    // Every step of the chain comes in two parts (first and second half of the keys, or of the
    // tokens), so that the products of one run beside the register step of the other.
    uint64_t* s_ready = bar + 2 * NST;      // [2] state parts written (8 warps)
    uint64_t* r_ready = s_ready + 2;        // [2] R's parts written (8 warps)
    uint64_t* u_ready = s_ready + 4;        // [2] l U's parts written (8 warps)
    uint64_t* p_ready = s_ready + 6;        // U's own parts written, for P U (8 warps)
    uint64_t* ks_full = s_ready + 7;        // K S formed
    uint64_t* u_full = s_ready + 8;         // U formed
    uint64_t* d_full = s_ready + 9;         // [2] the increment formed
    uint64_t* o_full = s_ready + 11;        // Q S and P U formed
    uint64_t* fin = s_ready + 12;
    uint64_t* o_empty = s_ready + 13;       // O read out (4 warps)
    uint32_t* holder = reinterpret_cast<uint32_t*>(s_ready + 14);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(s_ready + 15);

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32, wg = warp / 4;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int dv0 = blockIdx.x * DVT;
    const bool wide = dv0 + 64 < a.dv;      // the tile's second half is inside dv
    const int n = a.nch;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 14; ++i) mbar_init(&s_ready[i], i < 7 ? 8 : i == 13 ? 4 : 1);
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
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            // (the whole warp walks the loop, an elected lane issues: as the MMA issuer below)
            int issued = 0;
            for (int m = 0; m < n; ++m, ++issued) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NST, t0 = m * C, at = bh * n + m;
                if (m >= NST) wait(&empty[st], ((m / NST) - 1) & 1, abort_flag, status, ERR_TMA);
                __syncwarp();
                uint8_t* sb = sm + st * L::STAGE;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&full[st], L::BYTES);
                    tma_load_4d(sb + L::V_OFF, &tmV, &full[st], 0, t0, dv0 / 64, bh);   // (slabs past dv: zeros)
                    tma_load_3d(sb + L::T_OFF, &tmT, &full[st], 0, 0, at);
                    tma_load_4d(sb + L::K_OFF, &tmK, &full[st], 0, t0, 0, bk);
                    bulk_load(sm + L::G_OFF + (m % NG) * L::GB, a.gates + (size_t)at * 4 * C, L::GB, &full[st]);
                    tma_load_4d(sb + L::Q_OFF, &tmQ, &full[st], 0, t0, 0, bk);
                    tma_load_3d(sb + L::P_OFF, &tmP, &full[st], 0, 0, at);
                }
                __syncwarp();
            }
            for (int m = max(0, issued - NST); m < issued; ++m) wait(&full[m % NST], (m / NST) & 1, abort_flag, status, ERR_TMA);
        } else if (warp == 2) {
            // ------------------------------------------------------ L2 prefetch, PF chunks ahead of the loads
            for (int m = 0; m + PF < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                if (m >= NST) wait(&empty[m % NST], ((m / NST) - 1) & 1, abort_flag, status, ERR_TMA);
                __syncwarp();
                const int t1 = (m + PF) * C, a1 = bh * n + m + PF;
                if (elect_one()) {
                    prefetch_l2_tile_4d(&tmV, 0, t1, dv0 / 64, bh);
                    if (blockIdx.x == 0) {
                        prefetch_l2_tile_3d(&tmT, 0, 0, a1);
                        prefetch_l2_tile_4d(&tmK, 0, t1, 0, bk);
                        prefetch_l2_tile_4d(&tmQ, 0, t1, 0, bk);
                        prefetch_l2_tile_3d(&tmP, 0, 0, a1);
                    }
                }
                __syncwarp();
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            // The whole warp walks the loop and one elected lane issues, so that descriptors stay
            // in uniform registers (issued from a divergent lane each product took about 60 to 100
            // cycles of moves, twice its time on the tensor cores).
            const uint32_t id64 = idesc_bf16(128, 64, false, false), idS = idesc_bf16(128, DK, false, true);
            const uint32_t idV = idesc_bf16(128, 64, true, false), idH = idesc_bf16(128, 64, false, true);
            const uint32_t s0 = smem_u32(sm);
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NST;
                const uint32_t sb = s0 + st * L::STAGE, ph = m & 1;
                const uint64_t dK = sdesc(sb + L::K_OFF, 16, 1024, kSwizzle128);
                const uint64_t dQ = sdesc(sb + L::Q_OFF, 16, 1024, kSwizzle128);
                const uint64_t dTh = sdesc(sb + L::T_OFF, 16, 1024, kSwizzle128);
                const uint64_t dTl = sdesc(sb + L::T_OFF + SLAB, 16, 1024, kSwizzle128);
                const uint64_t dP = sdesc(sb + L::P_OFF, 16, 1024, kSwizzle128);
                const uint64_t dPl = sdesc(sb + L::P_OFF + SLAB, 16, 1024, kSwizzle128);
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
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&s_ready[part], ph, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
                        // (K S)^T: A the state's parts, B = K (64 tokens by keys, K-major)
#pragma unroll
                        for (int kk = part * (DK / 32); kk < (part + 1) * (DK / 32); ++kk) {
                            const uint64_t o = ((kk >> 2) * SLAB + (kk & 3) * 32) >> 4;
                            mma_ts(tm + L::tKs, tm + L::tSh + kk * 8, dK + o, id64, kk > 0);
                            mma_ts(tm + L::tKs, tm + L::tSl + kk * 8, dK + o, id64, 1);
                        }
                        if (part) mma_commit(ks_full);
                    }
                }
                // (Q S)^T in two halves, in the gaps that R's and U's register steps leave
                auto qs = [&](uint32_t s, uint32_t first) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk)
                        mma_ts(tm + L::tOq, tm + s + kk * 8, dQ + (((kk >> 2) * SLAB + (kk & 3) * 32) >> 4), id64,
                               !first || kk > 0);
                };
                if (m > 0) wait(o_empty, (m - 1) & 1, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) qs(L::tSh, 1);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&r_ready[part], ph, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
                        // U^T += R^T T^T: B = T (rows i, columns j: K-major)
#pragma unroll
                        for (int kk = 2 * part; kk < 2 * part + 2; ++kk) {
                            const uint64_t o = (kk * 32) >> 4;
                            mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTh + o, id64, 1);
                            mma_ts(tm + L::tX, tm + L::tRl + kk * 8, dTh + o, id64, 1);
                            mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTl + o, id64, 1);
                        }
                        if (part) {
                            mma_commit(u_full);
                            qs(L::tSl, 0);
                        }
                    }
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&u_ready[part], ph, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
                        // the increment (l U)^T K: B = K with the keys along N (MN-major); the second
                        // part's products one half of the keys after the other (dk = 128: a slab each)
                        constexpr int NH = DK == 128 ? 2 : 1;
#pragma unroll
                        for (int nh = 0; nh < (part ? NH : 1); ++nh) {
#pragma unroll
                            for (int kk = 2 * part; kk < 2 * part + 2; ++kk) {
                                const uint64_t o = (kk * 2048 + nh * SLAB) >> 4;
                                const uint32_t id = part && NH == 2 ? idH : idS;
                                mma_ts(tm + L::tD + nh * 64, tm + L::tRh + kk * 8, dKn + o, id, kk > 0);
                                mma_ts(tm + L::tD + nh * 64, tm + L::tRl + kk * 8, dKn + o, id, 1);
                            }
                            if (part) mma_commit(&d_full[nh]);
                        }
                        if (part && NH == 1) mma_commit(&d_full[1]);
                    }
                }
                wait(p_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // (P U)^T: U's parts lie in X, eight columns each in the place of 16 tokens
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint32_t u = tm + L::tX + kk * 16;
                        mma_ts(tm + L::tOp, u, dP + ((kk * 32) >> 4), id64, kk > 0);
                        mma_ts(tm + L::tOp, u + 8, dP + ((kk * 32) >> 4), id64, 1);
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
        // Group g owns, of part p, the keys p DK/2 + g DK/4 .. and the tokens 32 p + 16 g ..
        constexpr int KP = DK / 4;                    // keys of one part
        const int grp = wg - 1, d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const bool in = dv0 + d < a.dv;
        const size_t sbase = (size_t)bh * DK * a.dv + dv0 + d;
        auto key = [&](int p) { return p * (DK / 2) + grp * KP; };
        auto signal = [&](uint64_t* b) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b);
        };
        float2 s[2][KP / 2];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int i = 0; i < KP / 2; ++i) {
                const size_t at = sbase + (size_t)(key(p) + 2 * i) * a.dv;
                s[p][i].x = a.S0 && in ? a.S0[at] : 0.f;
                s[p][i].y = a.S0 && in ? a.S0[at + a.dv] : 0.f;
            }
        auto put_state = [&](int p) {
            uint32_t hi[KP / 2], lo[KP / 2];
#pragma unroll
            for (int i = 0; i < KP / 2; ++i) split2(s[p][i], hi[i], lo[i]);
#pragma unroll
            for (int i = 0; i < KP / 2; i += 8) {
                tmem_st8(tm + lb + L::tSh + key(p) / 2 + i, hi + i);
                tmem_st8(tm + lb + L::tSl + key(p) / 2 + i, lo + i);
            }
            signal(&s_ready[p]);
        };
        if (n > 0) {
            put_state(0);
            put_state(1);
        }
        for (int m = 0; m < n; ++m) {
            const int st = m % NST;
            const uint32_t ph = m & 1;
            const uint32_t gt = smem_u32(sm) + L::G_OFF + (m % NG) * L::GB;
            wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_EPI);
            const float gend = lds1(gt + (2 * C - 1) * 4);
            float4 g[8];
            auto gates = [&](int row) {
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = lds4(gt + (row * C + (i >> 2) * 32 + grp * 16 + 4 * (i & 3)) * 4);
            };
            // 16 tokens of part p times their gate, in two parts, to R's place
            auto put_tokens = [&](int p, const uint32_t (&x)[16]) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 e = g[4 * p + i];
                    split2(mul2(make_float2(e.x, e.y), f2(x[4 * i], x[4 * i + 1])), hi[2 * i], lo[2 * i]);
                    split2(mul2(make_float2(e.z, e.w), f2(x[4 * i + 2], x[4 * i + 3])), hi[2 * i + 1], lo[2 * i + 1]);
                }
                tmem_st8(tm + lb + L::tRh + p * 16 + grp * 8, hi);
                tmem_st8(tm + lb + L::tRl + p * 16 + grp * 8, lo);
            };
            uint32_t x0[16], x1[16];
            gates(3);                                 // -e
            wait(ks_full, ph, abort_flag, status, ERR_EPI);
            tc_fence_after();
            tmem_ld16(tm + lb + L::tKs + grp * 16, x0);
            tmem_ld16(tm + lb + L::tKs + 32 + grp * 16, x1);
            tmem_wait_ld();
            put_tokens(0, x0);
            signal(&r_ready[0]);
            put_tokens(1, x1);
            signal(&r_ready[1]);
            gates(2);                                 // l
            wait(u_full, ph, abort_flag, status, ERR_EPI);
            tc_fence_after();
            tmem_ld16(tm + lb + L::tX + grp * 16, x0);
            tmem_ld16(tm + lb + L::tX + 32 + grp * 16, x1);
            tmem_wait_ld();
            put_tokens(0, x0);
            signal(&u_ready[0]);
            put_tokens(1, x1);
            signal(&u_ready[1]);
            // U's own parts, off the chain: the increment's products run meanwhile
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    split2(p ? f2(x1[2 * i], x1[2 * i + 1]) : f2(x0[2 * i], x0[2 * i + 1]), hi[i], lo[i]);
                tmem_st8(tm + lb + L::tX + p * 32 + grp * 16, hi);
                tmem_st8(tm + lb + L::tX + p * 32 + grp * 16 + 8, lo);
            }
            signal(p_ready);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                wait(&d_full[p], ph, abort_flag, status, ERR_EPI);
                tc_fence_after();
                uint32_t x[KP];
#pragma unroll
                for (int c = 0; c < KP; c += 16)
                    tmem_ld16(tm + lb + L::tD + key(p) + c, *reinterpret_cast<uint32_t(*)[16]>(x + c));
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < KP / 2; ++i)
                    s[p][i] = fma2(make_float2(gend, gend), s[p][i], f2(x[2 * i], x[2 * i + 1]));
                if (m + 1 < n) put_state(p);
            }
        }
        if (a.ST && in) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < KP / 2; ++i) {
                    const size_t at = sbase + (size_t)(key(p) + 2 * i) * a.dv;
                    a.ST[at] = s[p][i].x;
                    a.ST[at + a.dv] = s[p][i].y;
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
            const uint32_t gt = smem_u32(sm) + L::G_OFF + (m % NG) * L::GB + C * 4;   // e
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
            if (lane == 0) mbar_arrive(o_empty);
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
cudaError_t launch_dk(const DeltaChain& a, const CUtensorMap (&m)[6], int* status, cudaStream_t s)
{
    using L = CL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_chain_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const dim3 g((a.dv + DVT - 1) / DVT, (unsigned)(a.B * a.H));
    gla_delta_chain_kernel<DK><<<g, NT, L::SMEM, s>>>(a, m[0], m[1], m[2], m[3], m[4], m[5], status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaChain& a, int* status, cudaStream_t s)
{
    const uint64_t bk = (uint64_t)a.B * a.Hk, bh = (uint64_t)a.B * a.H, nc = bh * a.nch;
    CUtensorMap m[6];
    if (!map_slabs(&m[0], a.k, a.dk, a.T, bk, a.dk / 64) || !map_slabs(&m[1], a.q, a.dk, a.T, bk, a.dk / 64) ||
        !map_slabs(&m[2], a.v, a.dv, a.T, bh, 2) || !map_pair(&m[3], a.t, nc) || !map_pair(&m[4], a.p, nc))
        return cudaErrorInvalidValue;
    {   // O: staged without a swizzle
        const uint64_t dims[3] = {(uint64_t)a.dv, (uint64_t)a.T, bh}, str[2] = {(uint64_t)a.dv * 2, (uint64_t)a.dv * a.T * 2};
        const uint32_t box[3] = {64, C, 1};
        if (!make_tmap(&m[5], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.O, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    }
    return a.dk == 64 ? launch_dk<64>(a, m, status, s) : launch_dk<128>(a, m, status, s);
}

}  // namespace gla
