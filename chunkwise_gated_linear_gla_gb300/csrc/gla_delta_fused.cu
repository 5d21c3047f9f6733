// gla_delta_fused: the whole chunk form of the gated delta rule in one kernel. Per 64-token chunk,
// with G the running sum of log_g in the chunk, e = exp(G), l = exp(G_end - G), D_ij = exp(G_i - G_j):
//
//   L_ij = (k_i . k_j) D_ij (j < i),   T = (1 / beta + L)^-1,   P_ij = scale (q_i . k_j) D_ij (j <= i),
//   R = -e K S,   U = T V + T R,   O = scale e (Q S) + P U,   S <- exp(G_end) S + K^T (l U).
//
// (U solves u_i = beta_i (v_i - e_i k_i S - sum_{j<i} L_ij u_j).) A CTA owns 128 columns of dv of one
// head (and of one segment of the sequence) and walks the chunks; T and P never leave the SM.
//
// The chain (four warpgroups' warps 4-11, products by warp 1). Everything is transposed, dv along the
// 128 tensor-memory lanes: the state, R and U are A operands read from tensor memory and a thread owns
// one column of dv, so nothing of the chain passes through shared memory; the state itself stays in
// fp32 registers. Every step comes in two halves (of the keys, or of the tokens), so that the
// products of one run beside the register step of the other. Every operand that is not an input (S,
// R, U, T, P) goes into the products in two bf16 parts, hi + lo, good to 2^-17; K, V and Q are exact:
// two products for K S, K^T U, Q S and T V, three for T R and P U. So the fp32 state is good to 3e-6 (4e-6
// without a gate; nearly all of it l U's rounding: with three parts of that 8e-7, the layer below 111 us)
// and O to its last rounding (with one part of P and U it was not: where keys repeat, P U is a sum of
// cancelling terms, 7.5e-3 off when all keys are the same).
//
// The prep (warps 16-23) runs one chunk ahead on the same SM: one product of 128 rows, K stacked on
// Q, against K^T; the masked L and P; then T in place of L: 8-row diagonal blocks by forward
// substitution in fp32, then three times the block rule, the inverse of [[X^-1, 0], [C, Y^-1]] has -Y C X
// below: once more in fp32, then on mma.sync fragments in two parts (16 x 16 and 32 x 32 pieces, too
// small for a tcgen05 tile). G is summed in pairs of floats (48 bits), so a steep gate costs no precision; D is a product
// of two factors around the chunk's middle while both stay within e^60, else one exponential per pair.
//
// Warps: 0 TMA, 1 products, 3 gates, 4-11 chain, 12-15 drain of O, 16-23 prep. Reads K, Q, V once
// and writes O once. 8 x 2048 tokens, 16 heads, dk = dv = 128: 103 us, 2.8 TB/s, 6100 cycles a chunk, of
// which the chain and the prep each need about as many: with the tensor pipe busy 51% and the issue slots
// 49% of the time, neither shortens the other by more warps (16 for the chain: 107 us; scores and inverse
// on eight warps each, a chunk apart: 110 us).
#include "gla_delta_dev.cuh"
#include "gla_delta_tri.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 768;
constexpr int NKQ = 3;            // K and Q stages: chunk m's, the next one's (read by the prep), one in flight
constexpr int NV = 2;             // V stages, T and P buffers
constexpr int NG = 4;             // gate slots (the drain is the last reader)
constexpr int DVT = 128;          // dv columns per CTA

enum { ERR_TMA = 0x641, ERR_MMA = 0x642, ERR_EPI = 0x643, ERR_DRAIN = 0x644, ERR_PREP = 0x645 };

template <int DK>
struct FL {
    static constexpr int KB = (DK / 64) * SLAB;
    static constexpr int KQ_OFF = 0;                       // [NKQ][K, Q]
    static constexpr int V_OFF = NKQ * 2 * KB;             // [NV]
    static constexpr int TP_OFF = V_OFF + NV * 2 * SLAB;   // [NV][T, T_lo, P, P_lo]
    static constexpr int O_OFF = TP_OFF + NV * 4 * SLAB;   // [2 halves of dv][64 tokens][64] bf16
    static constexpr int GB = 8 * C * 4;                   // beta, e, l, -e, the factors of D, G in two floats
    static constexpr int G_OFF = O_OFF + 2 * SLAB;
    static constexpr int W_OFF = G_OFF + NG * GB;          // 32 rows of [32 values, their low parts]
    static constexpr int D_OFF = W_OFF + 32 * 128;         // diagonal blocks of beta L, fp32
    static constexpr int BAR_OFF = D_OFF + 4 * 16 * LDD * 4;
    static constexpr int SMEM = BAR_OFF + 320 + 1024;
    // tensor memory columns
    static constexpr int tD = 0;                           // the state's increment, [dv][DK]
    static constexpr int tSh = DK, tSl = tSh + DK / 2;     // the state's parts
    static constexpr int tX = 2 * DK;                      // U; then its parts
    static constexpr int tRh = tX + 64, tRl = tRh + 32;    // R's parts, then l U's
    static constexpr int tOq = tRl + 32, tOp = tOq + 64;   // Q S, P U
    // K S and the prep's product: at dk = 128 over the increment's two halves, which are read
    // before the one is formed and not formed again before the other is read
    static constexpr int tKs = DK == 128 ? tD : tOp + 64, tG = DK == 128 ? tD + 64 : tOp + 128;
    static_assert(tG + 64 <= 512 && tOp + 64 <= 512 && tKs + 64 <= 512, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct FusedArgs {
    const float* log_g; const __nv_bfloat16* beta;
    const float* S_in; float* S_out;      // + bh * s_bh + segment * s_seg
    long long in_bh, in_seg, out_bh, out_seg;
    int H, Hk, T, dv, nch, cps, nseg, per, tiles;   // without O cps are the chunks of `per` segments
    float scale;
    int* status;
};
struct FusedMaps { CUtensorMap k, q, v, o; };

// OUT: O is formed (and its products and drain run). Without it the state alone, from zero, and in the
// tiles after dv's the state that starts from the identity without V: the segment's transition. Its scores are L
// alone and are formed on the drain's warps, two chunks ahead, in P U's place, while the prep's warps form T
// one chunk ahead: 2.4 us a chunk against 2.7 with both on the prep's warps (with O there is no such place:
// the product lies over the increment's second half for as long as that is free).
template <int DK, bool OUT>
__global__ void __launch_bounds__(NT, 1)
gla_delta_fused_kernel(FusedArgs a, const __grid_constant__ FusedMaps mp)
{
    using L = FL<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* kq_full = bar;                // [NKQ]
    uint64_t* kq_empty = bar + NKQ;         // [NKQ]
    uint64_t* v_full = kq_empty + NKQ;      // [NV]
    uint64_t* v_empty = v_full + NV;        // [NV]
    uint64_t* s_ready = v_empty + NV;       // [2] state parts written (8 warps)
    uint64_t* r_ready = s_ready + 2;        // [2] R's parts written (8 warps)
    uint64_t* u_ready = s_ready + 4;        // [2] l U's parts written (8 warps)
    uint64_t* p_ready = s_ready + 6;        // U's own parts written, for P U (8 warps)
    uint64_t* g_read = s_ready + 7;         // the prep's product read (8 warps)
    uint64_t* t_ready = s_ready + 8;        // [2] a chunk's T, P and gates written (8 warps), even and odd chunks
    uint64_t* ks_full = s_ready + 10;       // K S formed
    uint64_t* u_full = s_ready + 11;        // U formed
    uint64_t* d_full = s_ready + 12;        // [2] the increment formed
    uint64_t* o_full = s_ready + 14;        // Q S and P U formed
    uint64_t* g_full = s_ready + 15;        // the prep's product formed
    uint64_t* fin = s_ready + 16;
    uint64_t* o_empty = s_ready + 17;       // O read out (4 warps)
    uint64_t* gt_ready = s_ready + 18;      // [NG] a chunk's gates written
    uint64_t* l_ready = gt_ready + NG;      // without O: L written (4 warps)
    uint64_t* d_free = l_ready + 1;         // and its diagonal blocks done with
    uint64_t* gt_free = l_ready + 2;        // [NG] a chunk's gates read by everyone (4 warps; without O 8)
    uint32_t* holder = reinterpret_cast<uint32_t*>(gt_free + NG);
    const Abort abort_flag(gt_free + NG + 1);
    static_assert((2 * NKQ + 2 * NV + 18 + 2 * NG + 4) * 8 <= 320, "barriers");
    const uint32_t tG = OUT ? L::tG : L::tOp;

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32, wg = warp / 4;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int seg = blockIdx.z, first = seg * a.cps, n = min(a.nch - first, a.cps);
    const bool ident = !OUT && (int)blockIdx.x >= a.tiles;
    const int dv0 = ident ? 0 : blockIdx.x * DVT;
    const bool wide = dv0 + 64 < a.dv;      // the tile's second half is inside dv

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * NKQ + 2 * NV; ++i) mbar_init(&bar[i], 1);
        for (int i = 0; i < 20 + 2 * NG; ++i) mbar_init(&s_ready[i], i == 7 && !OUT ? 4 : i < 10 ? 8 : i == 17 || i == 18 + NG || (OUT && i >= 20 + NG) ? 4 : i >= 20 + NG ? 8 : 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *holder;
    int* status = a.status;

    if (wg == 0) {
        regs_dec<48>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            int kq = 0, v = 0;
            bool ok = true;                 // this lane's waits so far have come to their ends
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int t0 = (first + m) * C, st = m % NKQ;
                if (m >= NKQ) ok &= wait(&kq_empty[st], ((m / NKQ) - 1) & 1, abort_flag, status, ERR_TMA);
                __syncwarp();
                if (elect_one() && ok) {
                    // K's and Q's slab of the same 64 keys side by side: 128 rows of one operand (without O
                    // K's twice, so that two warps read the product's longer rows)
                    mbar_arrive_expect_tx(&kq_full[st], 2 * L::KB);
                    uint8_t* sb = sm + L::KQ_OFF + st * 2 * L::KB;
#pragma unroll
                    for (int i = 0; i < DK / 64; ++i) {
                        tma_load_3d(sb + 2 * i * SLAB, &mp.k, &kq_full[st], 64 * i, t0, bk);
                        tma_load_3d(sb + (2 * i + 1) * SLAB, OUT ? &mp.q : &mp.k, &kq_full[st], 64 * i, t0, bk);
                    }
                }
                __syncwarp();
                kq += ok;
                if (ident) continue;
                if (m >= NV) ok &= wait(&v_empty[m % NV], ((m / NV) - 1) & 1, abort_flag, status, ERR_TMA);
                __syncwarp();
                if (elect_one() && ok) {
                    mbar_arrive_expect_tx(&v_full[m % NV], 2 * SLAB);
                    // (slabs past dv: zeros)
                    tma_load_4d(sm + L::V_OFF + (m % NV) * 2 * SLAB, &mp.v, &v_full[m % NV], 0, t0, dv0 / 64, bh);
                }
                __syncwarp();
                v += ok;
            }
            // no copy may land after the CTA has ended
            if (elect_one()) {
                for (int m = max(0, kq - NKQ); m < kq; ++m) mbar_wait(&kq_full[m % NKQ], (m / NKQ) & 1, kTimeoutNs);
                for (int m = max(0, v - NV); m < v; ++m) mbar_wait(&v_full[m % NV], (m / NV) & 1, kTimeoutNs);
            }
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------ gates, up to NG chunks ahead
            const float* lg = a.log_g ? a.log_g + (size_t)bh * a.T : nullptr;
            const __nv_bfloat16* bp = a.beta + (size_t)bh * a.T;
            float x0, x1, b0, b1;                           // two tokens of the next chunk
            auto fetch = [&](int m) {
                const int t = (first + m) * C + 2 * lane;
                const bool p = t < a.T, q = t + 1 < a.T;    // tokens past T: no decay, beta 0
                x0 = lg && p ? lg[t] : 0.f;
                x1 = lg && q ? lg[t + 1] : 0.f;
                b0 = p ? __bfloat162float(bp[t]) : 0.f;
                b1 = q ? __bfloat162float(bp[t + 1]) : 0.f;
            };
            if (n > 0) fetch(0);
            for (int m = 0; m < n; ++m) {
                // A slot's barrier cannot get ahead of this wait: its next phase is chunk m's own. (One that also
                // counts the chunks between could: two of them done and a wait by parity sees the third's, which
                // cannot complete without chunk m's gates.)
                const bool ok = m < NG || wait(&gt_free[m % NG], ((m / NG) - 1) & 1, abort_flag, status, ERR_PREP);
                if (!__all_sync(~0u, ok)) break;
                chunk_gates(x0, x1, b0, b1, sm + L::G_OFF + (m % NG) * L::GB);
                __syncwarp();
                if (lane == 0) mbar_arrive(&gt_ready[m % NG]);
                if (m + 1 < n) fetch(m + 1);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ products
            // The whole warp walks the loop and one elected lane issues, so that descriptors stay
            // in uniform registers (issued from a divergent lane each product took 60 to 100
            // cycles of moves, twice its time on the tensor cores).
            const uint32_t id64 = idesc_bf16(128, 64, false, false), idS = idesc_bf16(128, DK, false, true);
            const uint32_t idV = idesc_bf16(128, 64, true, false), idH = idesc_bf16(128, 64, false, true);
            // chunk m's K on Q (128 rows) against K
            auto gram = [&](int m) {
                const int st = m % NKQ;
                wait(&kq_full[st], (m / NKQ) & 1, abort_flag, status, ERR_MMA);
                __syncwarp();
                if (elect_one()) {
                    const uint64_t d0 = sdesc(s0 + L::KQ_OFF + st * 2 * L::KB, 16, 1024, kSwizzle128);
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t d = d0 + (((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4);
                        mma_ss(tm + tG, d, d, id64, kk > 0);
                    }
                    mma_commit(g_full);
                }
                __syncwarp();
            };
            if (n > 0) gram(0);
            if (!OUT && n > 1) {
                wait(g_read, 0, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                gram(1);
            }
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NKQ, vt = m % NV;
                const uint32_t sb = s0 + L::KQ_OFF + st * 2 * L::KB, tp = s0 + L::TP_OFF + vt * 4 * SLAB, ph = m & 1;
                const uint64_t dK = sdesc(sb, 16, 1024, kSwizzle128), dQ = sdesc(sb + SLAB, 16, 1024, kSwizzle128);
                const uint64_t dKn = sdesc(sb, 2 * SLAB, 1024, kSwizzle128);          // keys along N
                const uint64_t dV = sdesc(s0 + L::V_OFF + vt * 2 * SLAB, SLAB, 1024, kSwizzle128);   // dv along M
                const uint64_t dTh = sdesc(tp, 16, 1024, kSwizzle128), dTl = sdesc(tp + SLAB, 16, 1024, kSwizzle128);
                const uint64_t dP = sdesc(tp + 2 * SLAB, 16, 1024, kSwizzle128), dPl = sdesc(tp + 3 * SLAB, 16, 1024, kSwizzle128);
                // (K S)^T: A the state's parts, B = K (64 tokens by keys, K-major)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&s_ready[part], ph, abort_flag, status, ERR_MMA);
                    // (the first product's buffer: chunk 0's product has been read by then)
                    if (OUT && part == 0 && m == 0) wait(g_read, 0, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = part * (DK / 32); kk < (part + 1) * (DK / 32); ++kk) {
                            const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4;
                            mma_ts(tm + L::tKs, tm + L::tSh + kk * 8, dK + o, id64, kk > 0);
                            mma_ts(tm + L::tKs, tm + L::tSl + kk * 8, dK + o, id64, 1);
                        }
                        if (part) mma_commit(ks_full);
                    }
                    __syncwarp();
                }
                // the next chunk's K on Q against K, then V^T T^T, in the gap of R's register step
                if (OUT && m + 1 < n) gram(m + 1);
                wait(&t_ready[m & 1], (m >> 1) & 1, abort_flag, status, ERR_MMA);
                if (!ident) {
                    wait(&v_full[vt], (m / NV) & 1, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk) {
                            const uint64_t o = (kk * 32) >> 4, v = (kk * 2048) >> 4;
                            mma_ss(tm + L::tX, dV + v, dTh + o, idV, kk > 0);
                            mma_ss(tm + L::tX, dV + v, dTl + o, idV, 1);
                        }
                        mma_commit(&v_empty[vt]);
                    }
                    __syncwarp();
                }
                // U^T += R^T T^T: B = T (rows i, columns j: K-major)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    wait(&r_ready[part], ph, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 2 * part; kk < 2 * part + 2; ++kk) {
                            const uint64_t o = (kk * 32) >> 4;
                            mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTh + o, id64, !ident || kk > 0);
                            mma_ts(tm + L::tX, tm + L::tRl + kk * 8, dTh + o, id64, 1);
                            mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTl + o, id64, 1);
                        }
                        if (part) mma_commit(u_full);
                    }
                    __syncwarp();
                }
                if (OUT) {
                    // (Q S)^T in the gap of U's register step
                    if (m > 0) wait(o_empty, (m - 1) & 1, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < DK / 16; ++kk) {
                            const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4;
                            mma_ts(tm + L::tOq, tm + L::tSh + kk * 8, dQ + o, id64, kk > 0);
                            mma_ts(tm + L::tOq, tm + L::tSl + kk * 8, dQ + o, id64, 1);
                        }
                    }
                    __syncwarp();
                }
                if (OUT && m + 1 < n) wait(g_read, (m + 1) & 1, abort_flag, status, ERR_MMA);
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
                                const uint64_t o = (kk * 2048 + nh * 2 * SLAB) >> 4;
                                const uint32_t id = part && NH == 2 ? idH : idS;
                                mma_ts(tm + L::tD + nh * 64, tm + L::tRh + kk * 8, dKn + o, id, kk > 0);
                                mma_ts(tm + L::tD + nh * 64, tm + L::tRl + kk * 8, dKn + o, id, 1);
                            }
                            if (part) mma_commit(&d_full[nh]);
                        }
                        if (part && NH == 1) mma_commit(&d_full[1]);
                        if (part && !OUT) mma_commit(&kq_empty[st]);
                    }
                    __syncwarp();
                }
                if (!OUT && m + 2 < n) {
                    // the scores are two chunks ahead; once their product is formed T's slot has been read
                    wait(g_read, (m + 1) & 1, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    gram(m + 2);
                }
                if (OUT) {
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
                        mma_commit(&kq_empty[st]);
                    }
                    __syncwarp();
                }
            }
            // no product may still run when the tensor memory is freed
            if (elect_one()) mma_commit(fin);
            __syncwarp();
            mbar_wait(fin, 0, kTimeoutNs);
        }
    } else if (wg < 3) {
        // ---------------------------------------------------------- the chain's register steps
        // Group g owns, of part p, the keys p DK/2 + g DK/4 .. and the tokens 32 p + 16 g ..
        regs_inc<OUT ? 128 : 120>();
        constexpr int KP = DK / 4;                    // keys of one part
        const int grp = wg - 1, d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const int dvs = ident ? DK : a.dv;            // columns of the state's rows in memory
        const bool in = dv0 + d < dvs;
        const size_t sbase = (size_t)dv0 + d;
        auto key = [&](int p) { return p * (DK / 2) + grp * KP; };
        auto signal = [&](uint64_t* x) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(x);
        };
        float2 s[2][KP / 2];
        {
            const float* S = a.S_in ? a.S_in + bh * a.in_bh + seg * a.in_seg : nullptr;
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < KP / 2; ++i) {
                    const int k = key(p) + 2 * i;
                    if (!OUT) s[p][i] = make_float2(ident && k == d ? 1.f : 0.f, ident && k + 1 == d ? 1.f : 0.f);
                    else s[p][i] = S && in ? make_float2(S[sbase + (size_t)k * a.dv], S[sbase + (size_t)(k + 1) * a.dv])
                                           : make_float2(0.f, 0.f);
                }
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
        // to pair j (without O: a transition lies after the states)
        auto put_out = [&](int j) {
            if (!a.S_out || !in) return;
            float* S = a.S_out + bh * a.out_bh + j * a.out_seg + (ident ? (size_t)DK * a.dv : 0);
            int w = dvs;
            asm volatile("" : "+r"(w));              // (64 addresses, not to be kept over the chunks)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int i = 0; i < KP / 2; ++i) {
                    float* o = S + sbase + (size_t)(key(p) + 2 * i) * w;
                    o[0] = s[p][i].x;
                    o[w] = s[p][i].y;
                }
        };
        if (n > 0) {
            put_state(0);
            put_state(1);
        }
        for (int m = 0; m < n; ++m) {
            if (__any_sync(~0u, *abort_flag)) break;
            const uint32_t ph = m & 1;
            const uint32_t gt = s0 + L::G_OFF + (m % NG) * L::GB;
            wait(&t_ready[m & 1], (m >> 1) & 1, abort_flag, status, ERR_EPI);
            const float gend = lds1(gt + (2 * C - 1) * 4);
            // 16 tokens of part p times their gate (a row of the gates), in two parts, to R's place
            auto put_tokens = [&](int p, const uint32_t (&x)[16], int row) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 e = lds4(gt + (row * C + p * 32 + grp * 16 + 4 * i) * 4);
                    split2(mul2(make_float2(e.x, e.y), f2(x[4 * i], x[4 * i + 1])), hi[2 * i], lo[2 * i]);
                    split2(mul2(make_float2(e.z, e.w), f2(x[4 * i + 2], x[4 * i + 3])), hi[2 * i + 1], lo[2 * i + 1]);
                }
                tmem_st8(tm + lb + L::tRh + p * 16 + grp * 8, hi);
                tmem_st8(tm + lb + L::tRl + p * 16 + grp * 8, lo);
            };
            uint32_t x0[16], x1[16];
            wait(ks_full, ph, abort_flag, status, ERR_EPI);
            tc_fence_after();
            tmem_ld16(tm + lb + L::tKs + grp * 16, x0);
            tmem_ld16(tm + lb + L::tKs + 32 + grp * 16, x1);
            tmem_wait_ld();
            put_tokens(0, x0, 3);         // -e
            signal(&r_ready[0]);
            put_tokens(1, x1, 3);
            signal(&r_ready[1]);
            wait(u_full, ph, abort_flag, status, ERR_EPI);
            tc_fence_after();
            tmem_ld16(tm + lb + L::tX + grp * 16, x0);
            tmem_ld16(tm + lb + L::tX + 32 + grp * 16, x1);
            tmem_wait_ld();
            put_tokens(0, x0, 2);         // l
            signal(&u_ready[0]);
            put_tokens(1, x1, 2);
            signal(&u_ready[1]);
            if (!OUT && lane == 0) mbar_arrive(&gt_free[m % NG]);    // (without O the chain is the last reader)
            if (OUT) {
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
            }
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
            // the first of two segments
            if (!OUT && a.per == 2 && m + 1 == a.cps / 2 && m + 1 < n) put_out(2 * seg);
        }
        // the state after the last segment; without O every segment's
        if (!OUT) put_out(seg * a.per + (a.per == 2 && n > a.cps / 2));
        else if (seg == a.nseg - 1) put_out(0);
    } else if (wg == 3) {
        // ---------------------------------------------------------- drain of O; without O, the scores
        regs_dec<OUT ? 48 : 64>();
        if (!OUT) {
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const float* gt = reinterpret_cast<const float*>(sm + L::G_OFF + (m % NG) * L::GB);
                float* diag = reinterpret_cast<float*>(sm + L::D_OFF);
                wait(&gt_ready[m % NG], (m / NG) & 1, abort_flag, status, ERR_PREP);
                wait(g_full, m & 1, abort_flag, status, ERR_PREP);
                if (m > 0) wait(d_free, (m - 1) & 1, abort_flag, status, ERR_PREP);
                tc_fence_after();
                // lanes 0-63: L's columns 0-31, 64-127: columns 32-63
                chunk_scores<true>(tm + tG, gt, 1.f, s0 + L::TP_OFF + (m % NV) * 4 * SLAB, diag, (warp & 3) + (warp & 2) * 2);
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(g_read);
                    mbar_arrive(l_ready);
                }
            }
        }
        if (OUT) {
            const int d = (warp & 3) * 32 + lane;
            const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t ob = s0 + L::O_OFF + (d >> 6) * SLAB + (d & 63) * 2;
            const bool lead = threadIdx.x == 384;
            for (int m = 0; m < n; ++m) {
                const uint32_t gt = s0 + L::G_OFF + (m % NG) * L::GB + C * 4;   // e
                wait(o_full, m & 1, abort_flag, status, ERR_DRAIN);
                tc_fence_after();
                // the tile's last store must have read it
                if (lead) bulk_wait_read0();
                if (named_bar_any(1, 128, *abort_flag)) break;
#pragma unroll 1
                for (int c = 0; c < 64; c += 16) {
                    uint32_t x[16], y[16];
                    tmem_ld16(tm + lb + L::tOq + c, x);
                    tmem_ld16(tm + lb + L::tOp + c, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 g = lds4(gt + (c + i) * 4);
                        sts_bf16(ob + (c + i) * 128, fmaf(a.scale * g.x, __uint_as_float(x[i]), __uint_as_float(y[i])));
                        sts_bf16(ob + (c + i + 1) * 128, fmaf(a.scale * g.y, __uint_as_float(x[i + 1]), __uint_as_float(y[i + 1])));
                        sts_bf16(ob + (c + i + 2) * 128, fmaf(a.scale * g.z, __uint_as_float(x[i + 2]), __uint_as_float(y[i + 2])));
                        sts_bf16(ob + (c + i + 3) * 128, fmaf(a.scale * g.w, __uint_as_float(x[i + 3]), __uint_as_float(y[i + 3])));
                    }
                }
                tc_fence_before();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(o_empty);
                    mbar_arrive(&gt_free[m % NG]);    // (the last reader of a chunk's gates)
                }
                named_bar_sync(1, 128);
                if (lead) {
                    tma_store_3d(&mp.o, sm + L::O_OFF, dv0, (first + m) * C, bh);
                    if (wide) tma_store_3d(&mp.o, sm + L::O_OFF + SLAB, dv0 + 64, (first + m) * C, bh);
                    bulk_commit();
                }
            }
            if (lead) bulk_wait0();
        }
    } else {
        // ---------------------------------------------------------- prep, one chunk ahead
        regs_dec<64>();
        const int pw = warp - 16;
        float* diag = reinterpret_cast<float*>(sm + L::D_OFF);
        for (int x = 0; x < NV; ++x) chunk_zeros(s0 + L::TP_OFF + x * 4 * SLAB, pw);
        for (int m = 0; m < n; ++m) {
            const float* gt = reinterpret_cast<const float*>(sm + L::G_OFF + (m % NG) * L::GB);
            const uint32_t tb = s0 + L::TP_OFF + (m % NV) * 4 * SLAB;
            if (OUT) {
                wait(&gt_ready[m % NG], (m / NG) & 1, abort_flag, status, ERR_PREP);
                wait(g_full, m & 1, abort_flag, status, ERR_PREP);
                tc_fence_after();
                chunk_scores<false>(tm + tG, gt, a.scale, tb, diag, pw);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(g_read);
                named_bar_sync(2, 256);
            } else {
                wait(l_ready, m & 1, abort_flag, status, ERR_PREP);
                __syncwarp();
            }
            if (!chunk_inverse(tb, s0 + L::W_OFF, gt, diag, pw, *abort_flag, [&] {
                    if (!OUT && threadIdx.x == 512) mbar_arrive(d_free);
                }))
                break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&t_ready[m & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// The states entering the segments: S_in[0] = S0, S_in[s + 1] = M_s S_in[s] + S*_s, with each segment's
// (S* [dk][dv], M [dk][dk]) side by side, in fp32 (what this rounds stays in the state over all segments).
// With two segments a CTA the second's pair is of both: S_in[2 s + 2] = M S_in[2 s] + S*, as S_in[2 s + 1] is of the
// first's. A block owns 16 columns of one head. Each of its four groups of 64 threads sums over a quarter of the
// keys, DK / 16 rows by four columns a thread (16-byte loads from shared memory are what bounds it: twice
// as many with smaller tiles and no groups, 4.3 us a segment against 3.2); neighbouring lanes take
// neighbouring rows of M, which are padded by 16 bytes: no bank conflicts. The next segment's M and S* are on
// their way during a product.
template <int DK>
struct SL {
    static constexpr int COLS = 16, LDM = DK + 4;
    static constexpr int M_FLOATS = DK * LDM, S_FLOATS = DK * COLS;
    static constexpr int SMEM = (2 * M_FLOATS + 5 * S_FLOATS) * 4;
};
template <int DK>
__global__ void __launch_bounds__(256) gla_delta_scan_kernel(const float* __restrict__ S0, const float* __restrict__ pair,
                                                             float* S_in, int dv, int nseg, int per)
{
    using L = SL<DK>;
    constexpr int R = DK / 16, F = DK / 64;      // rows of a thread's tile; float4s of the block's columns a thread
    extern __shared__ __align__(16) float scan_smem[];
    float* M = scan_smem;                        // [2][DK][LDM]
    float* S = scan_smem + 2 * L::M_FLOATS;      // [DK][COLS]
    float* part = S + L::S_FLOATS;               // [4][DK][COLS]
    const int bh = blockIdx.y, tid = threadIdx.x, kg = tid / 64, rg = tid % 64 / 4;
    const int r0 = tid / 4, c = tid % 4 * 4, col = blockIdx.x * L::COLS + c;
    const bool in = col < dv;                    // dv is a multiple of 16
    const size_t st = (size_t)DK * dv, step = st + DK * DK;
    const float* pp = pair + (size_t)bh * (nseg - 1) * step;
    float* out = S_in + (size_t)bh * nseg * st + col;
    auto fetch = [&](int g) {
        const float* m = pp + g * step + st;
        const uint32_t d = smem_u32(M + (g & 1) * L::M_FLOATS);
        for (int i = tid; i < DK * DK / 4; i += 256)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         ::"r"(d + (i / (DK / 4) * L::LDM + i % (DK / 4) * 4) * 4), "l"(m + i * 4) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    // a thread's rows r0 + 64 i of the state, and of the next S*
    float4 x[F], own[F];
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int r = r0 + 64 * i;
        x[i] = S0 && in ? *reinterpret_cast<const float4*>(S0 + bh * st + (size_t)r * dv + col) : zero;
        own[i] = in ? *reinterpret_cast<const float4*>(pp + (size_t)r * dv + col) : zero;
    }
    for (int g = 0;; ++g) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int r = r0 + 64 * i;
            if (per == 1 || !(g & 1)) *reinterpret_cast<float4*>(S + r * L::COLS + c) = x[i];
            if (in) *reinterpret_cast<float4*>(out + g * st + (size_t)r * dv) = x[i];
        }
        if (g + 1 == nseg) break;
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        if (g + 2 < nseg) fetch(g + 1);
        float2 y[R][2] = {};
        const float* m = M + (g & 1) * L::M_FLOATS + rg * L::LDM + kg * (DK / 4);
        const float* s = S + kg * (DK / 4) * L::COLS + c;
#pragma unroll 2
        for (int j = 0; j < DK / 4; j += 4) {
            float4 f[R], v[4];
#pragma unroll
            for (int i = 0; i < R; ++i) f[i] = *reinterpret_cast<const float4*>(m + 16 * i * L::LDM + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const float4*>(s + (j + e) * L::COLS);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const float w = e == 0 ? f[i].x : e == 1 ? f[i].y : e == 2 ? f[i].z : f[i].w;
                    y[i][0] = fma2(make_float2(w, w), make_float2(v[e].x, v[e].y), y[i][0]);
                    y[i][1] = fma2(make_float2(w, w), make_float2(v[e].z, v[e].w), y[i][1]);
                }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            *reinterpret_cast<float4*>(part + (kg * DK + rg + 16 * i) * L::COLS + c) = make_float4(y[i][0].x, y[i][0].y, y[i][1].x, y[i][1].y);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const int r = r0 + 64 * i;
            x[i] = own[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 p = *reinterpret_cast<const float4*>(part + (k * DK + r) * L::COLS + c);
                x[i].x += p.x; x[i].y += p.y; x[i].z += p.z; x[i].w += p.w;
            }
            if (g + 2 < nseg && in) own[i] = *reinterpret_cast<const float4*>(pp + (g + 1) * step + (size_t)r * dv + col);
        }
    }
}

template <int DK, bool OUT>
cudaError_t launch_pass(const FusedArgs& a, const FusedMaps& m, dim3 grid, cudaStream_t s)
{
    using L = FL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_fused_kernel<DK, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    gla_delta_fused_kernel<DK, OUT><<<grid, NT, L::SMEM, s>>>(a, m);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_dk(const DeltaChunks& p, const FusedMaps& m, int* status, cudaStream_t s)
{
    const unsigned BH = (unsigned)(p.B * p.H);
    const long long st = (long long)p.dk * p.dv;
    FusedArgs a;
    a.log_g = p.log_g; a.beta = static_cast<const __nv_bfloat16*>(p.beta);
    a.H = p.H; a.Hk = p.Hk; a.T = p.T; a.dv = p.dv; a.nch = p.nch; a.cps = p.cps; a.nseg = p.nseg; a.per = 1;
    a.tiles = (p.dv + DVT - 1) / DVT;
    a.scale = p.scale; a.status = status;
    const unsigned tiles = (unsigned)a.tiles;
    if (p.nseg > 1) {
        // every segment but the last: its state from zero and its transition
        a.S_in = nullptr; a.in_bh = a.in_seg = 0;
        a.S_out = p.pair; a.out_seg = st + (long long)p.dk * p.dk; a.out_bh = a.out_seg * (p.nseg - 1);
        a.per = p.per; a.cps = p.cps * p.per; a.nch = (p.nseg - 1) * p.cps;
        cudaError_t e = launch_pass<DK, false>(a, m, dim3(tiles + 1, BH, p.per == 2 ? p.nseg / 2 : p.nseg - 1), s);
        if (e != cudaSuccess) return e;
        constexpr int smem = SL<DK>::SMEM, cols = SL<DK>::COLS;
        e = cudaFuncSetAttribute(gla_delta_scan_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        gla_delta_scan_kernel<DK><<<dim3((p.dv + cols - 1) / cols, BH), 256, smem, s>>>(p.S0, p.pair, p.seg_in, p.dv, p.nseg, p.per);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        a.cps = p.cps; a.nch = p.nch;
        a.S_in = p.seg_in; a.in_bh = st * p.nseg; a.in_seg = st;
    } else {
        a.S_in = p.S0; a.in_bh = st; a.in_seg = 0;
    }
    a.S_out = p.ST; a.out_bh = st; a.out_seg = 0;
    return launch_pass<DK, true>(a, m, dim3(tiles, BH, p.nseg), s);
}

}  // namespace

cudaError_t launch_delta_chunks(const DeltaChunks& p, int* status, cudaStream_t s)
{
    const uint64_t bk = (uint64_t)p.B * p.Hk, bh = (uint64_t)p.B * p.H;
    FusedMaps m;
    if (!map_rows(&m.k, p.k, p.dk, p.T, bk) || !map_rows(&m.q, p.q, p.dk, p.T, bk) || !map_slabs(&m.v, p.v, p.dv, p.T, bh, 2))
        return cudaErrorInvalidValue;
    {   // O: staged without a swizzle
        const uint64_t dims[3] = {(uint64_t)p.dv, (uint64_t)p.T, bh}, str[2] = {(uint64_t)p.dv * 2, (uint64_t)p.dv * p.T * 2};
        const uint32_t box[3] = {64, C, 1};
        if (!make_tmap(&m.o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.O, dims, str, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    }
    return p.dk == 64 ? launch_dk<64>(p, m, status, s) : launch_dk<128>(p, m, status, s);
}

}  // namespace gla
