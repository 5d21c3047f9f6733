// gla_delta_grads: the chunk-parallel half of the delta rule's backward. For one chunk, with S the
// state entering it, dS the gradient of the state leaving it, U, dV (the sweeps' results),
// e = exp(G), l = exp(G_end - G), D_ij = exp(G_i - G_j):
//
//   W_ij = scale D_ij (dO_i . u_j)  (j <= i),     M_ij = -D_ij (dV_i . u_j)  (j < i),
//   dQ  = scale e (dO S^T) + W K,
//   dK  = [M K - e (dV S^T)]  +  [M^T K + W^T Q + l (U dS^T)]      (row role + column role),
//   dbeta_i = (dV_i . u_i) / beta_i^2,
//   dlog_g_t = sum over i >= t of (q_i . scale e (dO S^T)_i - k_i . e (dV S^T)_i)    (the state entering, read at i)
//            + sum over j < t of k_j . l (U dS^T)_j                                    (token j in the state leaving)
//            + exp(G_end) <dS, S> + sum over i >= t > j of Z_ij,   Z_ij = W_ij (q_i . k_j) + M_ij (k_i . k_j).
//
// dlog_g_t is the sum over all that decays across token t, pair by pair, and is formed as that: as the running sum of
// q . dQ + k . dK_row - k . dK_col, which is the same, it cancels what both of a pair's tokens lie behind t, and of a steep
// gate's gradient few digits were left (2e-4 off at decays around e^-6, none right at e^-14). Its terms have both signs, so every operand
// that is not an input comes in two bf16 parts and products keep hi hi + hi lo + lo hi. To use 128 tensor-memory lanes
// the operands are stacked: [dO; dV] on the left of U^T and of S^T, [U; U_lo] on the left of
// dS^T (both halves of the result belong to one row and are added at the end), [W; M] on the left
// of K, and transposed, hi over lo, on the left of [Q; K].
//
// One persistent CTA per SM (the operands and accumulators fill its shared and tensor memory) walks
// the chunks; the next chunk's dO, dV, U and S are loaded as soon as this one's are used. Bound by its
// loads, 240 KB per chunk at dk = dv = 128, and the latency of its own steps, about equally: 245 us for
// 8 x 2048 tokens of 16 heads, 4.6 TB/s (of which the pairs' sums 13; with a CTA per chunk and nothing loaded ahead
// it was 345 to 231).
#include "gla_delta_dev.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 256;

enum { ERR_LOAD = 0x631, ERR_MMA = 0x632 };

template <int DK>
struct GL {
    static constexpr int NS = DK / 64;
    static constexpr int QK_OFF = 0;                          // [Q slab, K slab] per 64 keys
    static constexpr int XA_OFF = QK_OFF + 2 * NS * SLAB;     // [dO slab, dV slab] x 2
    static constexpr int XB_OFF = XA_OFF + 4 * SLAB;          // [zeros, dV_lo slab] x 2
    static constexpr int U_OFF = XB_OFF + 4 * SLAB;           // U, U_lo: 128 rows of dv by 64 tokens
    static constexpr int S_OFF = U_OFF + 4 * SLAB;            // S, S_lo (then dS): slabs of 128 rows by 64 keys
    static constexpr int SB = NS * 2 * SLAB;                  // one part
    static constexpr int G_OFF = S_OFF + 2 * SB;              // gates, 8 x 64 floats
    static constexpr int R_OFF = G_OFF + 8 * C * 4;           // row sums 4 x 64, state sums 4 x 64, 8 partials
    static constexpr int F_OFF = R_OFF + 8 * C * 4 + 64;      // the pairs' part of dlog_g: 8 warps and two suffix sums x 32
    static constexpr int BAR_OFF = F_OFF + 10 * 32 * 4;
    static constexpr int SMEM = BAR_OFF + 128 + 1024;
    static constexpr int W_OFF = XB_OFF;                      // [W; M] in two parts, once dV_lo is used
    static constexpr int E_OFF = XB_OFF;                      // then dK's partial rows (fp32), when W is used
    static_assert(64 * DK * 4 <= 4 * SLAB, "exchange buffer");
    static constexpr int t1 = 0, tG = 64, t2 = 128, t3 = 256, tH = 384, tH2 = 0;   // tG: [Q; K] K^T, until tH2 is formed
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct GMaps { CUtensorMap q, k, dO, xh, xl, uh, ul, sh, sl, dh, dl; };

__device__ __forceinline__ void load8(uint32_t a, float (&x)[8])
{
    uint32_t u[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "r"(a));
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = bf_lo(u[i]); x[2 * i + 1] = bf_hi(u[i]); }
}

template <int DK>
__global__ void __launch_bounds__(NT, 1)
gla_delta_grads_kernel(DeltaGrads a, const __grid_constant__ GMaps mp, int* status)
{
    using L = GL<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* b_qk = bar;        // Q, K, gates loaded
    uint64_t* b_xa = bar + 1;    // dO, dV loaded
    uint64_t* b_xb = bar + 2;    // dV_lo loaded
    uint64_t* b_u = bar + 3;     // U loaded
    uint64_t* b_s = bar + 4;     // S loaded
    uint64_t* b_d = bar + 5;     // dS loaded
    uint64_t* m_1 = bar + 6;     // products with U^T and S^T done
    uint64_t* m_3 = bar + 7;     // products with dS^T done
    uint64_t* m_h = bar + 8;     // products of W and M done
    uint64_t* m_g = bar + 9;     // the scores done
    uint64_t* fin = bar + 10;    // every product done
    uint32_t* holder = reinterpret_cast<uint32_t*>(bar + 11);
    const Abort abort_flag(bar + 12);
    float* gt = reinterpret_cast<float*>(sm + L::G_OFF);
    float* rs = reinterpret_cast<float*>(sm + L::R_OFF);        // [4][64] row sums
    float* ss = rs + 4 * C;                                     // [4][64] k . (l U dS^T)
    float* ip = ss + 4 * C;                                     // [8] warps' parts of <dS, S>
    float* fz = reinterpret_cast<float*>(sm + L::F_OFF);        // [8][32] and [2][32]

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
    const int ntile = (a.dv + 127) / 128;
    const int total = a.B * a.H * a.nch;

    if (tid == 0) {
        for (int i = 0; i < 11; ++i) mbar_init(&bar[i], 1);
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, 512);
        tmem_relinquish();
    }
    auto zero_slabs = [&]() {
        for (int i = tid; i < 2 * SLAB / 16; i += NT)
            *reinterpret_cast<uint4*>(sm + L::XB_OFF + (i / (SLAB / 16)) * 2 * SLAB + i % (SLAB / 16) * 16) = make_uint4(0u, 0u, 0u, 0u);
    };
    zero_slabs();
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *holder;

    int it = 0, cnt = 0;                // chunks done, and tiles of dv: the barriers' phases
    // this thread's waits so far have come to their ends (else it issues nothing any more); in the thread that
    // loads, the barriers that it has armed and the parities of their next phases
    bool ok = true;
    uint32_t armed = 0, next = 0;
    auto arm = [&](uint64_t* x, uint32_t bytes) {
        armed |= 1u << (x - bar);
        next ^= 1u << (x - bar);
        mbar_arrive_expect_tx(x, bytes);
    };
    for (int at = blockIdx.x; at < total; at += gridDim.x, ++it) {
    const int c = at % a.nch, bh = at / a.nch, t0 = c * C;
    const int b = bh / a.H, h = bh % a.H, bk = b * a.Hk + h / (a.H / a.Hk);
    auto load_s = [&](int chunk, int dv0) {
        arm(b_s, 2 * L::SB);
#pragma unroll
        for (int i = 0; i < L::NS; ++i) {
            tma_load_3d(sm + L::S_OFF + i * 2 * SLAB, &mp.sh, b_s, 64 * i, dv0, chunk);
            tma_load_3d(sm + L::S_OFF + L::SB + i * 2 * SLAB, &mp.sl, b_s, 64 * i, dv0, chunk);
        }
    };
    // (tiles of dv that end inside the pair of slabs are filled with zeros)
    auto load_xa = [&](int chunk, int dv0) {
        arm(b_xa, 4 * SLAB);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            tma_load_3d(sm + L::XA_OFF + 2 * i * SLAB, &mp.dO, b_xa, dv0 + 64 * i, chunk % a.nch * C, chunk / a.nch);
            tma_load_3d(sm + L::XA_OFF + (2 * i + 1) * SLAB, &mp.xh, b_xa, dv0 + 64 * i, chunk % a.nch * C, chunk / a.nch);
        }
    };
    auto load_u = [&](int chunk, int dv0) {
        arm(b_u, 4 * SLAB);
        tma_load_3d(sm + L::U_OFF, &mp.uh, b_u, 0, dv0, chunk);
        tma_load_3d(sm + L::U_OFF + 2 * SLAB, &mp.ul, b_u, 0, dv0, chunk);
    };
    const bool more = at + (int)gridDim.x < total;
    float inner = 0.f;
    for (int vt = 0; vt < ntile; ++vt, ++cnt) {
        const int dv0 = vt * 128;
        const uint32_t ph = cnt & 1;
        if (warp == 0) {
            if (lane == 0 && ok) {
                if (vt == 0) {
                    arm(b_qk, 2 * L::NS * SLAB + 8 * C * 4);
#pragma unroll
                    for (int i = 0; i < L::NS; ++i) {
                        tma_load_3d(sm + L::QK_OFF + 2 * i * SLAB, &mp.q, b_qk, 64 * i, t0, bk);
                        tma_load_3d(sm + L::QK_OFF + (2 * i + 1) * SLAB, &mp.k, b_qk, 64 * i, t0, bk);
                    }
                    bulk_load(gt, a.gates + (size_t)at * 8 * C, 8 * C * 4, b_qk);
                }
                arm(b_xb, 2 * SLAB);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    tma_load_3d(sm + L::XB_OFF + (2 * i + 1) * SLAB, &mp.xl, b_xb, dv0 + 64 * i, t0, bh);
                if (it == 0 || vt > 0) {              // (else they are there or on their way)
                    load_xa(at, dv0);
                    load_u(at, dv0);
                    load_s(at, dv0);
                }
            }
            __syncwarp();
            const uint64_t dXa = sdesc(s0 + L::XA_OFF, 16, 1024, kSwizzle128), dXb = sdesc(s0 + L::XB_OFF, 16, 1024, kSwizzle128);
            const uint64_t dU = sdesc(s0 + L::U_OFF, 2 * SLAB, 1024, kSwizzle128);
            const uint64_t dS = sdesc(s0 + L::S_OFF, 2 * SLAB, 1024, kSwizzle128);
            const uint32_t id1 = idesc_bf16(128, 64, false, true), id2 = idesc_bf16(128, DK, false, true);
            ok &= wait(b_xa, ph, abort_flag, status, ERR_LOAD);
            ok &= wait(b_u, ph, abort_flag, status, ERR_LOAD);
            __syncwarp();
            if (elect_one() && ok) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4, r = (kk * 2048) >> 4;
                    mma_ss(tm + L::t1, dXa + o, dU + r, id1, vt > 0 || kk > 0);
                    mma_ss(tm + L::t1, dXa + o, dU + (2 * SLAB >> 4) + r, id1, 1);
                }
            }
            ok &= wait(b_s, ph, abort_flag, status, ERR_LOAD);
            __syncwarp();
            if (elect_one() && ok) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4, r = (kk * 2048) >> 4;
                    mma_ss(tm + L::t2, dXa + o, dS + r, id2, vt > 0 || kk > 0);
                    mma_ss(tm + L::t2, dXa + o, dS + (L::SB >> 4) + r, id2, 1);
                }
            }
            ok &= wait(b_xb, ph, abort_flag, status, ERR_LOAD);
            __syncwarp();
            if (elect_one() && ok) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4, r = (kk * 2048) >> 4;
                    mma_ss(tm + L::t1, dXb + o, dU + r, id1, 1);
                    mma_ss(tm + L::t2, dXb + o, dS + r, id2, 1);
                }
                mma_commit(m_1);
            }
            __syncwarp();
        }
        if (warp == 1) {
            // dS on its way into L2 (more tiles than these would only queue before the loads)
            if (elect_one())
                for (int i = 0; i < L::NS; ++i) {
                    prefetch_l2_tile_3d(&mp.dh, 64 * i, dv0, at);
                    prefetch_l2_tile_3d(&mp.dl, 64 * i, dv0, at);
                }
            __syncwarp();
        }
        // S of this tile to registers, for <dS, S> (dS takes its place)
        constexpr int NP = 128 * DK / 8 / NT;        // pieces of eight keys a thread
        auto piece = [&](int p) {
            const int i = tid + p * NT, r = i / (DK / 8), k = i % (DK / 8);
            return s0 + L::S_OFF + (k >> 3) * 2 * SLAB + r * 128 + (((k & 7) ^ (r & 7)) << 4);
        };
        float sv[NP][8];
        ok &= wait(b_s, ph, abort_flag, status, ERR_LOAD);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float v[8];
            load8(piece(p), sv[p]);
            load8(piece(p) + L::SB, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sv[p][e] += v[e];
        }
        ok &= wait(m_1, ph, abort_flag, status, ERR_MMA);
        __syncthreads();            // S is read by everyone: dS may take its place
        if (warp == 0) {
            if (lane == 0 && ok) {
                arm(b_d, 2 * L::SB);
#pragma unroll
                for (int i = 0; i < L::NS; ++i) {
                    tma_load_3d(sm + L::S_OFF + i * 2 * SLAB, &mp.dh, b_d, 64 * i, dv0, at);
                    tma_load_3d(sm + L::S_OFF + L::SB + i * 2 * SLAB, &mp.dl, b_d, 64 * i, dv0, at);
                }
                if (more && vt == ntile - 1) load_xa(at + gridDim.x, 0);   // (the next chunk's)
            }
            __syncwarp();
            if (vt == ntile - 1 && a.dlog_g) {
                // the scores, for the gate, while dS is on its way
                ok &= wait(b_qk, it & 1, abort_flag, status, ERR_LOAD);
                __syncwarp();
                const uint32_t idG = idesc_bf16(128, 64, false, false);
                const uint64_t dG = sdesc(s0 + L::QK_OFF, 16, 1024, kSwizzle128), dG2 = sdesc(s0 + L::QK_OFF + SLAB, 16, 1024, kSwizzle128);
                if (elect_one() && ok) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4;
                        mma_ss(tm + L::tG, dG + o, dG2 + o, idG, kk > 0);
                    }
                    mma_commit(m_g);
                }
                __syncwarp();
            }
            const uint64_t dU = sdesc(s0 + L::U_OFF, 2 * SLAB, 1024, kSwizzle128);   // tokens along M: U on U_lo
            const uint64_t dS = sdesc(s0 + L::S_OFF, 2 * SLAB, 1024, kSwizzle128);
            const uint32_t id3 = idesc_bf16(128, DK, true, true);
            ok &= wait(b_d, ph, abort_flag, status, ERR_LOAD);
            __syncwarp();
            if (elect_one() && ok) {
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const uint64_t r = (kk * 2048) >> 4;
                    mma_ss(tm + L::t3, dU + r, dS + r, id3, vt > 0 || kk > 0);
                    mma_ss(tm + L::t3, dU + r, dS + (L::SB >> 4) + r, id3, 1);
                }
                mma_commit(m_3);
            }
            __syncwarp();
        }
        ok &= wait(b_d, ph, abort_flag, status, ERR_LOAD);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            float u[8], v[8];
            load8(piece(p), u);
            load8(piece(p) + L::SB, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) inner = fmaf(sv[p][e], u[e] + v[e], inner);
        }
        if (vt + 1 < ntile) {       // one set of tiles: the next load waits for these products
            ok &= wait(m_3, ph, abort_flag, status, ERR_MMA);
            __syncthreads();
        }
    }

    // W and M: lanes 0-63 rows of dO U^T, 64-127 of dV U^T; warps 0-3 the first 32 columns
    const int quarter = warp & 3, hf = warp >> 2;
    const int row = quarter * 32 + lane, i = row & 63;
    const bool low = row < 64;
    const uint32_t lb = (uint32_t)(quarter * 32) << 16;
    tc_fence_after();
    ok &= wait(b_qk, it & 1, abort_flag, status, ERR_LOAD);
    const int c0 = hf * 32;
    float x[32];                  // this row's W or M, and its scores
    uint32_t kqk[32];
    {
        uint32_t r[32];
        tmem_ld32(tm + lb + L::t1 + c0, r);
        tmem_wait_ld();
        const bool near = gt[4 * C] != 0.f;
        const float f = low ? a.scale : -1.f;
        const int last = low ? i : i - 1;
        if (!low && i >= c0 && i < c0 + 32) {
            float d = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) d = c0 + j == i ? __uint_as_float(r[j]) : d;
            const float be = gt[i];
            if (a.dbeta && t0 + i < a.T)
                static_cast<__nv_bfloat16*>(a.dbeta)[(size_t)bh * a.T + t0 + i] = __float2bfloat16_rn(d / be / be);
        }
        if (near) {
            const float fi = f * gt[4 * C + i];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 q = *reinterpret_cast<const float4*>(gt + 5 * C + c0 + j);
                x[j] = __uint_as_float(r[j]) * (fi * q.x);
                x[j + 1] = __uint_as_float(r[j + 1]) * (fi * q.y);
                x[j + 2] = __uint_as_float(r[j + 2]) * (fi * q.z);
                x[j + 3] = __uint_as_float(r[j + 3]) * (fi * q.w);
            }
        } else {
            const float gh = gt[6 * C + i], gl = gt[7 * C + i];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = f * __uint_as_float(r[j]) * expf((gh - gt[6 * C + c0 + j]) + (gl - gt[7 * C + c0 + j]));
        }
        // (nothing above the diagonal; there x may be anything)
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = c0 + j <= last ? x[j] : 0.f;
        if (a.dlog_g) {                 // (the products of W and M lie over the scores)
            ok &= wait(m_g, it & 1, abort_flag, status, ERR_MMA);
            tc_fence_after();
            tmem_ld32(tm + lb + L::tG + c0, kqk);
            tmem_wait_ld();
        }
        // rows of 64 values, hi then lo; the products with dO and dV, whose place this is, are done
        const uint32_t wo = s0 + L::W_OFF + row * 128;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 8 * p + 2 * e;
                split2(x[j], x[j + 1], hi[e], lo[e]);
            }
            const uint32_t o = wo + (((hf * 4 + p) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(o), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(o + 2 * SLAB), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3]));
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        const uint64_t dW = sdesc(s0 + L::W_OFF, 16, 1024, kSwizzle128);             // rows along M
        const uint64_t dWt = sdesc(s0 + L::W_OFF, 2 * SLAB, 1024, kSwizzle128);      // columns along M: hi on lo
        const uint64_t dQ = sdesc(s0 + L::QK_OFF, 2 * SLAB, 1024, kSwizzle128);      // 128 rows [Q; K], keys along N
        const uint64_t dK = sdesc(s0 + L::QK_OFF + SLAB, 2 * SLAB, 1024, kSwizzle128);
        const uint32_t idH = idesc_bf16(128, DK, false, true), idT = idesc_bf16(128, DK, true, true);
        if (elect_one() && ok) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint64_t o = (kk * 32) >> 4, r = (kk * 2048) >> 4;
                mma_ss(tm + L::tH, dW + o, dK + r, idH, kk > 0);
                mma_ss(tm + L::tH, dW + (2 * SLAB >> 4) + o, dK + r, idH, 1);
            }
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                const uint64_t r = (kk * 2048) >> 4;
                mma_ss(tm + L::tH2, dWt + r, dQ + r, idT, kk > 0);
            }
            mma_commit(m_h);
        }
        __syncwarp();
    }
    if (a.dlog_g) {
        // While those products run: the pairs across token t = c0 + j, of this row for j' in c0 .. t - 1, if the row is not
        // before t; then over the warp's rows, which leaves token c0 + lane with a lane (halves of the 32 values are
        // exchanged for halves of the lanes, five times).
        float z[32], run = 0.f;
        z[0] = 0.f;
        if (hf == 0 || (quarter & 1)) {         // (the first rows have no pairs in the second half)
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                z[j] = i >= c0 + j ? run : 0.f;
                run = fmaf(x[j], __uint_as_float(kqk[j]), run);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const bool up = lane & o;
#pragma unroll
                for (int j = 0; j < o; ++j) {
                    const float other = __shfl_xor_sync(~0u, up ? z[j] : z[j + o], o);
                    z[j] = (up ? z[j + o] : z[j]) + other;
                }
            }
        }
        fz[warp * 32 + lane] = z[0];
        // a row of the second half has all of the first half's columns before every t of its own half
        if (hf == 0 && (quarter & 1)) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float later = __shfl_down_sync(~0u, run, o);
                if (lane + o < 32) run += later;
            }
            fz[(8 + (quarter >> 1)) * 32 + lane] = run;
        }
    }
    ok &= wait(m_3, (cnt - 1) & 1, abort_flag, status, ERR_MMA);
    ok &= wait(m_h, it & 1, abort_flag, status, ERR_MMA);
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && more && ok) {
        // U and dS are used (and everyone has read dS): the next chunk's U and S take their place
        load_u(at + gridDim.x, 0);
        load_s(at + gridDim.x, 0);
    }
    {
        // one row and half of the keys a thread
        const float e = gt[C + i], l = gt[2 * C + i];
        const float f2s = low ? a.scale * e : -e;
        float sum = 0.f, st = 0.f;
        float* ex = reinterpret_cast<float*>(sm + L::E_OFF) + i * DK;   // groups of four in another order by row
        auto slot = [&](int k) { return ((k >> 2) ^ (i & 7)) * 4; };
        const bool in = t0 + i < a.T;
        const size_t orow = ((size_t)bh * a.T + t0 + i) * DK;
        auto store = [&](void* out, float* part, int k, const float (&x)[16]) {
            if (!in) return;
            if (part) {
#pragma unroll
                for (int j = 0; j < 16; j += 4)
                    *reinterpret_cast<float4*>(part + orow + k + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            } else {
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + orow + k);
                o[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                o[1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
            }
        };
        float col[DK / 2];            // this row's part of dK's column role
#pragma unroll
        for (int kc = 0; kc < DK / 2; kc += 16) {
            const int k = hf * (DK / 2) + kc;
            uint32_t g2[16], g3[16], g4[16], g5[16];
            tmem_ld16(tm + lb + L::t2 + k, g2);
            tmem_ld16(tm + lb + L::tH + k, g4);
            tmem_ld16(tm + lb + L::t3 + k, g3);
            tmem_ld16(tm + lb + L::tH2 + k, g5);
            float q[16], kr[16];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int key = k + 8 * p;
                const uint32_t o = s0 + L::QK_OFF + (key >> 6) * 2 * SLAB + i * 128 + ((((key & 63) >> 3) ^ (i & 7)) << 4);
                load8(o + SLAB, *reinterpret_cast<float(*)[8]>(&kr[8 * p]));
                if (low) load8(o, *reinterpret_cast<float(*)[8]>(&q[8 * p]));
            }
            tmem_wait_ld();
            float x[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float read = f2s * __uint_as_float(g2[j]);
                const float own = fmaf(f2s, __uint_as_float(g2[j]), __uint_as_float(g4[j]));
                const float state = l * __uint_as_float(g3[j]);
                const float cr = state + __uint_as_float(g5[j]);
                sum = fmaf(low ? q[j] : kr[j], read, sum);
                st = fmaf(kr[j], state, st);
                col[kc + j] = cr;
                x[j] = low ? own : own + cr;
            }
            if (low) {
                store(a.dq, a.part_q, k, x);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(ex + slot(k + j)) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
            }
        }
        rs[((low ? 0 : 1) + 2 * hf) * C + i] = sum;
        ss[((low ? 0 : 1) + 2 * hf) * C + i] = st;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) inner += __shfl_xor_sync(~0u, inner, o);
        if (lane == 0) ip[warp] = inner;
        __syncthreads();
        if (low) {
#pragma unroll
            for (int kc = 0; kc < DK / 2; kc += 16) {
                const int k = hf * (DK / 2) + kc;
                float x[16];
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(ex + slot(k + j));
                    x[j] = col[kc + j] + f.x; x[j + 1] = col[kc + j + 1] + f.y;
                    x[j + 2] = col[kc + j + 2] + f.z; x[j + 3] = col[kc + j + 3] + f.w;
                }
                store(a.dk_out, a.part_k, k, x);
            }
        }
        if (warp == 4 && a.dlog_g) {
            // two tokens a lane: what reads the state behind them, what they find written, the pairs across, the state
            // through the chunk
            const int p = 2 * lane, half = p >> 5;
            float r0 = 0.f, r1 = 0.f, w0 = 0.f, w1 = 0.f, f0 = 0.f, f1 = 0.f;
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                r0 += rs[z * C + p];
                r1 += rs[z * C + p + 1];
                w0 += ss[z * C + p];
                w1 += ss[z * C + p + 1];
                f0 += fz[(half * 4 + z) * 32 + (p & 31)];
                f1 += fz[(half * 4 + z) * 32 + (p & 31) + 1];
            }
            if (half) {
#pragma unroll
                for (int z = 8; z < 10; ++z) {
                    f0 += fz[z * 32 + (p & 31)];
                    f1 += fz[z * 32 + (p & 31) + 1];
                }
            }
            float in8 = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) in8 += ip[w];
            const float s = gt[2 * C - 1] * in8;
            float y = r0 + r1, x = w0 + w1;          // over the later lanes, over the earlier ones
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float u = __shfl_down_sync(~0u, y, o), v = __shfl_up_sync(~0u, x, o);
                if (lane + o < 32) y += u;
                if (lane >= o) x += v;
            }
            y = __shfl_down_sync(~0u, y, 1);
            x = __shfl_up_sync(~0u, x, 1);
            if (lane == 31) y = 0.f;
            if (lane == 0) x = 0.f;
            float* out = a.dlog_g + (size_t)bh * a.T + t0 + p;
            if (t0 + p < a.T) out[0] = ((y + r1) + r0) + x + f0 + s;
            if (t0 + p + 1 < a.T) out[1] = (y + r1) + (x + w0) + f1 + s;
        }
    }
    __syncthreads();        // the exchange is read
    zero_slabs();
    fence_proxy_async_smem();
    tc_fence_before();
    // everything of this chunk is read: the next one's loads may land
    const bool quit = __syncthreads_or(!ok);
    tc_fence_after();
    if (quit) break;
    }
    // nothing may be in flight when the CTA ends (it is not, unless a wait has run out)
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < 6; ++i)
                if (armed >> i & 1) mbar_wait(&bar[i], (next >> i & 1) ^ 1, kTimeoutNs);
        __syncwarp();
        if (elect_one()) mma_commit(fin);
        __syncwarp();
        mbar_wait(fin, 0, kTimeoutNs);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

bool map_tall(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch)
{
    const uint64_t dims[3] = {cols, rows, batch}, str[2] = {cols * 2, cols * rows * 2};
    const uint32_t box[3] = {64, 128, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int DK>
cudaError_t launch_dk(const DeltaGrads& a, const GMaps& m, int* status, cudaStream_t s)
{
    using L = GL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_grads_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const long long n = (long long)a.B * a.H * a.nch;
    gla_delta_grads_kernel<DK><<<(unsigned)(n < a.sms ? n : a.sms), NT, L::SMEM, s>>>(a, m, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_grads(const DeltaGrads& a, int* status, cudaStream_t s)
{
    const uint64_t bk = (uint64_t)a.B * a.Hk, bh = (uint64_t)a.B * a.H, nc = bh * a.nch;
    GMaps m;
    if (!map_rows(&m.q, a.q, a.dk, a.T, bk) || !map_rows(&m.k, a.k, a.dk, a.T, bk) ||
        !map_rows(&m.dO, a.dO, a.dv, a.T, bh) || !map_rows(&m.xh, a.x_hi, a.dv, a.T, bh) ||
        !map_rows(&m.xl, a.x_lo, a.dv, a.T, bh) || !map_tall(&m.uh, a.u_hi, C, a.dv, nc) ||
        !map_tall(&m.ul, a.u_lo, C, a.dv, nc) || !map_tall(&m.sh, a.s_hi, a.dk, a.dv, nc) ||
        !map_tall(&m.sl, a.s_lo, a.dk, a.dv, nc) || !map_tall(&m.dh, a.d_hi, a.dk, a.dv, nc) ||
        !map_tall(&m.dl, a.d_lo, a.dk, a.dv, nc))
        return cudaErrorInvalidValue;
    return a.dk == 64 ? launch_dk<64>(a, m, status, s) : launch_dk<128>(a, m, status, s);
}

}  // namespace gla
