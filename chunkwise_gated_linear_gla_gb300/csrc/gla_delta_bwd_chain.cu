// gla_delta_sweep: the two serial passes of the delta rule's backward, built like the forward
// chain (gla_delta_fused.cu): dv along the tensor-memory lanes, the state in fp32 registers,
// every operand that feeds it in two bf16 parts. With e = exp(G), l = exp(G_end - G):
//
//   forward:  U = T (V - e K S),              S  <- exp(G_end) S + K^T (l U)
//   reverse:  dU = P^T dO + l (K dS),
//             dV = T^T dU,                    dS <- exp(G_end) dS + Q^T (scale e dO) - K^T (e dV)
//
// The forward sweep stores the state entering each chunk and U, the reverse one the gradient of
// the state leaving each chunk and dV; the gradients of q, k and the gates are then formed chunk
// by chunk in parallel. (dV = beta times the gradient of T's right-hand side, as T holds beta.)
//
// Four warps off the chain take the results out: they read the parts (and U or dV, still fp32 in
// tensor memory) into one 32 KB buffer and store it by TMA, hi, then lo, then U or dV; in
// reverse they also form the parts of scale e dO. 8 x 2048 tokens, 16 heads, dk = dv = 128: 107 us forward
// (145 KB a chunk read and written, 5.5 TB/s), 120 us in reverse (177 KB, 6.0 TB/s): bound by those bytes.
#include "gla_delta_dev.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 512;
constexpr int NST = 2;
constexpr int DVT = 128;

enum { ERR_TMA = 0x621, ERR_MMA = 0x622, ERR_EPI = 0x623, ERR_DRAIN = 0x624 };

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

template <int DK, bool REV>
struct CL {
    static constexpr int KB = (DK / 64) * SLAB;
    static constexpr int K_OFF = 0, V_OFF = KB, T_OFF = V_OFF + 2 * SLAB, Q_OFF = T_OFF + 2 * SLAB,
                         P_OFF = Q_OFF + (REV ? KB : 0), G_OFF = P_OFF + (REV ? 2 * SLAB : 0);
    static constexpr int STAGE = G_OFF + 1024;
    static constexpr int BYTES = G_OFF + 4 * C * 4;
    static constexpr int O_OFF = NST * STAGE;            // staging for the stores, 32 KB
    static constexpr int BAR_OFF = O_OFF + 4 * SLAB;
    static constexpr int SMEM = BAR_OFF + 256 + 1024;
    static constexpr int tD = 0, tSh = DK, tSl = tSh + DK / 2, tX = 2 * DK, tRh = tX + 64, tRl = tRh + 32,
                         tYh = tRl + 32, tYl = tYh + 32, tKs = tYl + 32;
    static constexpr int TCOLS = 512;
    static_assert(tKs + 64 <= TCOLS, "tensor memory");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap k, v, t, q, p;             // loads
    CUtensorMap sh, sl, xh, xl;            // stores: the state's parts; U's parts or dV's
};

template <int DK, bool REV>
__global__ void __launch_bounds__(NT, 1)
gla_delta_sweep_kernel(DeltaSweep a, const __grid_constant__ Maps mp, int* status)
{
    using L = CL<DK, REV>;
    constexpr int HC = DK / 2;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(sm);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);
    uint64_t* full = bar;             // [NST]
    uint64_t* empty = bar + NST;      // [NST]: the products' commit and four drain warps
    uint64_t* s_ready = bar + 2 * NST;
    uint64_t* ks_full = s_ready + 1;
    uint64_t* r_ready = s_ready + 2;
    uint64_t* u_full = s_ready + 3;
    uint64_t* u_ready = s_ready + 4;
    uint64_t* d_full = s_ready + 5;
    uint64_t* sp_free = s_ready + 6;  // the drain has read the state's parts (4 warps)
    uint64_t* x_free = s_ready + 7;   // and X (4 warps)
    uint64_t* y_ready = s_ready + 8;  // and written the parts of scale e dO (4 warps; reverse)
    uint64_t* fin = s_ready + 9;
    uint32_t* holder = reinterpret_cast<uint32_t*>(s_ready + 10);
    const Abort abort_flag(s_ready + 11);

    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32, wg = warp / 4;
    const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
    const int dv0 = blockIdx.x * DVT;
    const bool wide = dv0 + 64 < a.dv;
    const int n = a.nch;
    auto chunk = [&](int m) { return REV ? n - 1 - m : m; };

    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 5);
        }
        for (int i = 0; i < 10; ++i) mbar_init(&s_ready[i], (i == 0 || i == 2 || i == 4) ? 8 : i >= 6 && i <= 8 ? 4 : 1);
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
            int issued = 0;
            bool ok = true;                 // this lane's waits so far have come to their ends
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NST, c = chunk(m), t0 = c * C, at = bh * n + c;
                if (m >= NST) ok &= wait(&empty[st], ((m / NST) - 1) & 1, abort_flag, status, ERR_TMA);
                __syncwarp();
                uint8_t* sb = sm + st * L::STAGE;
                if (elect_one() && ok) {
                    mbar_arrive_expect_tx(&full[st], L::BYTES);
                    tma_load_4d(sb + L::V_OFF, &mp.v, &full[st], 0, t0, dv0 / 64, bh);   // (slabs past dv: zeros)
                    tma_load_3d(sb + L::T_OFF, &mp.t, &full[st], 0, 0, at);
                    if (REV) tma_load_3d(sb + L::P_OFF, &mp.p, &full[st], 0, 0, at);
                    tma_load_4d(sb + L::K_OFF, &mp.k, &full[st], 0, t0, 0, bk);
                    bulk_load(sb + L::G_OFF, a.gates + (size_t)at * 8 * C, 4 * C * 4, &full[st]);
                    if (REV) tma_load_4d(sb + L::Q_OFF, &mp.q, &full[st], 0, t0, 0, bk);
                }
                __syncwarp();
                issued += ok;
            }
            // no copy may land after the CTA has ended
            if (elect_one())
                for (int m = max(0, issued - NST); m < issued; ++m) mbar_wait(&full[m % NST], (m / NST) & 1, kTimeoutNs);
            __syncwarp();
        } else if (warp == 1) {
            const uint32_t id64 = idesc_bf16(128, 64, false, false), id64n = idesc_bf16(128, 64, false, true);
            const uint32_t idS = idesc_bf16(128, DK, false, true);
            const uint32_t idV = idesc_bf16(128, 64, true, REV);
            for (int m = 0; m < n; ++m) {
                if (__any_sync(~0u, *abort_flag)) break;
                const int st = m % NST;
                const uint32_t sb = s0 + st * L::STAGE, ph = m & 1;
                const uint64_t dK = sdesc(sb + L::K_OFF, 16, 1024, kSwizzle128);
                const uint64_t dKn = sdesc(sb + L::K_OFF, SLAB, 1024, kSwizzle128);   // keys along N
                const uint64_t dQn = sdesc(sb + L::Q_OFF, SLAB, 1024, kSwizzle128);
                const uint64_t dV = sdesc(sb + L::V_OFF, SLAB, 1024, kSwizzle128);    // dv along M
                // T: forward as U^T = . T^T (rows along N, K-major), reverse as . T (columns along N)
                const uint64_t dTh = sdesc(sb + L::T_OFF, REV ? SLAB : 16, 1024, kSwizzle128);
                const uint64_t dTl = sdesc(sb + L::T_OFF + SLAB, REV ? SLAB : 16, 1024, kSwizzle128);
                const uint64_t dPh = sdesc(sb + L::P_OFF, SLAB, 1024, kSwizzle128);
                const uint64_t dPl = sdesc(sb + L::P_OFF + SLAB, SLAB, 1024, kSwizzle128);
                constexpr uint32_t step = (REV ? 2048 : 32) >> 4;   // 16 tokens of T's contraction
                wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_MMA);
                if (m > 0) wait(x_free, (m - 1) & 1, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
                    // V^T T^T, or dO^T P, both from shared memory
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint64_t v = (kk * 2048) >> 4;
                        mma_ss(tm + L::tX, dV + v, (REV ? dPh : dTh) + kk * step, idV, kk > 0);
                        mma_ss(tm + L::tX, dV + v, (REV ? dPl : dTl) + kk * step, idV, 1);
                    }
                }
                wait(s_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < DK / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * SLAB + (kk & 3) * 32) >> 4;
                        mma_ts(tm + L::tKs, tm + L::tSh + kk * 8, dK + o, id64, kk > 0);
                        mma_ts(tm + L::tKs, tm + L::tSl + kk * 8, dK + o, id64, 1);
                    }
                    mma_commit(ks_full);
                }
                if (REV) {
                    wait(y_ready, ph, abort_flag, status, ERR_MMA);
                    __syncwarp();
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < C / 16; ++kk) {
                            const uint64_t o = (kk * 2048) >> 4;
                            mma_ts(tm + L::tD, tm + L::tYh + kk * 8, dQn + o, idS, kk > 0);
                            mma_ts(tm + L::tD, tm + L::tYl + kk * 8, dQn + o, idS, 1);
                        }
                    }
                }
                wait(r_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTh + kk * step, REV ? id64n : id64, !REV || kk > 0);
                        mma_ts(tm + L::tX, tm + L::tRl + kk * 8, dTh + kk * step, REV ? id64n : id64, 1);
                        mma_ts(tm + L::tX, tm + L::tRh + kk * 8, dTl + kk * step, REV ? id64n : id64, 1);
                    }
                    mma_commit(u_full);
                }
                wait(u_ready, ph, abort_flag, status, ERR_MMA);
                __syncwarp();
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < C / 16; ++kk) {
                        const uint64_t o = (kk * 2048) >> 4;
                        mma_ts(tm + L::tD, tm + L::tRh + kk * 8, dKn + o, idS, REV || kk > 0);
                        mma_ts(tm + L::tD, tm + L::tRl + kk * 8, dKn + o, idS, 1);
                    }
                    mma_commit(d_full);
                    mma_commit(&empty[st]);
                }
                __syncwarp();
            }
            if (elect_one()) mma_commit(fin);
            __syncwarp();
            mbar_wait(fin, 0, kTimeoutNs);
        }
    } else if (wg < 3) {
        // ---------------------------------------------------------- the chain's register steps
        regs_inc<176>();
        const int grp = wg - 1, d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const int k0 = grp * HC, i0 = grp * 32;
        const bool in = dv0 + d < a.dv;
        const size_t sbase = (size_t)bh * DK * a.dv + (size_t)k0 * a.dv + dv0 + d;
        float2 s[HC / 2];
#pragma unroll
        for (int i = 0; i < HC / 2; ++i) {
            s[i].x = a.S_in && in ? a.S_in[sbase + (size_t)(2 * i) * a.dv] : 0.f;
            s[i].y = a.S_in && in ? a.S_in[sbase + (size_t)(2 * i + 1) * a.dv] : 0.f;
        }
        uint32_t hi[16], lo[16];
        for (int m = 0; m < n; ++m) {
            const int st = m % NST;
            const uint32_t ph = m & 1;
            const uint32_t gt = s0 + st * L::STAGE + L::G_OFF;
            if (__any_sync(~0u, *abort_flag)) break;
            if (m > 0) wait(sp_free, (m - 1) & 1, abort_flag, status, ERR_EPI);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HC; c += 32) {
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(s[c / 2 + i], hi[i], lo[i]);
                tmem_st16(tm + lb + L::tSh + (k0 + c) / 2, hi);
                tmem_st16(tm + lb + L::tSl + (k0 + c) / 2, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_ready);
            wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_EPI);
            const float gend = lds1(gt + (2 * C - 1) * 4);
            {
                float4 g[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = lds4(gt + ((REV ? 2 : 3) * C + i0 + 4 * i) * 4);   // l, or -e
                wait(ks_full, ph, abort_flag, status, ERR_EPI);
                tc_fence_after();
                uint32_t x[32], y[32];
                tmem_ld32(tm + lb + L::tKs + i0, x);
                if (REV) tmem_ld32(tm + lb + L::tX + i0, y);   // dO^T P: committed with K dS
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 gi = (i & 1) ? make_float2(g[i / 2].z, g[i / 2].w) : make_float2(g[i / 2].x, g[i / 2].y);
                    const float2 z = REV ? fma2(gi, f2(x[2 * i], x[2 * i + 1]), f2(y[2 * i], y[2 * i + 1]))
                                         : mul2(gi, f2(x[2 * i], x[2 * i + 1]));
                    split2(z, hi[i], lo[i]);
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
                for (int i = 0; i < 8; ++i) g[i] = lds4(gt + ((REV ? 3 : 2) * C + i0 + 4 * i) * 4);   // -e, or l
                wait(u_full, ph, abort_flag, status, ERR_EPI);
                tc_fence_after();
                uint32_t x[32];
                tmem_ld32(tm + lb + L::tX + i0, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 gi = (i & 1) ? make_float2(g[i / 2].z, g[i / 2].w) : make_float2(g[i / 2].x, g[i / 2].y);
                    split2(mul2(gi, f2(x[2 * i], x[2 * i + 1])), hi[i], lo[i]);
                }
                tmem_st16(tm + lb + L::tRh + i0 / 2, hi);
                tmem_st16(tm + lb + L::tRl + i0 / 2, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(u_ready);
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
        }
        if (a.S_out && in) {
#pragma unroll
            for (int i = 0; i < HC / 2; ++i) {
                a.S_out[sbase + (size_t)(2 * i) * a.dv] = s[i].x;
                a.S_out[sbase + (size_t)(2 * i + 1) * a.dv] = s[i].y;
            }
        }
    } else {
        // ---------------------------------------------------------- results out, four warps
        regs_dec<104>();
        const int d = (warp & 3) * 32 + lane;
        const uint32_t lb = (uint32_t)((warp & 3) * 32) << 16;
        const bool lead = threadIdx.x == NT - 128;
        const uint32_t ob = s0 + L::O_OFF;
        // the buffer's last stores must have read it; false, to all four warps, when they have to quit
        auto buffer_free = [&]() {
            if (lead) bulk_wait_read0();
            return !named_bar_any(1, 128, *abort_flag);
        };
        bool on = true;
        auto buffer_full = [&]() {
            fence_proxy_async_smem();
            named_bar_sync(1, 128);
        };
        // 32 packed values (64 of a row's bf16) of this thread's row d to slab `slab` of 128 rows
        auto put_row = [&](int slab, int c, const uint32_t (&x)[16]) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 ob + slab * 2 * SLAB + d * 128 + (((c / 8 + i) ^ (d & 7)) << 4)),
                             "r"(x[4 * i]), "r"(x[4 * i + 1]), "r"(x[4 * i + 2]), "r"(x[4 * i + 3]));
        };
        for (int m = 0; m < n; ++m) {
            const int st = m % NST, c = chunk(m), at = bh * n + c;
            const uint32_t ph = m & 1, sb = s0 + st * L::STAGE, gt = sb + L::G_OFF;
            if (REV) {
                // parts of scale e dO, dv along the lanes
                wait(&full[st], (m / NST) & 1, abort_flag, status, ERR_DRAIN);
                const uint32_t vb = sb + L::V_OFF + (d >> 6) * SLAB + (d & 7) * 2;
                const int pc = (d & 63) >> 3;
                const bool in = dv0 + d < a.dv;
#pragma unroll
                for (int t0 = 0; t0 < C; t0 += 32) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 g = lds4(gt + (C + t0 + 4 * i) * 4);
                        float v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = t0 + 4 * i + k;
                            uint16_t w;
                            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(vb + t * 128 + ((pc ^ (t & 7)) << 4)));
                            v[k] = in ? __uint_as_float((uint32_t)w << 16) * a.scale : 0.f;
                        }
                        split2(g.x * v[0], g.y * v[1], hi[2 * i], lo[2 * i]);
                        split2(g.z * v[2], g.w * v[3], hi[2 * i + 1], lo[2 * i + 1]);
                    }
                    tmem_st16(tm + lb + L::tYh + t0 / 2, hi);
                    tmem_st16(tm + lb + L::tYl + t0 / 2, lo);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(y_ready);
            }
            // the state's parts: [dv][DK] bf16 each
            wait(s_ready, ph, abort_flag, status, ERR_DRAIN);
            tc_fence_after();
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                on = on && buffer_free();
                if (!on) break;
#pragma unroll
                for (int x = 0; x < DK / 2; x += 16) {
                    uint32_t r[16];
                    tmem_ld16(tm + lb + (part ? L::tSl : L::tSh) + x, r);
                    tmem_wait_ld();
                    put_row(x / 32, (x % 32) * 2, r);
                }
                if (part) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sp_free);
                }
                buffer_full();
                if (lead) {
#pragma unroll
                    for (int i = 0; i < DK / 64; ++i)
                        tma_store_3d(part ? &mp.sl : &mp.sh, sm + L::O_OFF + i * 2 * SLAB, 64 * i, dv0, at);
                    bulk_commit();
                }
            }
            if (!on) break;
            // U: [dv][64 tokens]; dV: [64 tokens][dv]
            wait(u_full, ph, abort_flag, status, ERR_DRAIN);
            tc_fence_after();
            on = buffer_free();
            if (!on) break;
#pragma unroll
            for (int x = 0; x < C; x += 32) {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(tm + lb + L::tX + x, r);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(f2(r[2 * i], r[2 * i + 1]), hi[i], lo[i]);
                if (REV) {
                    const uint32_t o = ob + (d >> 6) * SLAB + (d & 63) * 2;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const uint16_t w = (uint16_t)((i & 1) ? hi[i / 2] >> 16 : hi[i / 2]);
                        const uint16_t z = (uint16_t)((i & 1) ? lo[i / 2] >> 16 : lo[i / 2]);
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(o + (x + i) * 128), "h"(w));
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(o + 2 * SLAB + (x + i) * 128), "h"(z));
                    }
                } else {
                    put_row(0, x, hi);
                    put_row(1, x, lo);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(x_free);
                mbar_arrive(&empty[st]);
            }
            buffer_full();
            if (lead) {
                if (REV) {
                    tma_store_3d(&mp.xh, sm + L::O_OFF, dv0, c * C, bh);
                    if (wide) tma_store_3d(&mp.xh, sm + L::O_OFF + SLAB, dv0 + 64, c * C, bh);
                    tma_store_3d(&mp.xl, sm + L::O_OFF + 2 * SLAB, dv0, c * C, bh);
                    if (wide) tma_store_3d(&mp.xl, sm + L::O_OFF + 3 * SLAB, dv0 + 64, c * C, bh);
                } else {
                    tma_store_3d(&mp.xh, sm + L::O_OFF, 0, dv0, at);
                    tma_store_3d(&mp.xl, sm + L::O_OFF + 2 * SLAB, 0, dv0, at);
                }
                bulk_commit();
            }
        }
        if (lead) bulk_wait0();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, L::TCOLS);
    }
}

bool map_box(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch, uint32_t box_rows, CUtensorMapSwizzle w)
{
    const uint64_t dims[3] = {cols, rows, batch}, str[2] = {cols * 2, cols * rows * 2};
    const uint32_t box[3] = {64, box_rows, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, w);
}

template <int DK, bool REV>
cudaError_t launch_dk(const DeltaSweep& a, const Maps& m, int* status, cudaStream_t s)
{
    using L = CL<DK, REV>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_sweep_kernel<DK, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    const dim3 g((a.dv + DVT - 1) / DVT, (unsigned)(a.B * a.H));
    gla_delta_sweep_kernel<DK, REV><<<g, NT, L::SMEM, s>>>(a, m, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_sweep(const DeltaSweep& a, int* status, cudaStream_t s)
{
    const uint64_t bk = (uint64_t)a.B * a.Hk, bh = (uint64_t)a.B * a.H, nc = bh * a.nch;
    const auto w128 = CU_TENSOR_MAP_SWIZZLE_128B, w0 = CU_TENSOR_MAP_SWIZZLE_NONE;
    Maps m;
    bool ok = map_slabs(&m.k, a.k, a.dk, a.T, bk, a.dk / 64) && map_slabs(&m.v, a.v, a.dv, a.T, bh, 2) &&
              map_pair(&m.t, a.t, nc) &&
              map_box(&m.sh, a.s_hi, a.dk, a.dv, nc, 128, w128) && map_box(&m.sl, a.s_lo, a.dk, a.dv, nc, 128, w128);
    if (a.reverse)
        ok = ok && map_slabs(&m.q, a.q, a.dk, a.T, bk, a.dk / 64) && map_pair(&m.p, a.p, nc) && map_box(&m.xh, a.x_hi, a.dv, a.T, bh, C, w0) &&
             map_box(&m.xl, a.x_lo, a.dv, a.T, bh, C, w0);
    else {
        m.q = m.p = m.k;   // not read
        ok = ok && map_box(&m.xh, a.u_hi, C, a.dv, nc, 128, w128) && map_box(&m.xl, a.u_lo, C, a.dv, nc, 128, w128);
    }
    if (!ok) return cudaErrorInvalidValue;
    if (a.reverse) return a.dk == 64 ? launch_dk<64, true>(a, m, status, s) : launch_dk<128, true>(a, m, status, s);
    return a.dk == 64 ? launch_dk<64, false>(a, m, status, s) : launch_dk<128, false>(a, m, status, s);
}

}  // namespace gla
