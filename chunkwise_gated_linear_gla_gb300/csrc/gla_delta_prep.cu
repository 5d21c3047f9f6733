// gla_delta_prep: what the backward's sweeps (gla_delta_bwd_chain.cu) need of every 64-token chunk
// and does not depend on the state, for all chunks at once; the forward pass forms the same on the
// fly (gla_delta_fused.cu). Within a chunk the corrections u solve
//
//     u_i = beta_i (v_i - exp(G_i) k_i S - sum_{j<i} L_ij u_j),   L_ij = (k_i . k_j) exp(G_i - G_j),
//
// so U = T (V - exp(G) K S) with T = (1 / beta + L)^-1. This kernel writes T, the scores
// P_ij = scale (q_i . k_j) exp(G_i - G_j), both in two bf16 parts (17 bits: the gate's gradient needs
// them), and the gates. One tcgen05 product of 128 rows, K stacked on Q, against K^T; then the steps
// of gla_delta_tri.cuh in the tiles' place.
//
// One CTA of eight warps per chunk and head, several per SM (76 KB less the tiles that T and P
// replace: 44 KB at dk = 128), so that one's solving hides behind the others' loads. Bound by its 66 KB
// of traffic a chunk and by the latency of the solve about equally: 4096 chunks in 49 us, 5.5 TB/s.
#include "gla_delta_dev.cuh"
#include "gla_delta_tri.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 256;

enum { ERR_LOAD = 0x601, ERR_MMA = 0x602 };

template <int DK>
struct PL {
    static constexpr int TILES = 2 * (DK / 64) * SLAB;        // [K slab, Q slab] per 64 keys; then T and P
    static constexpr int G_OFF = 4 * SLAB;
    static constexpr int W_OFF = G_OFF + 8 * C * 4;
    static constexpr int D_OFF = W_OFF + kExchangeBytes;
    static constexpr int BAR_OFF = D_OFF + kDiagBytes;
    static constexpr int SMEM = BAR_OFF + 64 + 1024;
};

template <int DK>
__global__ void __launch_bounds__(NT, 4)
gla_delta_prep_kernel(DeltaPrep a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmT, const __grid_constant__ CUtensorMap tmP, int* status)
{
    using L = PL<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t s0 = smem_u32(sm);
    float* gt = reinterpret_cast<float*>(sm + L::G_OFF);
    float* diag = reinterpret_cast<float*>(sm + L::D_OFF);
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);   // loaded, multiplied
    uint32_t* holder = reinterpret_cast<uint32_t*>(bar + 2);
    const Abort abort_flag(bar + 3);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
    const int at = blockIdx.x, c = at % a.nch, bh = at / a.nch;
    const int b = bh / a.H, h = bh % a.H, bk = b * a.Hk + h / (a.H / a.Hk);
    const int t0 = c * C;

    if (warp == 1) {
        if (lane == 0) {
            mbar_init(&bar[0], 1);
            mbar_init(&bar[1], 1);
            *abort_flag = 0;
            mbar_fence_init();
            mbar_arrive_expect_tx(&bar[0], L::TILES);
#pragma unroll
            for (int i = 0; i < DK / 64; ++i) {
                tma_load_3d(sm + 2 * i * SLAB, &tmK, &bar[0], 64 * i, t0, bk);
                tma_load_3d(sm + (2 * i + 1) * SLAB, &tmQ, &bar[0], 64 * i, t0, bk);
            }
        }
        __syncwarp();
        tmem_alloc(holder, 64);
        tmem_relinquish();
    }
    if (warp == 0) {
        const int t = t0 + 2 * lane;
        const bool p = t < a.T, q = t + 1 < a.T;      // tokens past T: no decay, beta 0
        const float* lg = a.log_g ? a.log_g + (long long)bh * a.T : nullptr;
        const __nv_bfloat16* bp = static_cast<const __nv_bfloat16*>(a.beta) + (long long)bh * a.T;
        const float x0 = lg && p ? lg[t] : 0.f, x1 = lg && q ? lg[t + 1] : 0.f;
        float b0 = p ? __bfloat162float(bp[t]) : 0.f, b1 = q ? __bfloat162float(bp[t + 1]) : 0.f;
        if (p && fabsf(b0) < a.beta_floor) b0 = a.beta_floor;
        if (q && fabsf(b1) < a.beta_floor) b1 = a.beta_floor;
        chunk_gates(x0, x1, b0, b1, gt);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tD = *holder;
    bool ok = true, issued = false;     // this thread's waits have come to their ends; it has products in flight
    if (tid < 8 * C / 4)
        reinterpret_cast<float4*>(a.gates + (size_t)at * 8 * C)[tid] = reinterpret_cast<const float4*>(gt)[tid];
    if (warp == 1) {
        ok = wait(&bar[0], 0, abort_flag, status, ERR_LOAD);
        __syncwarp();
        const uint32_t id = idesc_bf16(128, 64, false, false);
        const uint64_t d0 = sdesc(s0, 16, 1024, kSwizzle128);   // K on Q: 128 rows; K alone: 64
        if (elect_one() && ok) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint64_t d = d0 + (((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4);
                mma_ss(tD, d, d, id, kk > 0);
            }
            mma_commit(&bar[1]);
            issued = true;
        }
        __syncwarp();
    }
    ok &= wait(&bar[1], 0, abort_flag, status, ERR_MMA);
    if (__syncthreads_or(!ok)) {
        // given up: what is in flight is waited for before the memory that it uses is left
        if (warp == 1) {
            mbar_wait(&bar[0], 0, kTimeoutNs);
            if (issued) mbar_wait(&bar[1], 0, kTimeoutNs);
            __syncwarp();
            tmem_dealloc(tD, 64);
        }
        return;
    }
    // the tiles are read: T and P may take their place
    tc_fence_after();
    chunk_zeros(s0, warp);
    chunk_scores<false>(tD, gt, a.scale, s0, diag, warp);
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tD, 64);
    }
    chunk_inverse(s0, s0 + L::W_OFF, gt, diag, warp, false, [] {});
    fence_proxy_async_smem();
    __syncthreads();
    if (warp == 1) {
        if (elect_one()) {
            tma_store_3d(&tmT, sm, 0, 0, at);
            tma_store_3d(&tmP, sm + 2 * SLAB, 0, 0, at);
            bulk_commit();
            bulk_wait_read0();
        }
        __syncwarp();
    }
}

template <int DK>
cudaError_t launch_dk(const DeltaPrep& a, const CUtensorMap (&m)[4], int* status, cudaStream_t s)
{
    using L = PL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    gla_delta_prep_kernel<DK><<<(unsigned)((long long)a.B * a.H * a.nch), NT, L::SMEM, s>>>(a, m[0], m[1], m[2], m[3], status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaPrep& a, int* status, cudaStream_t s)
{
    CUtensorMap m[4];
    const uint64_t bk = (uint64_t)a.B * a.Hk, nc = (uint64_t)a.B * a.H * a.nch;
    if (!map_rows(&m[0], a.k, a.dk, a.T, bk) || !map_rows(&m[1], a.q, a.dk, a.T, bk) || !map_pair(&m[2], a.t, nc) ||
        !map_pair(&m[3], a.p, nc))
        return cudaErrorInvalidValue;
    return a.dk == 64 ? launch_dk<64>(a, m, status, s) : launch_dk<128>(a, m, status, s);
}

}  // namespace gla
