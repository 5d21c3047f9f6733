// gla_delta_prep: what the backward's sweeps (gla_delta_bwd_chain.cu) need of every 64-token chunk
// and does not depend on the state; the forward pass forms the same on the fly (gla_delta_fused.cu). Within a chunk the corrections u solve
//
//     u_i = beta_i (v_i - exp(G_i) k_i S) - sum_{j<i} A_ij u_j,
//     A_ij = beta_i (k_i . k_j) exp(G_i - G_j),
//
// so U = T (V - exp(G) K S) with T = (I + A)^-1 diag(beta). This kernel forms T and the scores
// P_ij = scale (q_i . k_j) exp(G_i - G_j).
//
// Products: one tcgen05 product of 128 rows, K stacked on Q, against K^T. The inverse of the
// unit lower triangular I + A in fp32: the four 16-row diagonal blocks by forward substitution
// (a warp each, a lane per column), then twice the block rule: the inverse of
// [[X, 0], [C, Y]] has -Y^-1 C X^-1 below. G is summed in pairs of floats (48 bits), so a
// steep gate costs no precision; exp(G_i - G_j) is a product of two factors around the chunk's
// middle while both stay within e^60, else one exponential per score. T leaves in two bf16
// parts (hi + lo, 17 bits), as the state's error has to stay below 1e-5.
//
// One CTA of eight warps per chunk and head, four per SM (53 KB of shared memory at dk = 128,
// 64 registers), so that one's substitution hides behind the others' loads and products.
#include "gla_delta_dev.cuh"
#include "gla_delta_internal.h"

namespace gla {
namespace {

using namespace sm100;
using namespace delta;

constexpr int NT = 256;
constexpr int LD = 68;            // row stride of the fp32 matrices: 16-byte rows, conflict-free
constexpr float kRange = 60.f;    // |G - G_mid| up to which the two-factor form is used

enum { ERR_LOAD = 0x601, ERR_MMA = 0x602 };

template <int DK>
struct PL {
    static constexpr int TILES = 2 * (DK / 64) * SLAB;        // [K slab, Q slab] per 64 keys
    static constexpr int T_OFF = 0;                            // the inverse, over the tiles once multiplied
    static constexpr int Y_OFF = C * LD * 4;                   // 32 x 36 floats
    static constexpr int TY = Y_OFF + 32 * 36 * 4;
    static constexpr int A_OFF = TILES > TY ? TILES : (TY + 1023) / 1024 * 1024;
    static constexpr int G_OFF = A_OFF + C * LD * 4;           // G, its factors, beta
    static constexpr int BAR_OFF = G_OFF + 6 * C * 4;
    static constexpr int SMEM = BAR_OFF + 64 + 1024;
};

// a (2 x 4 outputs) += L rows i, i + 1 (k = 0..N-1) times R (rows k, four columns), both row-major
// with stride LD or LDR; four k per step.
template <int N, int LDR>
__device__ __forceinline__ void block_product(const float* l0, const float* l1, const float* r, float2 (&y)[2][2])
{
#pragma unroll 4
    for (int k = 0; k < N; k += 4) {
        const float4 p = *reinterpret_cast<const float4*>(l0 + k), q = *reinterpret_cast<const float4*>(l1 + k);
        const float pa[4] = {p.x, p.y, p.z, p.w}, qa[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 x = *reinterpret_cast<const float4*>(r + (k + e) * LDR);
            y[0][0] = fma2(make_float2(pa[e], pa[e]), make_float2(x.x, x.y), y[0][0]);
            y[0][1] = fma2(make_float2(pa[e], pa[e]), make_float2(x.z, x.w), y[0][1]);
            y[1][0] = fma2(make_float2(qa[e], qa[e]), make_float2(x.x, x.y), y[1][0]);
            y[1][1] = fma2(make_float2(qa[e], qa[e]), make_float2(x.z, x.w), y[1][1]);
        }
    }
}

template <int DK>
__global__ void __launch_bounds__(NT, 4)
gla_delta_prep_kernel(DeltaPrep a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                      int* status)
{
    using L = PL<DK>;
    extern __shared__ uint8_t raw[];
    uint8_t* sm = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float* T = reinterpret_cast<float*>(sm + L::T_OFF);
    float* Y = reinterpret_cast<float*>(sm + L::Y_OFF);
    float* A = reinterpret_cast<float*>(sm + L::A_OFF);
    float* gh = reinterpret_cast<float*>(sm + L::G_OFF);   // G, high part
    float* gl = gh + C;                                    // G, low part
    float* fa = gl + C;                                    // exp(G - G_mid)
    float* fb = fa + C;                                    // exp(G_mid - G)
    float* be = fb + C;                                    // beta
    float* mx = be + C;                                    // [0]: max |G - G_mid|
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + L::BAR_OFF);   // loaded, multiplied
    uint32_t* holder = reinterpret_cast<uint32_t*>(bar + 2);
    const Abort abort_flag(bar + 3);

    const int tid = threadIdx.x, warp = __shfl_sync(~0u, tid / 32, 0), lane = tid % 32;
    const int c = blockIdx.x % a.nch, bhi = blockIdx.x / a.nch;
    const int b = bhi / a.H, h = bhi % a.H;
    const long long bh = bhi;
    const int bk = b * a.Hk + h / (a.H / a.Hk);
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
        // running sum of the gate over the chunk, two tokens a lane; tokens past T: no decay
        const float* lg = a.log_g ? a.log_g + bh * a.T : nullptr;
        const __nv_bfloat16* bp = static_cast<const __nv_bfloat16*>(a.beta) + bh * a.T;
        const int t = t0 + 2 * lane;
        float x0 = lg && t < a.T ? lg[t] : 0.f, x1 = lg && t + 1 < a.T ? lg[t + 1] : 0.f;
        float b0 = t < a.T ? __bfloat162float(bp[t]) : 0.f, b1 = t + 1 < a.T ? __bfloat162float(bp[t + 1]) : 0.f;
        if (a.beta_floor > 0.f) {
            if (t < a.T && fabsf(b0) < a.beta_floor) b0 = a.beta_floor;
            if (t + 1 < a.T && fabsf(b1) < a.beta_floor) b1 = a.beta_floor;
        }
        // below -1e5 exp() is zero whatever comes later
        const bool bad = __any_sync(~0u, x0 != x0 || x1 != x1);   // a NaN gate reaches the state through exp(G)
        x0 = fminf(fmaxf(x0, -1e5f), 1e5f);
        x1 = fminf(fmaxf(x1, -1e5f), 1e5f);
        Two s = two_add(Two{x0, 0.f}, Two{x1, 0.f});
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Two y = {__shfl_up_sync(~0u, s.h, o), __shfl_up_sync(~0u, s.l, o)};
            if (lane >= o) s = two_add(s, y);
        }
        const Two g1 = s, g0 = two_add(s, Two{-x1, 0.f});
        const Two mid = {__shfl_sync(~0u, g1.h, 15), __shfl_sync(~0u, g1.l, 15)};   // G at token 31
        const Two end = {__shfl_sync(~0u, g1.h, 31), __shfl_sync(~0u, g1.l, 31)};
        auto minus = [](Two x, Two y) { return (x.h - y.h) + (x.l - y.l); };
        const float d0 = minus(g0, mid), d1 = minus(g1, mid);
        float m = fmaxf(fabsf(d0), fabsf(d1));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if (lane == 0) mx[0] = m;
        const int i = 2 * lane;
        gh[i] = g0.h; gh[i + 1] = g1.h;
        gl[i] = g0.l; gl[i + 1] = g1.l;
        fa[i] = expf(d0); fa[i + 1] = expf(d1);
        fb[i] = expf(-d0); fb[i + 1] = expf(-d1);
        be[i] = b0; be[i + 1] = b1;
        const float nan = __int_as_float(0x7fc00000);
        const float e0 = bad ? nan : expf(g0.h + g0.l), e1 = bad ? nan : expf(g1.h + g1.l);
        float2* go = reinterpret_cast<float2*>(a.gates + (bh * a.nch + c) * 8 * C) + lane;
        go[0] = make_float2(b0, b1);
        go[C / 2] = make_float2(e0, e1);
        go[C] = make_float2(expf(minus(end, g0)), expf(minus(end, g1)));
        go[3 * C / 2] = make_float2(-e0, -e1);
        // for the gradients: the factors of exp(G_i - G_j) (zeros where the chunk's gate is too
        // steep for them), and G
        const bool near = m <= kRange;
        go[2 * C] = near ? make_float2(fa[i], fa[i + 1]) : make_float2(0.f, 0.f);
        go[5 * C / 2] = near ? make_float2(fb[i], fb[i + 1]) : make_float2(0.f, 0.f);
        go[3 * C] = make_float2(g0.h, g1.h);
        go[7 * C / 2] = make_float2(g0.l, g1.l);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tD = *holder;
    if (warp == 1) {
        wait(&bar[0], 0, abort_flag, status, ERR_LOAD);
        __syncwarp();
        const uint32_t id = idesc_bf16(128, 64, false, false);
        const uint64_t d0 = sdesc(smem_u32(sm), 16, 1024, kSwizzle128);   // K on Q: 128 rows; K alone: 64
        if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < DK / 16; ++kk) {
                const uint64_t d = d0 + (((kk >> 2) * 2 * SLAB + (kk & 3) * 32) >> 4);
                mma_ss(tD, d, d, id, kk > 0);
            }
            mma_commit(&bar[1]);
        }
        __syncwarp();
    }
    wait(&bar[1], 0, abort_flag, status, ERR_MMA);
    __syncthreads();     // the tiles are read: the inverse may take their place
    tc_fence_after();

    {
        // tensor-memory lanes 0-63: rows of A, to shared memory; 64-127: rows of P, to global
        // memory; warps 0-3 the first 32 columns, 4-7 the others
        const int quarter = warp & 3, c0 = (warp >> 2) * 32;
        const int i = (quarter & 1) * 32 + lane;
        const bool isP = quarter >= 2, near = mx[0] <= kRange;
        const float f = isP ? a.scale : be[i];
        const int last = isP ? i : i - 1;
        uint32_t r[32];
        tmem_ld32(tD + ((uint32_t)(quarter * 32) << 16) + c0, r);
        tmem_wait_ld();
        tc_fence_before();
        float x[32];
        if (near) {
            const float fi = f * fa[i];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 q = *reinterpret_cast<const float4*>(fb + c0 + j);
                x[j] = __uint_as_float(r[j]) * (fi * q.x);
                x[j + 1] = __uint_as_float(r[j + 1]) * (fi * q.y);
                x[j + 2] = __uint_as_float(r[j + 2]) * (fi * q.z);
                x[j + 3] = __uint_as_float(r[j + 3]) * (fi * q.w);
            }
        } else {
            const float hi_i = gh[i], lo_i = gl[i];
#pragma unroll
            for (int j = 0; j < 32; ++j)
                x[j] = f * __uint_as_float(r[j]) * expf((hi_i - gh[c0 + j]) + (lo_i - gl[c0 + j]));
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = c0 + j <= last ? x[j] : 0.f;
        if (!isP) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(A + i * LD + c0 + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        } else {
            uint4* ph = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.p) + ((bh * a.nch + c) * 2 * C + i) * C + c0);
            uint4* pl = ph + C * C / 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h8[4], l8[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) split2(x[8 * j + 2 * e], x[8 * j + 2 * e + 1], h8[e], l8[e]);
                ph[j] = make_uint4(h8[0], h8[1], h8[2], h8[3]);
                pl[j] = make_uint4(l8[0], l8[1], l8[2], l8[3]);
            }
        }
    }
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tD, 64);
    }
    if (warp < 4) {
        // diagonal block `warp`: column cc of its inverse by forward substitution, a lane each
        const int o = warp * 16, cc = lane & 15;
        float2 x[8];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float2 s0 = make_float2(i == cc ? 1.f : 0.f, 0.f), s1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                // A is zero from its diagonal on, and the x there are not yet set: leave them out
                const float4 r = *reinterpret_cast<const float4*>(A + (o + i) * LD + o + j);
                if (j + 1 < i) s0 = fma2(make_float2(-r.x, -r.y), x[j / 2], s0);
                else s0.x = fmaf(-r.x, x[j / 2].x, s0.x);
                if (j + 3 < i) s1 = fma2(make_float2(-r.z, -r.w), x[j / 2 + 1], s1);
                else if (j + 2 < i) s1.x = fmaf(-r.z, x[j / 2 + 1].x, s1.x);
            }
            const float v = (s0.x + s0.y) + (s1.x + s1.y);
            if (i & 1) x[i / 2].y = v;
            else x[i / 2].x = v;
        }
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) T[(o + i) * LD + o + cc] = (i & 1) ? x[i / 2].y : x[i / 2].x;
        }
    }
    __syncthreads();
    {
        // 16 -> 32: the lower-left block of pair p, 2 x 4 outputs a thread (32 threads a pair)
        const int p = tid >> 5, i = (tid & 31) >> 2 << 1, cc = (tid & 3) * 4, o = 32 * p;
        if (tid < 64) {
            float2 y[2][2] = {};
            block_product<16, LD>(A + (o + 16 + i) * LD + o, A + (o + 17 + i) * LD + o, T + o * LD + o + cc, y);
            float* yo = Y + (16 * p + i) * 36 + cc;
            *reinterpret_cast<float4*>(yo) = make_float4(y[0][0].x, y[0][0].y, y[0][1].x, y[0][1].y);
            *reinterpret_cast<float4*>(yo + 36) = make_float4(y[1][0].x, y[1][0].y, y[1][1].x, y[1][1].y);
            __syncwarp();
            float2 z[2][2] = {};
            block_product<16, 36>(T + (o + 16 + i) * LD + o + 16, T + (o + 17 + i) * LD + o + 16, Y + 16 * p * 36 + cc, z);
            float* to = T + (o + 16 + i) * LD + o + cc;
            *reinterpret_cast<float4*>(to) = make_float4(-z[0][0].x, -z[0][0].y, -z[0][1].x, -z[0][1].y);
            *reinterpret_cast<float4*>(to + LD) = make_float4(-z[1][0].x, -z[1][0].y, -z[1][1].x, -z[1][1].y);
        } else if (tid < 192) {
            // the pairs' upper-right blocks are zero (read as such below)
            const int q = (tid - 64) >> 6, r = ((tid - 64) & 63) >> 2, x = (tid & 3) * 4;
            *reinterpret_cast<float4*>(T + (32 * q + r) * LD + 32 * q + 16 + x) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __syncthreads();
    {
        // 32 -> 64: 2 x 4 outputs for each of 128 threads
        const int i = (tid & 127) >> 3 << 1, cc = (tid & 7) * 4;
        if (tid < 128) {
            float2 y[2][2] = {};
            block_product<32, LD>(A + (32 + i) * LD, A + (33 + i) * LD, T + cc, y);
            float* yo = Y + i * 36 + cc;
            *reinterpret_cast<float4*>(yo) = make_float4(y[0][0].x, y[0][0].y, y[0][1].x, y[0][1].y);
            *reinterpret_cast<float4*>(yo + 36) = make_float4(y[1][0].x, y[1][0].y, y[1][1].x, y[1][1].y);
            named_bar_sync(1, 128);
            float2 z[2][2] = {};
            block_product<32, 36>(T + (32 + i) * LD + 32, T + (33 + i) * LD + 32, Y + cc, z);
            float* to = T + (32 + i) * LD + cc;
            *reinterpret_cast<float4*>(to) = make_float4(-z[0][0].x, -z[0][0].y, -z[0][1].x, -z[0][1].y);
            *reinterpret_cast<float4*>(to + LD) = make_float4(-z[1][0].x, -z[1][0].y, -z[1][1].x, -z[1][1].y);
        }
    }
    __syncthreads();
    {
        // T diag(beta) in two parts: a quarter of a row a thread, zero above the diagonal
        const int i = tid >> 2, c0 = (tid & 3) * 16;
        uint4* th = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.t) + ((bh * a.nch + c) * 2 * C + i) * C + c0);
        uint4* tl = th + C * C / 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            uint32_t h8[4], l8[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = c0 + 8 * j + 4 * e;
                float4 f = *reinterpret_cast<const float4*>(T + i * LD + col);
                const float4 g = *reinterpret_cast<const float4*>(be + col);
                f.x = col <= i ? f.x * g.x : 0.f; f.y = col + 1 <= i ? f.y * g.y : 0.f;
                f.z = col + 2 <= i ? f.z * g.z : 0.f; f.w = col + 3 <= i ? f.w * g.w : 0.f;
                split2(f.x, f.y, h8[2 * e], l8[2 * e]);
                split2(f.z, f.w, h8[2 * e + 1], l8[2 * e + 1]);
            }
            th[j] = make_uint4(h8[0], h8[1], h8[2], h8[3]);
            tl[j] = make_uint4(l8[0], l8[1], l8[2], l8[3]);
        }
    }
}

template <int DK>
cudaError_t launch_dk(const DeltaPrep& a, const CUtensorMap& k, const CUtensorMap& q, int* status, cudaStream_t s)
{
    using L = PL<DK>;
    cudaError_t e = cudaFuncSetAttribute(gla_delta_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
    if (e != cudaSuccess) return e;
    gla_delta_prep_kernel<DK><<<(unsigned)((long long)a.B * a.H * a.nch), NT, L::SMEM, s>>>(a, k, q, status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_prep(const DeltaPrep& a, int* status, cudaStream_t s)
{
    CUtensorMap mk, mq;
    const uint64_t bk = (uint64_t)a.B * a.Hk;
    if (!map_rows(&mk, a.k, a.dk, a.T, bk) || !map_rows(&mq, a.q, a.dk, a.T, bk)) return cudaErrorInvalidValue;
    return a.dk == 64 ? launch_dk<64>(a, mk, mq, status, s) : launch_dk<128>(a, mk, mq, status, s);
}

}  // namespace gla
