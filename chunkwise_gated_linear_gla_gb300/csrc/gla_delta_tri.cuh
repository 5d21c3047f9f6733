// The parts of a 64-token chunk of the gated delta rule that do not depend on the state, formed by
// eight warps of which warp w reads the tensor-memory lanes of quarter w % 4: the gates, the masked
// products L and P, and T in place of L. Used by the forward pass one chunk ahead of its chain
// (gla_delta_fused.cu) and by the backward's prep for all chunks at once (gla_delta_prep.cu).
//
// A chunk's matrices lie in shared memory as four slabs of 64 rows of 128 swizzled bytes: T, its low
// part, P, its low part. Its gates are rows of 64 floats: beta, exp(G), exp(G_end - G), -exp(G), the two
// factors of D_ij = exp(G_i - G_j) (zeros where the gate is too steep for them), G in two floats.
#pragma once

#include "gla_delta_dev.cuh"

namespace gla {
namespace delta {

constexpr int LDD = 20;           // row stride of the fp32 diagonal blocks
constexpr int kDiagBytes = 4 * 16 * LDD * 4, kExchangeBytes = 32 * 128;
constexpr float kRange = 60.f;    // |G - G_mid| up to which the two-factor form of D is used

__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }

// ---- mma.sync on 16-row pieces of a swizzled 64 x 64 bf16 matrix (128-byte rows)
__device__ __forceinline__ uint32_t sw(uint32_t base, int row, int col8) { return base + row * 128 + ((col8 ^ (row & 7)) << 4); }
__device__ __forceinline__ void ldm_a(uint32_t base, int r0, int k0, uint32_t (&a)[4])
{
    const int lane = threadIdx.x & 31;
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(sw(base, r0 + (lane & 15), k0 / 8 + (lane >> 4))) : "memory");
}
__device__ __forceinline__ void ldm_b(uint32_t base, int k0, int n0, uint32_t (&b)[2])
{
    const int lane = threadIdx.x & 31;
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                 : "=r"(b[0]), "=r"(b[1]) : "r"(sw(base, k0 + (lane & 15), n0 / 8)) : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// c (16 x 8) += Y Z over K values: Y's rows from (yr, yc) of a matrix whose low parts lie ylo bytes
// behind, or in the rows' other halves (ylo = 64); Z's from (zr, zc), low parts SLAB behind.
template <int K>
__device__ __forceinline__ void block_product(uint32_t y, int yr, int yc, uint32_t ylo, uint32_t z, int zr, int zc, float (&c)[4])
{
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t ah[4], al[4], bh[2], bl[2];
        ldm_a(y, yr, yc + k, ah);
        if (ylo == 64) ldm_a(y, yr, yc + k + 32, al);
        else ldm_a(y + ylo, yr, yc + k, al);
        ldm_b(z, zr + k, zc, bh);
        ldm_b(z + SLAB, zr + k, zc, bl);
        mma16(c, ah, bh);
        mma16(c, al, bh);
        mma16(c, ah, bl);
    }
}
// X (16 x 8 at column n0 of the block) = -(Y C) Z for K-wide pieces: Y at (yr, yc), C at (yc, zc) and Z at
// (zc, zc) of the matrix whose parts start at hi and hi + SLAB. Columns n0 .. n0 + 7 of the product.
template <int K>
__device__ __forceinline__ void block_rule(uint32_t hi, int yr, int yc, int zc, int n0, float (&x)[4])
{
    float w[K / 8][4];
#pragma unroll
    for (int i = 0; i < K / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[i][e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t ah[4], al[4];
        ldm_a(hi, yr, yc + k, ah);
        ldm_a(hi + SLAB, yr, yc + k, al);
#pragma unroll
        for (int i = 0; i < K / 8; ++i) {
            uint32_t bh[2], bl[2];
            ldm_b(hi, yc + k, zc + 8 * i, bh);
            ldm_b(hi + SLAB, yc + k, zc + 8 * i, bl);
            mma16(w[i], ah, bh);
            mma16(w[i], al, bh);
            mma16(w[i], ah, bl);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = 0.f;
#pragma unroll
    for (int k = 0; k < K; k += 16) {
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            split2(-w[k / 8 + e][0], -w[k / 8 + e][1], ah[2 * e], al[2 * e]);
            split2(-w[k / 8 + e][2], -w[k / 8 + e][3], ah[2 * e + 1], al[2 * e + 1]);
        }
        ldm_b(hi, zc + k, zc + n0, bh);
        ldm_b(hi + SLAB, zc + k, zc + n0, bl);
        mma16(x, ah, bh);
        mma16(x, al, bh);
        mma16(x, ah, bl);
    }
}
// The 16 x 8 fragment times f to rows r0.., columns c0.. of both parts (the low one as above).
__device__ __forceinline__ void put_fragment(uint32_t hi, int r0, int c0, uint32_t lo, const float (&x)[4], float f)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        uint32_t h, l;
        split2(f * x[2 * e], f * x[2 * e + 1], h, l);
        const uint32_t a = sw(hi, r0 + g + 8 * e, c0 / 8) + t * 4;
        const uint32_t b = lo == 64 ? sw(hi, r0 + g + 8 * e, c0 / 8 + 4) + t * 4 : a + lo;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(h) : "memory");
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(b), "r"(l) : "memory");
    }
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// One warp: the gates of a chunk from two tokens' log_g (x0, x1) and beta a lane, to `out`.
__device__ __forceinline__ void chunk_gates(float x0, float x1, float b0, float b1, void* out)
{
    const int lane = threadIdx.x & 31;
    // running sum of the gate over the chunk
    const bool bad = __any_sync(~0u, x0 != x0 || x1 != x1);   // a NaN gate reaches the state through exp(G)
    // below -1e5 exp() is zero whatever comes later
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
    const bool near = __all_sync(~0u, fmaxf(fabsf(d0), fabsf(d1)) <= kRange);
    const float nan = __int_as_float(0x7fc00000);
    const float e0 = bad ? nan : expf(g0.h + g0.l), e1 = bad ? nan : expf(g1.h + g1.l);
    float2* o = static_cast<float2*>(out) + lane;
    o[0] = make_float2(b0, b1);
    o[C / 2] = make_float2(e0, e1);
    o[C] = make_float2(expf(minus(end, g0)), expf(minus(end, g1)));
    o[3 * C / 2] = make_float2(-e0, -e1);
    // the factors of D (zeros where the gate is too steep for them) and G
    o[2 * C] = near ? make_float2(expf(d0), expf(d1)) : make_float2(0.f, 0.f);
    o[5 * C / 2] = near ? make_float2(expf(-d0), expf(-d1)) : make_float2(0.f, 0.f);
    o[3 * C] = make_float2(g0.h, g1.h);
    o[7 * C / 2] = make_float2(g0.l, g1.l);
}

// The 32 x 32 pieces of T and P above the diagonal, zero for good: once per buffer.
__device__ __forceinline__ void chunk_zeros(uint32_t tb, int pw)
{
    const int quarter = pw & 3, i = (quarter & 1) * 32 + (threadIdx.x & 31);
    if ((quarter & 1) || pw < 4) return;
    for (int x = 0; x < 8; ++x)
        sts4(sw(tb + (quarter >= 2 ? 2 * SLAB : 0) + (x >> 2) * SLAB, i, 4 + (x & 3)), 0u, 0u, 0u, 0u);
}

// K on Q (KK: on K again) against K, 128 tensor-memory lanes from tG, to L's pieces below the 16-row diagonal
// blocks and to P, both masked and decayed; L's diagonal blocks to fp32. A warp takes 32 rows, its quarter
// of the lanes, by 32 columns.
template <bool KK>
__device__ __forceinline__ void chunk_scores(uint32_t tG, const float* gt, float scale, uint32_t tb, float* diag, int pw)
{
    const int lane = threadIdx.x & 31, quarter = pw & 3, c0 = (pw >> 2) * 32;
    const bool isP = !KK && quarter >= 2;
    const int i = (quarter & 1) * 32 + lane;      // row of the chunk
    // of the warps' 32 x 32 pieces the one above the diagonal is zero, the one below needs no mask
    const bool above = !(quarter & 1) && c0 > 0, below = (quarter & 1) && c0 == 0;
    if (!above) {
        const bool near = gt[4 * C] != 0.f;
        const float f = isP ? scale : 1.f;
        const int last = below ? C : isP ? i : i - 1;
        const float fi = f * gt[4 * C + i];
#pragma unroll 1
        for (int c = c0; c < c0 + 32; c += 16) {
            uint32_t r[16];
            sm100::tmem_ld16(tG + ((uint32_t)(quarter * 32) << 16) + c, r);
            sm100::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < 2; ++q) {          // eight columns at a time
                const int cq = c + 8 * q;
                float2 x[4];
                if (near) {
                    const float4 u = *reinterpret_cast<const float4*>(gt + 5 * C + cq);
                    const float4 v = *reinterpret_cast<const float4*>(gt + 5 * C + cq + 4);
                    const float2 ff = make_float2(fi, fi);
                    x[0] = mul2(f2(r[8 * q], r[8 * q + 1]), mul2(ff, make_float2(u.x, u.y)));
                    x[1] = mul2(f2(r[8 * q + 2], r[8 * q + 3]), mul2(ff, make_float2(u.z, u.w)));
                    x[2] = mul2(f2(r[8 * q + 4], r[8 * q + 5]), mul2(ff, make_float2(v.x, v.y)));
                    x[3] = mul2(f2(r[8 * q + 6], r[8 * q + 7]), mul2(ff, make_float2(v.z, v.w)));
                } else {
                    const float gh = gt[6 * C + i], gl = gt[7 * C + i];
                    auto D = [&](int j) { return f * expf((gh - gt[6 * C + cq + j]) + (gl - gt[7 * C + cq + j])); };
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        x[j] = mul2(f2(r[8 * q + 2 * j], r[8 * q + 2 * j + 1]), make_float2(D(2 * j), D(2 * j + 1)));
                }
                if (!below) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[j].x = cq + 2 * j <= last ? x[j].x : 0.f;
                        x[j].y = cq + 2 * j + 1 <= last ? x[j].y : 0.f;
                    }
                }
                if (!isP && !below && (cq >> 4) == (i >> 4)) {
                    // the row's diagonal block: to fp32, times beta in its 8-row halves (which are
                    // solved), plain in the quarter below the diagonal (which enters the block rule)
                    const float be = (cq >> 3) == (i >> 3) ? gt[i] : 1.f;
                    float* dd = diag + (i >> 4) * 16 * LDD + (i & 15) * LDD + (cq & 15);
                    *reinterpret_cast<float4*>(dd) = make_float4(be * x[0].x, be * x[0].y, be * x[1].x, be * x[1].y);
                    *reinterpret_cast<float4*>(dd + 4) = make_float4(be * x[2].x, be * x[2].y, be * x[3].x, be * x[3].y);
                } else {
                    uint32_t h8[4], l8[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split2(x[e], h8[e], l8[e]);
                    const uint32_t o = sw(isP ? tb + 2 * SLAB : tb, i, cq / 8);
                    sts4(o, h8[0], h8[1], h8[2], h8[3]);
                    sts4(o + SLAB, l8[0], l8[1], l8[2], l8[3]);
                }
            }
        }
    }
}

// T in place of L, from the diagonal blocks up. All 256 threads; ends without a barrier. `read` is called
// once the fp32 diagonal blocks are done with. False, to all of them, and nothing more done if one has to quit.
template <typename F>
__device__ __forceinline__ bool chunk_inverse(uint32_t tb, uint32_t wb, const float* gt, float* diag, int pw, bool quit, F read)
{
    const int lane = threadIdx.x & 31;
    if (pw < 4) {
        // The 16-row diagonal block `pw`, in place in fp32: its two 8-row halves by forward
        // substitution, a lane per column, then the block rule, two outputs a lane.
        const int cc = lane & 7, rr = lane >> 3, hb = rr & 1;
        float* B = diag + pw * 16 * LDD;
        float* A = B + hb * 8 * (LDD + 1);
        float x[8];
#pragma unroll
        for (int ii = 0; ii < 8; ++ii) {
            float u = ii == cc ? 1.f : 0.f, v = 0.f;
            if (ii > 0) {
                const float4 q = *reinterpret_cast<const float4*>(A + ii * LDD);
                u = fmaf(-q.x, x[0], u);
                if (ii > 1) v = fmaf(-q.y, x[1], v);
                if (ii > 2) u = fmaf(-q.z, x[2], u);
                if (ii > 3) v = fmaf(-q.w, x[3], v);
            }
            if (ii > 4) {
                const float4 q = *reinterpret_cast<const float4*>(A + ii * LDD + 4);
                u = fmaf(-q.x, x[4], u);
                if (ii > 5) v = fmaf(-q.y, x[5], v);
                if (ii > 6) u = fmaf(-q.z, x[6], u);
            }
            x[ii] = u + v;
        }
        const float be = gt[16 * pw + 8 * hb + cc];
        __syncwarp();                        // the half's rows are read
        if (lane < 16) {
#pragma unroll
            for (int ii = 0; ii < 8; ++ii) A[ii * LDD + cc] = be * x[ii];
        }
        __syncwarp();
        float w[2] = {0.f, 0.f}, y[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 8; ++k) {        // rows rr and rr + 4 of C Z
            const float z = B[k * LDD + cc];
            w[0] = fmaf(B[(8 + rr) * LDD + k], z, w[0]);
            w[1] = fmaf(B[(12 + rr) * LDD + k], z, w[1]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {        // and of -Y (C Z)
            const float z = __shfl_sync(~0u, w[k >> 2], (k & 3) * 8 + cc);
            y[0] = fmaf(-B[(8 + rr) * LDD + 8 + k], z, y[0]);
            y[1] = fmaf(-B[(12 + rr) * LDD + 8 + k], z, y[1]);
        }
        __syncwarp();                        // C is read
        B[(8 + rr) * LDD + cc] = y[0];
        B[(12 + rr) * LDD + cc] = y[1];
        __syncwarp();
        const int row = lane >> 1, col = (lane & 1) * 8;
        uint32_t h8[4], l8[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float4 q = *reinterpret_cast<const float4*>(B + row * LDD + col + 4 * e);
            split2(q.x, q.y, h8[2 * e], l8[2 * e]);
            split2(q.z, q.w, h8[2 * e + 1], l8[2 * e + 1]);
        }
        const uint32_t o = sw(tb, 16 * pw + row, 2 * pw + (lane & 1));
        sts4(o, h8[0], h8[1], h8[2], h8[3]);
        sts4(o + SLAB, l8[0], l8[1], l8[2], l8[3]);
    }
    if (named_bar_any(2, 256, quit)) return false;
    read();
    {
        // 16 -> 32, eight columns a warp for each of the two pairs
        float x[4];
        const int o = 32 * (pw >> 1), n0 = (pw & 1) * 8;
        if (pw < 4) block_rule<16>(tb, o + 16, o + 16, o, n0, x);
        sm100::named_bar_sync(2, 256);
        if (pw < 4) put_fragment(tb, o + 16, o + n0, SLAB, x, 1.f);
    }
    sm100::named_bar_sync(2, 256);
    {
        // 32 -> 64: 16 rows by eight columns a warp, Y C by way of shared memory
        const int r0 = (pw >> 2) * 16, n0 = (pw & 3) * 8;
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        block_product<32>(tb, 32 + r0, 32, SLAB, tb, 32, n0, x);
        put_fragment(wb, r0, n0, 64, x, -1.f);
        sm100::named_bar_sync(2, 256);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = 0.f;
        block_product<32>(wb, r0, 0, 64, tb, 0, n0, x);
        put_fragment(tb, 32 + r0, n0, SLAB, x, 1.f);
    }
    return true;
}

}  // namespace delta
}  // namespace gla
