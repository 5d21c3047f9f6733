// Device helpers shared by the chunk form's kernels of the gated delta rule.
#pragma once

#include <cuda_bf16.h>

#include "gla_internal.h"
#include "sm100.cuh"
#include "tma_host.h"

namespace gla {
namespace delta {

constexpr int C = kChunk;
constexpr int SLAB = C * 128;                     // 64 rows of 128 bytes: one swizzled TMA box
constexpr uint64_t kTimeoutNs = 2000000000ull;    // of the waits, after a role's loop, for what is in flight

// One lane of a converged warp. Code that issues from an elected lane of a warp whose control
// flow is uniform keeps its addresses and descriptors in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(sm100::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(sm100::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A CTA's abort flag and the time at which its waits give up: between 4.3 and 8.6 seconds after its
// start (the upper word of the nanosecond clock, two steps on).
struct Abort {
    volatile int* flag;
    uint32_t deadline;
    __device__ __forceinline__ explicit Abort(void* p) : flag(static_cast<volatile int*>(p)) {
        asm volatile("mov.u32 %0, %%globaltimer_hi;" : "=r"(deadline));
        deadline += 2;
    }
    __device__ __forceinline__ volatile int& operator*() const { return *flag; }
};

// Bounded wait; false when it runs out. All of a CTA's roles give up at the same time; the status word
// reports it. From then on
//   - a thread that issues copies issues none any more (its own waits tell it; of the products, which stay in
//     the CTA's own memories, the rest of a chunk's may follow: asking at each costs the passes 3%),
//   - roles leave their loops at the next look at the flag: a warp on its own by a vote, warps that share
//     a named barrier by that barrier's word (the same for all of them); until then they go on without
//     waiting, on what their buffers hold,
//   - who issued copies or products waits for them, with a limit of its own, before the CTA frees its
//     tensor memory and ends.
// The loop is short on purpose: it is copied to every wait, and code that pushes the roles' steps out of
// the instruction caches costs them dearly.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Abort& abort_flag, int* status, int code)
{
#pragma unroll 1
    while (!sm100::mbar_try_wait(bar, parity)) {
        uint32_t now;
        asm volatile("mov.u32 %0, %%globaltimer_hi;" : "=r"(now));
        if ((int)(now - abort_flag.deadline) >= 0) {
            *abort_flag = 1;
            atomicExch(status, code);
            return false;
        }
    }
    return true;
}

// bar.sync of `n` threads that tells all of them the same: whether any of them said yes.
__device__ __forceinline__ bool named_bar_any(int id, int n, bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
                 "bar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(id), "r"(n), "r"((uint32_t)x) : "memory");
    return r != 0;
}

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// a b + c on two fp32 values in one packed instruction (each half rounds as fmaf).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// x in two bf16 parts: hi = bf16(x), lo = bf16(x - hi); |x - hi - lo| <= 2^-17 |x|.
__device__ __forceinline__ void split2(float2 x, uint32_t& hi, uint32_t& lo)
{
    hi = sm100::pack_bf16(x.x, x.y);
    const float2 r = fma2(make_float2(bf_lo(hi), bf_hi(hi)), make_float2(-1.f, -1.f), x);
    lo = sm100::pack_bf16(r.x, r.y);
}
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    split2(make_float2(x0, x1), hi, lo);
}

// A sum of floats kept with its rounding errors (Knuth's two-sum, renormalised).
struct Two { float h, l; };
__device__ __forceinline__ Two two_add(Two a, Two b)
{
    const float s = __fadd_rn(a.h, b.h), t = __fadd_rn(s, -a.h);
    const float e = __fadd_rn(__fadd_rn(a.h, -__fadd_rn(s, -t)), __fadd_rn(b.h, -t)) + (a.l + b.l);
    const float h = __fadd_rn(s, e);
    return Two{h, __fadd_rn(e, -__fadd_rn(h, -s))};
}

// Shared-memory accesses by 32-bit address. A pointer into the aligned dynamic buffer is generic
// to the compiler, and a generic load may not pass a generic store; these stay in order among
// the volatile statements around them (waits, fences) and overlap freely otherwise.
__device__ __forceinline__ float4 lds4(uint32_t a)
{
    float4 f;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w) : "r"(a));
    return f;
}
__device__ __forceinline__ float lds1(uint32_t a)
{
    float f;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a));
    return f;
}
__device__ __forceinline__ void sts_bf16(uint32_t a, float x)
{
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(a), "h"(*reinterpret_cast<const uint16_t*>(&h)));
}

// Row-major [rows][cols] bf16 with a batch dimension, in boxes of 64 columns x 64 rows.
inline bool map_rows(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch)
{
    const uint64_t dims[3] = {cols, rows, batch}, str[2] = {cols * 2, cols * rows * 2};
    const uint32_t box[3] = {64, C, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// The same rows of `slabs` 64-column slabs in one box: each slab's 64 rows after the other's.
inline bool map_slabs(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t batch, uint32_t slabs)
{
    const uint64_t dims[4] = {64, rows, cols / 64, batch}, str[3] = {cols * 2, 128, cols * rows * 2};
    const uint32_t box[4] = {64, C, slabs, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// The prep's 64 x 64 matrices, both parts in one box of 128 rows.
inline bool map_pair(CUtensorMap* m, const void* base, uint64_t chunks)
{
    const uint64_t dims[3] = {C, 2 * C, chunks}, str[2] = {C * 2, 2 * C * C * 2};
    const uint32_t box[3] = {C, 2 * C, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace delta
}  // namespace gla
