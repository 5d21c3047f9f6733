// Internal declarations of the gated delta rule: the planner in gla_delta_api.cu and the
// kernel launchers. Not part of the public ABI (include/gla.h is).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "gla_internal.h"

namespace gla {

constexpr int kDeltaMaxDk = 256;    // widest keys of the recurrent form (its state rows per thread)
// AUTO: the shortest call that the chunk form takes. With 128 heads (dk = dv = 128) 9 tokens are 14 us
// against 18 in the recurrent form; with 4 to 16 heads both are launch latency up to 24 tokens (13 us).
constexpr int kDeltaChunkMinT = 9, kDeltaChunkMinTFew = 24, kDeltaFewTiles = 64;
// The longest: a CTA that walks 2^25 tokens (half a million chunks at 3.3 us) is done within the four
// seconds after which its waits give up.
constexpr int kDeltaChunkMaxT = 1 << 25;
// The longest sequence of the recurrent form: it counts tokens in steps of 16, and the step past the last
// token stays an int.
constexpr int kDeltaMaxT = 0x7fffffff - 15;
constexpr int kDeltaKeep = 16;      // recurrent backward: tokens between two kept states

// The recurrent form (gla_delta_step.cu): the recurrence token by token, the state tile in
// registers. With `keep` non-null, the state entering every kDeltaKeep-th token goes there
// ([BH][ceil(T / kDeltaKeep)][dk][dv] fp32) and O may be null.
struct DeltaStep {
    const void* q; const void* k; const void* v; const float* log_g; const void* beta;
    const float* S0; void* O; float* ST; float* keep;
    int B, H, Hk, T, dk, dv;
    float scale;
    gla_dtype dtype;
    int sms;
};
cudaError_t launch_delta_step(const DeltaStep& a, cudaStream_t s);

// The recurrent backward (gla_delta_bwd_step.cu). keep: the states that launch_delta_step
// left. part: per dv tile of kDeltaBwdTile columns, the partial dq, dk ([tiles][BH][T][dk]
// each) and dlog_g, dbeta ([tiles][BH][T] each), fp32; scratch: kDeltaKeep states per tile
// and head. The results go through launch_delta_bwd_sum.
constexpr int kDeltaBwdTile = 64;
struct DeltaBwdStep {
    const void* q; const void* k; const void* v; const float* log_g; const void* beta;
    const float* keep; const void* dO; const float* dST;
    void* dv_out; float* dS0;
    float* part_q; float* part_k; float* part_g; float* part_b; float* scratch;
    int B, H, Hk, T, dk, dv;
    float scale;
    gla_dtype dtype;
};
cudaError_t launch_delta_bwd_step(const DeltaBwdStep& a, cudaStream_t s);
// Sums partials over the dv tiles (and, for rows of q and k, over the H / Hk heads that share
// one) in a fixed order and rounds to the outputs' types. Null outputs are skipped.
struct DeltaBwdSum {
    const float* part_q; const float* part_k; const float* part_g; const float* part_b;
    void* dq; void* dk_out; float* dlog_g; void* dbeta;
    int tiles, B, H, Hk, T, dk;
    gla_dtype dtype;
    int sms;
};
cudaError_t launch_delta_bwd_sum(const DeltaBwdSum& a, cudaStream_t s);

// The chunk form (bf16, dk in {64, 128}, dv a multiple of 64), 64-token chunks on tcgen05.
// The backward's prep (gla_delta_prep.cu), chunk by chunk in parallel: with G the running sum of log_g in the
// chunk, A[i][j] = beta_i (k_i . k_j) exp(G_i - G_j) for j < i, it writes
//   t [BH][nch][2][64][64] bf16      : (I + A)^-1 diag(beta) in two parts (17 bits),
//   p, the same                      : scale (q_i . k_j) exp(G_i - G_j) for j <= i, else 0,
//   gates [BH][nch][8][64] fp32      : beta, exp(G), exp(G_end - G), -exp(G), exp(G - G_mid),
//                                      exp(G_mid - G) (both 0 where too steep) and G in two floats.
struct DeltaPrep {
    const void* q; const void* k; const float* log_g; const void* beta;
    void* t; void* p; float* gates;
    int B, H, Hk, T, dk, nch;
    float scale;
    float beta_floor;   // > 0: smaller |beta| are taken as this (the backward divides by it)
};
cudaError_t launch_delta_prep(const DeltaPrep& a, int* status, cudaStream_t s);

// The forward pass of the chunk form (gla_delta_fused.cu): one kernel, or with nseg > 1 segments of cps
// chunks three: every segment's state from zero and its dk x dk transition (pair: [BH][nseg - 1] of
// [dk][dv] and [dk][dk]), the states entering the segments (seg_in [BH][nseg][dk][dv]), and the pass.
struct DeltaChunks {
    const void* q; const void* k; const void* v; const float* log_g; const void* beta;
    const float* S0; void* O; float* ST; float* pair; float* seg_in;
    int B, H, Hk, T, dk, dv, nch, cps, nseg, per;   // per: segments that one CTA of the first walk takes
    float scale;
};
cudaError_t launch_delta_chunks(const DeltaChunks& a, int* status, cudaStream_t s);

// The backward's serial passes (gla_delta_bwd_chain.cu). Forward sweep: from S0, the state
// entering every chunk and the chunk's U to the workspace. Reverse sweep: from dST, the
// gradient of the state leaving every chunk, the gradient of V (rounded to bf16: the output)
// and what that rounding left, and dS0. All in two bf16 parts; x_hi of the reverse sweep is the
// caller's grad_v.
//   s_hi, s_lo [BH][nch][dv][dk];  u_hi, u_lo [BH][nch][dv][64];  x_hi, x_lo [BH][T][dv]
struct DeltaSweep {
    const void* q; const void* k; const void* v;      // v: V, or dO in reverse
    const void* t; const void* p; const float* gates;
    const float* S_in; float* S_out;
    void* s_hi; void* s_lo; void* u_hi; void* u_lo; void* x_hi; void* x_lo;
    int B, H, Hk, T, dk, dv, nch;
    float scale;
    bool reverse;
};
cudaError_t launch_delta_sweep(const DeltaSweep& a, int* status, cudaStream_t s);

// Chunk-parallel gradients (gla_delta_grads.cu) from the sweeps' results. dq, dk_out: bf16
// [BH][T][dk] when part_q is null (H == Hk), else fp32 partials per head to part_q, part_k.
struct DeltaGrads {
    const void* q; const void* k; const void* dO;
    const void* s_hi; const void* s_lo; const void* u_hi; const void* u_lo;
    const void* d_hi; const void* d_lo; const void* x_hi; const void* x_lo;
    const float* log_g; const float* gates;
    void* dq; void* dk_out; float* part_q; float* part_k; float* dlog_g; void* dbeta;
    int B, H, Hk, T, dk, dv, nch, sms;
    float scale;
};
cudaError_t launch_delta_grads(const DeltaGrads& a, int* status, cudaStream_t s);

}  // namespace gla
