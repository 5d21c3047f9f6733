// Internal declarations of the gated delta rule: the planner in gla_delta_api.cu and the
// kernel launchers. Not part of the public ABI (include/gla.h is).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "gla_internal.h"

namespace gla {

constexpr int kDeltaMaxDk = 256;    // widest keys of the recurrent form (its state rows per thread)
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

}  // namespace gla
