// mixer.h -- host-side launchers of the gated delta rule and of the norms
// around a block (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_gb300.h"

namespace moe {

// Which tokens and which state a sequence has: its rows come from cu_seqlens
// (N rows in all) or, without them, are b * T .. b * T + T - 1.
struct DeltaSeqs {
  const int32_t *cu_seqlens;  // [B + 1] or nullptr
  int N, B, T;
  const int32_t *slots;  // [B] or nullptr
  int n_slots;
  const float *state_in;  // nullable
  float *state_out;       // nullable
  uint32_t *status;
};

// Token by token, the state in registers (any length).
cudaError_t launch_delta_recurrent(const moe_delta_dims &d, const moe_delta_inputs &in,
                                   const DeltaSeqs &seq, moe_bf16 *out, int64_t out_ld,
                                   cudaStream_t s);

// In chunks of 64 tokens; ws holds delta_chunk_workspace bytes.
size_t delta_chunk_workspace(const moe_delta_dims &d, int N, int B);
cudaError_t launch_delta_chunk(const moe_delta_dims &d, const moe_delta_inputs &in,
                               const DeltaSeqs &seq, void *ws, moe_bf16 *out, int64_t out_ld,
                               cudaStream_t s);

// a.rows > 0; vec = 8 or 2: width and every stride are multiples of it (the
// rows start on 16- or 4-byte boundaries), otherwise 1.
cudaError_t launch_norm_gate_residual(const moe_norm_args &a, int vec, cudaStream_t s);

}  // namespace moe
