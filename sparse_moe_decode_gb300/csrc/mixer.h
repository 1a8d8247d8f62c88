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

// A prompt call's sequences of so few tokens run token by token.  One (32 value
// heads of 128) takes 17.0 us in the chunked form whatever its length up to 64
// (8 heads of 64 10.8 us), in a graph, and 1.7 us and 0.43 us for each token in
// the recurrent one (12.0 and 11.0 us at 24); each of many takes 3.1 us in the
// former, 0.6 us and 0.11 us a token in the latter.  With fewer heads both sides
// are nearer to one another: 25 tokens of 1 to 8 heads take 10.3 to 11.8 us in
// chunks and 11.7 to 12.8 us token by token, of 16 heads 14.3 and 12.8 us, of 32
// heads 16.9 and 12.9 us.
constexpr int kDeltaShort = 24;

// Token by token, the state in registers: the sequences of up to `most` tokens.
// `bad`: null, or a word that is not 0 when a bound of the call is bad (without
// it every warp looks at all bounds).
cudaError_t launch_delta_recurrent(const moe_delta_dims &d, const moe_delta_inputs &in,
                                   const DeltaSeqs &seq, int most, const uint32_t *bad,
                                   moe_bf16 *out, int64_t out_ld, cudaStream_t s);

// In chunks of 64 tokens, the sequences of up to kDeltaShort tokens token by
// token after the others; ws holds delta_chunk_workspace bytes.
size_t delta_chunk_workspace(const moe_delta_dims &d, int N, int B);
cudaError_t launch_delta_chunk(const moe_delta_dims &d, const moe_delta_inputs &in,
                               const DeltaSeqs &seq, void *ws, moe_bf16 *out, int64_t out_ld,
                               cudaStream_t s);

// a.rows > 0; vec = 8 or 2: width and every stride are multiples of it (the
// rows start on 16- or 4-byte boundaries), otherwise 1.
cudaError_t launch_norm_gate_residual(const moe_norm_args &a, int vec, cudaStream_t s);

}  // namespace moe
