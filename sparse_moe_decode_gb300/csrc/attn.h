// attn.h -- host-side launchers of paged attention, its cache and the
// verification of drafts (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_gb300.h"

namespace moe {

constexpr int64_t kMaxPositions = int64_t(1) << 30;  // of a sequence
constexpr int kAttnMaxGroup = 64;  // query heads of a key/value head
// Blocks of an attention kernel: what the workspace has room for.
constexpr int kStreamMaxCtas = 480;
constexpr int kStreamRows = 16;  // rows (token, head of a group) of a tile
constexpr int kTcMaxCtas = 160;     // one an SM; 256 rows, 128 with a head_dim of 256

// What the kernels multiply the products of q and k by: weights are powers of two.
inline float attn_scale_log2(const moe_attn_dims &d) { return d.scale * 1.44269504088896340736f; }

// A batch as the kernels take it.
struct AttnBatch {
  const int32_t *cu;    // [B + 1] or nullptr: T rows each
  const int32_t *lens;  // [B]
  const int32_t *table;
  int64_t table_ld;
  int32_t cols, N, B, T;
  int32_t group, kv_heads, page_shift, window;
  int32_t pages;
  uint64_t group_inverse;  // of rows below 2^26: row / group = row * this >> 32
  uint32_t *status;
};

inline AttnBatch attn_batch(const moe_attn_dims &d, const moe_kv_cache &c, const moe_kv_batch &b,
                            void *ws) {
  AttnBatch a;
  a.cu = b.cu_seqlens, a.lens = b.seq_lens, a.table = b.page_table;
  a.table_ld = b.table_ld;
  a.cols = b.table_cols, a.N = b.N, a.B = b.B;
  a.T = b.cu_seqlens ? 0 : b.N / b.B;
  a.group = d.q_heads / d.kv_heads, a.kv_heads = d.kv_heads;
  a.page_shift = 0;
  while ((1 << a.page_shift) < d.page_size) ++a.page_shift;
  a.window = d.window < kMaxPositions ? d.window : 0;  // (places plus it stay in 32 bits)
  a.pages = static_cast<int32_t>(c.pages);
  a.group_inverse = (uint64_t(1) << 32) / a.group + 1;
  a.status = static_cast<uint32_t *>(ws);
  return a;
}

cudaError_t launch_kv_write(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                            const moe_bf16 *k, int64_t k_ld, const moe_bf16 *v, int64_t v_ld,
                            cudaStream_t s);
cudaError_t launch_kv_read(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                           moe_bf16 *k, int64_t k_ld, moe_bf16 *v, int64_t v_ld, cudaStream_t s);

size_t attn_workspace(const moe_attn_dims &d);
cudaError_t launch_attention(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                             const moe_bf16 *q, int64_t q_ld, moe_bf16 *out, int64_t out_ld,
                             void *ws, cudaStream_t s);

struct DraftArgs {
  int B, T, V;
  const float *target;
  int64_t target_seq_ld, target_ld;
  const float *draft;
  int64_t draft_seq_ld, draft_ld;
  const int32_t *draft_tokens;
  const float *uniform;
  int32_t *tokens, *accepted;
  uint32_t *status;
};
cudaError_t launch_verify_draft(const DraftArgs &a, cudaStream_t s);

}  // namespace moe
