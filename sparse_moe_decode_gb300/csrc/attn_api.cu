// attn_api.cu -- the extern "C" entry points of paged attention, its cache and
// the verification of drafts: argument checks and launches on the caller's
// stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_checks.h"
#include "attn.h"
#include "moe_gb300.h"

namespace moe {
namespace {

constexpr int kMaxTokens = 1 << 20, kMaxSeqs = 65536, kMaxHeads = 1024;
constexpr int64_t kMaxRows = int64_t(1) << 31;       // of a cache (coordinates of a copy)
constexpr int kMaxDraft = 1024, kMaxVocab = 1 << 24;

moe_status check_dims(const moe_attn_dims *d) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads > kMaxHeads || d->q_heads % d->kv_heads ||
      d->q_heads / d->kv_heads > kAttnMaxGroup)
    return MOE_ERR_UNSUPPORTED;
  if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return MOE_ERR_UNSUPPORTED;
  if (d->page_size < 16 || d->page_size > 256 || (d->page_size & (d->page_size - 1)))
    return MOE_ERR_UNSUPPORTED;
  if (d->kv_type < MOE_KV_BF16 || d->kv_type > MOE_KV_E4M3) return MOE_ERR_UNSUPPORTED;
  if (d->window < 0 || !isfinite(attn_scale_log2(*d))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// What every call on a cache checks: `spans` receives the cache's four buffers.
moe_status check_call(const moe_attn_dims *d, const moe_kv_cache *c, const moe_kv_batch *b,
                      Span (&spans)[4]) {
  const moe_status st = check_dims(d);
  if (st != MOE_OK) return st;
  if (!c || !b || b->N < 0 || b->B < 0) return MOE_ERR_INVALID_ARG;
  if (b->N > kMaxTokens || b->B > kMaxSeqs) return MOE_ERR_UNSUPPORTED;
  if (!opt_ok(b->cu_seqlens, 4) || !opt_ok(b->seq_lens, 4) || !opt_ok(b->page_table, 4))
    return MOE_ERR_INVALID_ARG;
  if (b->N > 0 && b->B < 1) return MOE_ERR_INVALID_ARG;  // rows of whom?
  if (!b->cu_seqlens && b->B > 0 && b->N % b->B) return MOE_ERR_INVALID_ARG;
  if (b->table_cols < 0 || b->table_ld < b->table_cols || b->table_ld > kMaxStride)
    return MOE_ERR_INVALID_ARG;
  if (int64_t(b->table_cols) * d->page_size > kMaxPositions) return MOE_ERR_UNSUPPORTED;
  if (c->pages < 1) return MOE_ERR_INVALID_ARG;
  const int64_t per_page = int64_t(d->kv_heads) * d->page_size;
  if (c->pages >= kMaxRows / per_page) return MOE_ERR_UNSUPPORTED;
  const bool codes = d->kv_type != MOE_KV_BF16;
  if (!ptr_ok(c->k) || !ptr_ok(c->v)) return MOE_ERR_INVALID_ARG;
  if (codes ? !ptr_ok(c->k_scale) || !ptr_ok(c->v_scale) : c->k_scale || c->v_scale)
    return MOE_ERR_INVALID_ARG;
  if (b->N > 0 && (!b->seq_lens || (!b->page_table && b->table_cols > 0)))
    return MOE_ERR_INVALID_ARG;
  const int64_t rows = c->pages * per_page, all = rows * d->head_dim;
  const int size = codes ? 1 : 2;
  spans[0] = Span{c->k, 1, all, all, size};
  spans[1] = Span{c->v, 1, all, all, size};
  spans[2] = Span{c->k_scale, 1, rows, rows, 4};
  spans[3] = Span{c->v_scale, 1, rows, rows, 4};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(spans[i], spans[j])) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool rows_ok(const moe_bf16 *p, int64_t ld, int64_t width) {
  return ptr_ok(p) && stride_ok(ld, width, 8);
}

bool apart(const Span &x, const Span (&spans)[4]) {
  for (const Span &s : spans)
    if (overlap(x, s)) return false;
  return true;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_attn_workspace_bytes(const moe_attn_dims *dims) {
  return check_dims(dims) == MOE_OK ? attn_workspace(*dims) : 0;
}

moe_status moe_kv_write(const moe_attn_dims *dims, const moe_kv_cache *cache,
                        const moe_kv_batch *batch, const moe_bf16 *k, int64_t k_ld,
                        const moe_bf16 *v, int64_t v_ld, void *workspace, size_t ws_bytes,
                        void *stream) {
  Span spans[4];
  moe_status st = check_call(dims, cache, batch, spans);
  if (st != MOE_OK) return st;
  const int64_t w = int64_t(dims->kv_heads) * dims->head_dim;
  if (batch->N > 0 && (!rows_ok(k, k_ld, w) || !rows_ok(v, v_ld, w) ||
                       !apart(Span{k, batch->N, w, k_ld, 2}, spans) ||
                       !apart(Span{v, batch->N, w, v_ld, 2}, spans)))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, 256)) != MOE_OK) return st;
  if (batch->N == 0) return MOE_OK;
  return cuda_status(launch_kv_write(*dims, *cache, attn_batch(*dims, *cache, *batch, workspace), k,
                                     k_ld, v, v_ld, static_cast<cudaStream_t>(stream)));
}

moe_status moe_kv_read(const moe_attn_dims *dims, const moe_kv_cache *cache,
                       const moe_kv_batch *batch, moe_bf16 *k, int64_t k_ld, moe_bf16 *v,
                       int64_t v_ld, void *workspace, size_t ws_bytes, void *stream) {
  Span spans[4];
  moe_status st = check_call(dims, cache, batch, spans);
  if (st != MOE_OK) return st;
  const int64_t w = int64_t(dims->kv_heads) * dims->head_dim;
  const Span ks{k, batch->N, w, k_ld, 2}, vs{v, batch->N, w, v_ld, 2};
  if (batch->N > 0 && ((k && !rows_ok(k, k_ld, w)) || (v && !rows_ok(v, v_ld, w)) ||
                       !apart(ks, spans) || !apart(vs, spans) || overlap(ks, vs)))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, 256)) != MOE_OK) return st;
  if (batch->N == 0 || (!k && !v)) return MOE_OK;
  return cuda_status(launch_kv_read(*dims, *cache, attn_batch(*dims, *cache, *batch, workspace), k,
                                    k_ld, v, v_ld, static_cast<cudaStream_t>(stream)));
}

moe_status moe_paged_attention(const moe_attn_dims *dims, const moe_kv_cache *cache,
                               const moe_kv_batch *batch, const moe_bf16 *q, int64_t q_ld,
                               moe_bf16 *out, int64_t out_ld, void *workspace, size_t ws_bytes,
                               void *stream) {
  Span spans[4];
  moe_status st = check_call(dims, cache, batch, spans);
  if (st != MOE_OK) return st;
  const int64_t w = int64_t(dims->q_heads) * dims->head_dim;
  const Span qs{q, batch->N, w, q_ld, 2}, os{out, batch->N, w, out_ld, 2};
  if (batch->N > 0 && (!rows_ok(q, q_ld, w) || !rows_ok(out, out_ld, w) || overlap(qs, os) ||
                       !apart(os, spans)))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(workspace, ws_bytes, attn_workspace(*dims))) != MOE_OK) return st;
  if (batch->N == 0) return MOE_OK;
  return cuda_status(launch_attention(*dims, *cache, attn_batch(*dims, *cache, *batch, workspace),
                                      q, q_ld, out, out_ld, workspace,
                                      static_cast<cudaStream_t>(stream)));
}

moe_status moe_verify_draft(int B, int T, int V, const float *target, int64_t target_seq_ld,
                            int64_t target_ld, const float *draft, int64_t draft_seq_ld,
                            int64_t draft_ld, const int32_t *draft_tokens, const float *uniform,
                            int32_t *tokens, int32_t *accepted, void *workspace, size_t ws_bytes,
                            void *stream) {
  if (B < 0 || T < 0 || V < 1) return MOE_ERR_INVALID_ARG;
  if (B > kMaxSeqs || T > kMaxDraft || V > kMaxVocab) return MOE_ERR_UNSUPPORTED;
  if (B > 0) {
    if (!ptr_ok(target, 4) || !opt_ok(draft, 4) || !opt_ok(draft_tokens, 4) ||
        (T > 0 && !draft_tokens) || !ptr_ok(uniform, 4) || !ptr_ok(tokens, 4) ||
        !ptr_ok(accepted, 4))
      return MOE_ERR_INVALID_ARG;
    // (rows may be shared: a stride of 0)
    const auto ld_ok = [](int64_t ld) { return ld >= 0 && ld <= (int64_t(1) << 40); };
    if (!ld_ok(target_seq_ld) || !ld_ok(target_ld) ||
        (draft && (!ld_ok(draft_seq_ld) || !ld_ok(draft_ld))))
      return MOE_ERR_INVALID_ARG;
    const Span outs[2] = {Span{tokens, 1, int64_t(B) * (T + 1), int64_t(B) * (T + 1), 4},
                          Span{accepted, 1, B, B, 4}};
    const int64_t p = (B - 1) * target_seq_ld + T * target_ld + V;
    const int64_t q = T > 0 ? (B - 1) * draft_seq_ld + (T - 1) * draft_ld + V : 0;
    const Span ins[4] = {Span{target, 1, p, p, 4}, Span{T > 0 ? draft : nullptr, 1, q, q, 4},
                         Span{draft_tokens, 1, int64_t(B) * T, int64_t(B) * T, 4},
                         Span{uniform, 1, int64_t(B) * (T + 1), int64_t(B) * (T + 1), 4}};
    if (overlap(outs[0], outs[1])) return MOE_ERR_INVALID_ARG;
    for (const Span &o : outs)
      for (const Span &i : ins)
        if (overlap(o, i)) return MOE_ERR_INVALID_ARG;
  }
  const moe_status st = check_ws(workspace, ws_bytes, 256);
  if (st != MOE_OK) return st;
  if (B == 0) return MOE_OK;
  const DraftArgs a{B, T, V, target, target_seq_ld, target_ld, draft, draft_seq_ld, draft_ld,
                    draft_tokens, uniform, tokens, accepted, static_cast<uint32_t *>(workspace)};
  return cuda_status(launch_verify_draft(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
