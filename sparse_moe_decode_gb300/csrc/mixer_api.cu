// mixer_api.cu -- the extern "C" entry points of the gated delta rule and of
// the norms around a block: argument checks and launches on the caller's
// stream.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "mixer.h"
#include "moe_gb300.h"

namespace moe {
namespace {

constexpr int kDeltaMaxTokens = 1 << 20;
constexpr int kDeltaMaxSeqs = 65536;
constexpr int kDeltaMaxHeads = 256;
// (each warp of the recurrent kernel looks at all bounds of such a call)
constexpr int kRecurrentSeqs = 64;
constexpr int kNormMaxWidth = 16384;
constexpr int64_t kNormMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxStride = int64_t(1) << 31;  // elements: offsets stay far inside 63 bits

bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool ptr_ok(const void *p, uintptr_t a = 16) { return p != nullptr && aligned(p, a); }
bool opt_ok(const void *p, uintptr_t a = 16) { return p == nullptr || aligned(p, a); }

// Rows of `w` elements of `size` bytes, `ld` elements apart.
struct Span {
  const void *p;
  int64_t rows, w, ld;
  int size;
};

bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + static_cast<uintptr_t>((a.rows - 1) * a.ld + a.w) * a.size;
  const uintptr_t eb = pb + static_cast<uintptr_t>((b.rows - 1) * b.ld + b.w) * b.size;
  if (pa >= eb || pb >= ea) return false;
  // columns of one buffer: equal strides keep them apart in every row
  const uintptr_t ld = static_cast<uintptr_t>(a.ld) * a.size;
  if (ld == 0 || ld != static_cast<uintptr_t>(b.ld) * b.size) return true;
  const uintptr_t d = (pb >= pa) ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;
  return d < static_cast<uintptr_t>(a.w) * a.size ||
         ld - d < static_cast<uintptr_t>(b.w) * b.size;
}

moe_status check_delta_dims(const moe_delta_dims *d) {
  if (!d) return MOE_ERR_INVALID_ARG;
  if (d->qk_heads < 1 || d->v_heads < 1 || d->v_heads % d->qk_heads ||
      d->v_heads > kDeltaMaxHeads)
    return MOE_ERR_UNSUPPORTED;
  if ((d->qk_dim != 64 && d->qk_dim != 128) || (d->v_dim != 64 && d->v_dim != 128))
    return MOE_ERR_UNSUPPORTED;
  if (!isfinite(d->scale)) return MOE_ERR_INVALID_ARG;
  if (d->qk_norm && !(d->qk_eps >= 0.0f && isfinite(d->qk_eps))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool stride_ok(int64_t ld, int64_t least, int64_t multiple) {
  return ld >= least && ld <= kMaxStride && ld % multiple == 0;
}

moe_status check_delta(const moe_delta_dims *d, const moe_delta_inputs *in, int64_t rows,
                       const int32_t *slots, int B, int n_slots, const float *state_in,
                       const float *state_out, const moe_bf16 *out, int64_t out_ld) {
  if (!in || !opt_ok(slots, 4) || n_slots < 0) return MOE_ERR_INVALID_ARG;
  if (!slots && (state_in || state_out) && n_slots < B) return MOE_ERR_INVALID_ARG;
  if (!opt_ok(state_in) || !opt_ok(state_out)) return MOE_ERR_INVALID_ARG;
  const int64_t kw = int64_t(d->qk_heads) * d->qk_dim, vw = int64_t(d->v_heads) * d->v_dim;
  const int64_t state = int64_t(d->v_heads) * d->v_dim * d->qk_dim;
  if (state_in != state_out && overlap(Span{state_in, n_slots, state, state, 4},
                                       Span{state_out, n_slots, state, state, 4}))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!ptr_ok(in->q) || !ptr_ok(in->k) || !ptr_ok(in->v) || !ptr_ok(in->g, 4) ||
      !ptr_ok(in->beta, 4) || !ptr_ok(out))
    return MOE_ERR_INVALID_ARG;
  if (!stride_ok(in->q_ld, kw, 8) || !stride_ok(in->k_ld, kw, 8) || !stride_ok(in->v_ld, vw, 8) ||
      !stride_ok(in->g_ld, d->v_heads, 1) || !stride_ok(in->beta_ld, d->v_heads, 1) ||
      !stride_ok(out_ld, vw, 8))
    return MOE_ERR_INVALID_ARG;
  const Span o{out, rows, vw, out_ld, 2};
  if (overlap(o, Span{in->q, rows, kw, in->q_ld, 2}) || overlap(o, Span{in->k, rows, kw, in->k_ld, 2}) ||
      overlap(o, Span{in->v, rows, vw, in->v_ld, 2}) ||
      overlap(o, Span{in->g, rows, d->v_heads, in->g_ld, 4}) ||
      overlap(o, Span{in->beta, rows, d->v_heads, in->beta_ld, 4}))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ptr_ok(ws, 256)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

DeltaSeqs delta_seqs(const int32_t *cu_seqlens, int N, int B, int T, const int32_t *slots,
                     int n_slots, const float *state_in, float *state_out, void *ws) {
  DeltaSeqs s;
  s.cu_seqlens = cu_seqlens;
  s.N = N, s.B = B, s.T = T;
  s.slots = slots;
  // without slots, sequence b has slot b (checked above where there are states)
  s.n_slots = slots ? n_slots : B;
  s.state_in = state_in, s.state_out = state_out;
  s.status = static_cast<uint32_t *>(ws);
  return s;
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_delta_workspace_bytes(const moe_delta_dims *dims, int N, int B) {
  if (check_delta_dims(dims) != MOE_OK || N < 0 || N > kDeltaMaxTokens || B < 0 ||
      B > kDeltaMaxSeqs)
    return 0;
  return delta_chunk_workspace(*dims, N, B);
}

moe_status moe_delta_chunk(const moe_delta_dims *dims, const moe_delta_inputs *in, int N,
                           const int32_t *cu_seqlens, int B, const int32_t *slots, int n_slots,
                           const float *state_in, float *state_out, moe_bf16 *out,
                           int64_t out_ld, void *workspace, size_t ws_bytes, void *stream) {
  moe_status st = check_delta_dims(dims);
  if (st != MOE_OK) return st;
  if (N < 0 || B < 0 || (!cu_seqlens && B != 1) || !opt_ok(cu_seqlens, 4))
    return MOE_ERR_INVALID_ARG;
  if (N > kDeltaMaxTokens || B > kDeltaMaxSeqs) return MOE_ERR_UNSUPPORTED;
  st = check_delta(dims, in, N, slots, B, n_slots, state_in, state_out, out, out_ld);
  if (st != MOE_OK) return st;
  st = check_ws(workspace, ws_bytes, moe_delta_workspace_bytes(dims, N, B));
  if (st != MOE_OK) return st;
  if (B == 0) return MOE_OK;
  const DeltaSeqs seq = delta_seqs(cu_seqlens, N, B, N, slots, n_slots, state_in, state_out,
                                   workspace);
  // no sequence can be longer: one kernel does
  if (N <= kDeltaShort && B <= kRecurrentSeqs)
    return cuda_status(launch_delta_recurrent(*dims, *in, seq, N, nullptr, out, out_ld,
                                              static_cast<cudaStream_t>(stream)));
  return cuda_status(launch_delta_chunk(*dims, *in, seq, workspace, out, out_ld,
                                        static_cast<cudaStream_t>(stream)));
}

moe_status moe_delta_step(const moe_delta_dims *dims, const moe_delta_inputs *in, int B, int T,
                          const int32_t *slots, int n_slots, const float *state_in,
                          float *state_out, moe_bf16 *out, int64_t out_ld, void *workspace,
                          size_t ws_bytes, void *stream) {
  moe_status st = check_delta_dims(dims);
  if (st != MOE_OK) return st;
  if (B < 0 || T < 0) return MOE_ERR_INVALID_ARG;
  if (B > kDeltaMaxSeqs || int64_t(B) * T > kDeltaMaxTokens) return MOE_ERR_UNSUPPORTED;
  st = check_delta(dims, in, int64_t(B) * T, slots, B, n_slots, state_in, state_out, out, out_ld);
  if (st != MOE_OK) return st;
  if ((st = check_ws(workspace, ws_bytes, 256)) != MOE_OK) return st;
  if (B == 0) return MOE_OK;
  const DeltaSeqs seq = delta_seqs(nullptr, B * T, B, T, slots, n_slots, state_in, state_out,
                                   workspace);
  return cuda_status(launch_delta_recurrent(*dims, *in, seq, T, nullptr, out, out_ld,
                                            static_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_gate_residual(const moe_norm_args *args, void *stream) {
  if (!args) return MOE_ERR_INVALID_ARG;
  const moe_norm_args &a = *args;
  if (a.rows < 0 || a.width < 1 || a.inner < 1) return MOE_ERR_INVALID_ARG;
  if (a.rows > kNormMaxRows || a.width > kNormMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (a.rows % a.inner) return MOE_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f && isfinite(a.eps)) || !isfinite(a.res_scale)) return MOE_ERR_INVALID_ARG;
  if (a.gate_kind < MOE_GATE_NONE || a.gate_kind > MOE_GATE_ROW ||
      a.gate_act < MOE_ACT_IDENTITY || a.gate_act > MOE_ACT_SILU)
    return MOE_ERR_INVALID_ARG;
  if (a.rows == 0) return MOE_OK;
  const int64_t w = int64_t(a.inner) * a.width, groups = a.rows / a.inner;
  const bool element = a.gate_kind == MOE_GATE_ELEMENT, per_row = a.gate_kind == MOE_GATE_ROW;
  if (!ptr_ok(a.x) || !opt_ok(a.gamma_post) || !opt_ok(a.resid_in) || !opt_ok(a.resid_out) ||
      !opt_ok(a.x_next) || !opt_ok(a.gamma_pre) || !opt_ok(a.gate))
    return MOE_ERR_INVALID_ARG;
  if ((!a.resid_out && !a.x_next) || !a.gamma_pre != !a.x_next ||
      !a.gate != (a.gate_kind == MOE_GATE_NONE))
    return MOE_ERR_INVALID_ARG;
  if (!stride_ok(a.x_ld, w, 1) || (a.resid_in && !stride_ok(a.resid_in_ld, w, 1)) ||
      (a.resid_out && !stride_ok(a.resid_out_ld, w, 1)) ||
      (a.x_next && !stride_ok(a.x_next_ld, w, 1)) || (element && !stride_ok(a.gate_ld, w, 1)) ||
      (per_row && !stride_ok(a.gate_ld, a.inner, 1)))
    return MOE_ERR_INVALID_ARG;
  Span gate{a.gate, 1, a.width, a.width, 2};
  if (element) gate = Span{a.gate, groups, w, a.gate_ld, 2};
  if (per_row) gate = Span{a.gate, groups, a.inner, a.gate_ld, 2};
  const Span ins[5] = {Span{a.x, groups, w, a.x_ld, 2},
                       Span{a.resid_in, groups, w, a.resid_in_ld, 2}, gate,
                       Span{a.gamma_post, 1, a.width, a.width, 2},
                       Span{a.gamma_pre, 1, a.width, a.width, 2}};
  const Span outs[2] = {Span{a.resid_out, groups, w, a.resid_out_ld, 2},
                        Span{a.x_next, groups, w, a.x_next_ld, 2}};
  if (overlap(outs[0], outs[1])) return MOE_ERR_INVALID_ARG;
  for (const Span &o : outs)
    for (int i = 0; i < 5; ++i) {
      // x or resid_in itself: each value is read before the thread that
      // reads it writes its place
      const bool in_place = i < 2 && o.p == ins[i].p && o.ld == ins[i].ld;
      if (!in_place && overlap(o, ins[i])) return MOE_ERR_INVALID_ARG;
    }
  // common divisors of everything that places a row
  int64_t by = a.width | a.x_ld;
  if (a.resid_in) by |= a.resid_in_ld;
  if (a.resid_out) by |= a.resid_out_ld;
  if (a.x_next) by |= a.x_next_ld;
  if (element) by |= a.gate_ld;
  const int vec = by % 8 == 0 ? 8 : by % 2 == 0 ? 2 : 1;
  return cuda_status(launch_norm_gate_residual(a, vec, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
