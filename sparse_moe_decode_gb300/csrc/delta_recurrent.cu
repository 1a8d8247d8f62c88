// delta_recurrent.cu -- the gated delta rule token by token: decode, draft
// verification, and sequences too short for the chunked form (100 of one token
// 83 us, against 308 there).
//
// Per token and value head, with S [dv][dk] (row r holds value r's memory):
//   a = e^g,  u = beta (v - a S k),  S <- a S + u k^T,  o = scale S q
//     = scale (a S_old q + u (k . q)).
// Both products with the old state are formed together, so each token costs
// one pass over the registers that hold the state and one reduction.
//
// Bound by memory where there are many sequences: each state is read and
// written once, 256 sequences of one token (32 heads of 128 x 128, 1.08 GB) in
// 154.5 us, 7.0 TB/s, 32 in 22.6 us.  One token of one sequence is latency:
// 2.1 us in a graph, and 0.43 us for each further token (a token's products,
// two shuffle reductions and the update follow one another).
#include <cuda_runtime.h>

#include "common.cuh"
#include "delta_seq.cuh"
#include "early.cuh"
#include "kernels.h"
#include "mixer.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Sums N values over the 32 lanes at once: each round halves the values a
// lane still carries (N + N/2 + ... shuffles in place of 5 N).  The total of
// value i ends in every lane l with l / (32 / N) == i.
template <int N>
__device__ __forceinline__ float reduce_spread(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      const float keep = up ? v[i + n] : v[i];
      v[i] = keep + __shfl_xor_sync(kFull, send, o);
    }
  }
  float r = v[0];
  for (; o >= 1; o >>= 1) r += __shfl_xor_sync(kFull, r, o);
  return r;
}

template <int V>
struct Vec;
template <>
struct Vec<4> {
  using F = float4;
  using H = uint2;
};
template <>
struct Vec<2> {
  using F = float2;
  using H = uint32_t;
};

__device__ __forceinline__ void unpack(uint2 w, float (&o)[4]) {
  o[0] = bf16_lo(w.x), o[1] = bf16_hi(w.x), o[2] = bf16_lo(w.y), o[3] = bf16_hi(w.y);
}
__device__ __forceinline__ void unpack(uint32_t w, float (&o)[2]) {
  o[0] = bf16_lo(w), o[1] = bf16_hi(w);
}
__device__ __forceinline__ void unpack(float4 w, float (&o)[4]) {
  o[0] = w.x, o[1] = w.y, o[2] = w.z, o[3] = w.w;
}
__device__ __forceinline__ void unpack(float2 w, float (&o)[2]) { o[0] = w.x, o[1] = w.y; }
__device__ __forceinline__ float4 pack(const float (&v)[4]) {
  return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ float2 pack(const float (&v)[2]) { return make_float2(v[0], v[1]); }

constexpr int kWarps = 4;

// One warp holds ROWS rows of one head's state, lane l columns V l .. V l +
// V - 1 of each (a row is one coalesced access).
// BLOCKS: blocks of an SM that the registers leave room for.  Three of 16 rows
// (four: 74.6 against 67.8 us for 64 sequences of 4 tokens, 23.3 against 22.4 for
// 32 of one), four of 8 (five: 10.6 against 8.8 us for 4 of 8).
template <int DK, int ROWS, int BLOCKS>
__global__ void __launch_bounds__(32 * kWarps, BLOCKS)
delta_recurrent_kernel(moe_delta_dims d, moe_delta_inputs in, DeltaSeqs seq, int most,
                       const uint32_t *any_bad, moe_bf16 *out, int64_t out_ld) {
  constexpr int V = DK / 32;
  constexpr int kPer = 16 / ROWS;  // lanes of a half warp that share a row's sums
  using VF = typename Vec<V>::F;
  using VH = typename Vec<V>::H;
  const int lane = threadIdx.x & 31, row = (lane & 15) / kPer;
  const uint32_t tiles = d.v_dim / ROWS;
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int tile = static_cast<int>(unit % tiles);
  const int h = static_cast<int>(unit / tiles % d.v_heads);
  const int b = static_cast<int>(unit / tiles / d.v_heads);
  early_begin();
  // a call with a bad bound does nothing
  if (!any_bad && seq.cu_seqlens) {
    bool bad = false;
    for (int i = lane; i < seq.B; i += 32) {
      const int lo = seq.cu_seqlens[i], hi = seq.cu_seqlens[i + 1];
      bad |= lo < 0 || lo > hi || hi > seq.N;
    }
    if (__any_sync(kFull, bad)) {
      if (lane == 0) set_status(seq.status, MOE_DEV_BAD_INDEX);
      return;
    }
  }
  const uint32_t stop = any_bad ? *any_bad : 0;
  const DeltaSeqRange r = delta_seq_range(seq, b);
  if (stop || !r.ok || r.len > most) return;
  const int hk = h / (d.v_heads / d.qk_heads);
  const int64_t at =
      ((static_cast<int64_t>(r.slot) * d.v_heads + h) * d.v_dim + tile * ROWS) * DK + lane * V;
  // A token's values are asked for one token ahead.
  const int64_t row0 = r.start;
  const moe_bf16 *kp = in.k + row0 * in.k_ld + hk * DK + lane * V;
  const moe_bf16 *qp = in.q + row0 * in.q_ld + hk * DK + lane * V;
  const moe_bf16 *vp =
      in.v + row0 * in.v_ld + h * d.v_dim + tile * ROWS + row;
  const float *gp = in.g + row0 * in.g_ld + h, *bp = in.beta + row0 * in.beta_ld + h;
  moe_bf16 *op = out + row0 * out_ld + h * d.v_dim + tile * ROWS + row;
  VH kw{}, qw{};
  uint16_t vw = 0;
  float gw = 0.0f, bw = 0.0f;
  const auto fetch = [&] {
    kw = *reinterpret_cast<const VH *>(kp), qw = *reinterpret_cast<const VH *>(qp);
    vw = *vp, gw = *gp, bw = *bp;
    kp += in.k_ld, qp += in.q_ld, vp += in.v_ld, gp += in.g_ld, bp += in.beta_ld;
  };
  if (r.len > 0) fetch();
  float s[ROWS][V];
  if (seq.state_in) {
    const float *p = seq.state_in + at;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) unpack(*reinterpret_cast<const VF *>(p + i * DK), s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) s[i][j] = 0.0f;
  }
  for (int t = 0; t < r.len; ++t, op += out_ld) {
    float k[V], q[V];
    unpack(kw, k);
    unpack(qw, q);
    const float v = bf16_to_f32(vw), a = expf(delta_log_decay(gw)), beta = bw;
    if (t + 1 < r.len) fetch();
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      kk = fmaf(k[j], k[j], kk);
      qq = fmaf(q[j], q[j], qq);
      kq = fmaf(k[j], q[j], kq);
    }
    kk = warp_sum(kk), qq = warp_sum(qq), kq = warp_sum(kq);
    float kn = 1.0f, qn = d.scale;
    if (d.qk_norm) {
      kn = rsqrtf(kk + d.qk_eps);
      qn = d.scale * rsqrtf(qq + d.qk_eps);
    }
    float part[2 * ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      float sk = 0.0f, sq = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sk = fmaf(s[i][j], k[j], sk);
        sq = fmaf(s[i][j], q[j], sq);
      }
      part[i] = sk;
      part[ROWS + i] = sq;
    }
    // lanes below 16: their row's S k; lane 16 + l: S q of lane l's row
    const float sum = reduce_spread(part, lane);
    const float sq = __shfl_down_sync(kFull, sum, 16);
    const float u = beta * (v - a * kn * sum);  // lanes < 16
    if (lane < 16 && lane % kPer == 0)
      *op = f32_to_bf16(qn * (a * sq + u * kn * kq));
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const float ui = __shfl_sync(kFull, u, i * kPer) * kn;
#pragma unroll
      for (int j = 0; j < V; ++j) s[i][j] = fmaf(a, s[i][j], ui * k[j]);
    }
  }
  if (seq.state_out) {
    float *p = seq.state_out + at;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) *reinterpret_cast<VF *>(p + i * DK) = pack(s[i]);
  }
}

}  // namespace

cudaError_t launch_delta_recurrent(const moe_delta_dims &d, const moe_delta_inputs &in,
                                   const DeltaSeqs &seq, int most, const uint32_t *bad,
                                   moe_bf16 *out, int64_t out_ld, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(seq.B) * d.v_heads * d.v_dim, sms = tc_sm_count();
  // Warps of 8 rows have half as much to do in a token's turn but load k and q
  // and sum their norms twice as often: faster up to 16 warps of 16 rows an SM
  // (4 sequences of 8 tokens 8.8 against 11.0 us, 8 of one 5.2 against 5.7),
  // slower beyond (32 of one 16.4 against 15.3 us, states in L2).
  const bool small = rows <= 16 * 16 * sms;
  // (a head has a multiple of 64 rows)
  const unsigned grid = static_cast<unsigned>(rows / (small ? 8 : 16) / kWarps);
  const bool wide = d.qk_dim == 128;
  const auto kernel =
      small ? (wide ? delta_recurrent_kernel<128, 8, 4> : delta_recurrent_kernel<64, 8, 4>)
            : (wide ? delta_recurrent_kernel<128, 16, 3> : delta_recurrent_kernel<64, 16, 3>);
  return launch_early(kernel, dim3(grid), 32 * kWarps, 0, s, d, in, seq, most, bad, out,
                      out_ld);
}

}  // namespace moe
