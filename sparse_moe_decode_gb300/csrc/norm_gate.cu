// norm_gate.cu -- the norm after a block, its gate, the scaled residual add
// and the norm before the next block, one pass over each row:
//   y = a act(gate) rms(x) g_post + resid,  r = bf16(y),  n = bf16(rms(r) g_pre).
// Bound by memory: x, resid and an element gate are read once and r and n
// written once; a row's values stay in registers between the two norms.
// Measured: 16384 rows of 2048 with an element gate (336 MB) 56.2 us, 6.0 TB/s;
// rows of 8 to 128 of the same bytes 54 to 55 us; 65536 rows of 128 (one per
// head, gated by silu(z), 50 MB) 11.6 us; a call of one row 6.4 us of the host's
// time.  Widths or strides that are no multiple of 8 go by groups of two values
// or one: 336 MB take 126 us at width 2046, 290 us at 2047, 226 to 253 us at 15 to
// 1023.
#include <cuda_runtime.h>

#include "common.cuh"
#include "early.cuh"
#include "kernels.h"
#include "mixer.h"
#include "pair.cuh"

namespace moe {
namespace {

// VEC consecutive bf16, held in VALUES as pairs of fp32 (VEC = 1: a pair whose
// second value is 0).
template <int VEC>
struct Bits;
template <>
struct Bits<8> {
  using T = uint4;
};
template <>
struct Bits<2> {
  using T = uint32_t;
};
template <>
struct Bits<1> {
  using T = uint16_t;
};

__device__ __forceinline__ void unpack(uint4 w, float2 (&v)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
}
__device__ __forceinline__ void unpack(uint32_t w, float2 (&v)[1]) {
  v[0] = make_float2(bf16_lo(w), bf16_hi(w));
}
__device__ __forceinline__ void unpack(uint16_t w, float2 (&v)[1]) {
  v[0] = make_float2(bf16_to_f32(w), 0.0f);
}

__device__ __forceinline__ uint4 pack(const float2 (&v)[4]) {
  return make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y),
                    pack_bf16(v[2].x, v[2].y), pack_bf16(v[3].x, v[3].y));
}
__device__ __forceinline__ void pack(const float2 (&v)[1], uint32_t &w) {
  w = pack_bf16(v[0].x, v[0].y);
}
__device__ __forceinline__ void pack(const float2 (&v)[1], uint16_t &w) {
  w = static_cast<uint16_t>(pack_bf16(v[0].x, 0.0f));
}
__device__ __forceinline__ void pack(const float2 (&v)[4], uint4 &w) { w = pack(v); }

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// exp's argument is rounded once: a relative error of the sigmoid of 2^-21 up
// to |z| = 8 and of |z| 2^-24 beyond, far below the one rounding to bf16; 0
// where it is below 2^-126 (z < -87).
__device__ __forceinline__ float sigmoid(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}

// z -> act(z); the kind is looked at once for all values.
template <int N>
__device__ __forceinline__ void activate(float2 (&z)[N], int kind) {
  if (kind == MOE_ACT_SIGMOID) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = make_float2(sigmoid(z[i].x), sigmoid(z[i].y));
  } else if (kind == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      z[i] = mul2(z[i], make_float2(sigmoid(z[i].x), sigmoid(z[i].y)));
  }
}

// Sum over the `lanes` threads of a row: a power of two up to 32 (groups of
// lanes of a warp), or the whole block (CTA).
template <bool CTA>
__device__ __forceinline__ float row_sum(float v, int lanes, float *tmp) {
  if constexpr (!CTA) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
  } else {
    v = warp_sum(v);
    const int lane = threadIdx.x & 31;
    if (lane == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (blockDim.x >> 5) ? tmp[lane] : 0.0f;
    return warp_sum(v);
  }
}

constexpr int kRowThreads = 256;  // of a block whose rows have up to 32 threads each

// Threads of an SM that the rows are spread over: what the registers allow
// (75 a thread with 16-byte groups, 64 in blocks of up to 1024, 32 to 40 with
// narrower groups).  One block more than fit costs a second round: 16384 rows
// of 2048 took 58 us at 768, 72 us at 1024.
template <int VEC, int NV, int MOST>
constexpr int kSmThreads = NV > 1 || (VEC == 8 && MOST > 256) ? 1024 : VEC == 8 ? 768 : 1536;

// `1 << shift` threads of a warp (or, CTA, the whole block) share a row,
// thread l the groups of VEC values l, l + lanes, ... (NV of them at most).
// Blocks stay and take row after row; with one group per thread (NV = 1) the
// next row's values are on their way while a row's sums are formed.
// MOST: threads of a block at most.
template <int VEC, int NV, bool CTA, int MOST>
__global__ void __launch_bounds__(MOST)
norm_gate_kernel(moe_norm_args a, int shift) {
  using W = typename Bits<VEC>::T;
  __shared__ float tmp[2][2][32];
  early_begin();
  const int l = CTA ? threadIdx.x : threadIdx.x & ((1 << shift) - 1);
  const int lanes = CTA ? blockDim.x : 1 << shift;
  const uint32_t per = CTA ? 1 : kRowThreads >> shift;  // rows of a block at a time
  const int step = lanes * VEC;
  const int n = a.width - l * VEC;  // values from this thread's first on
  const bool element = a.gate_kind == MOE_GATE_ELEMENT;

  constexpr int kP = (VEC + 1) / 2;  // pairs of a group
  struct Row {
    uint32_t outer, in_row;
    W x[NV], z[NV], r[NV];
    float factor;
  };
  // where a tensor's row lies (strides are below 2^32)
  const auto at = [&](const Row &w, int64_t ld) {
    return static_cast<uint64_t>(w.outer) * static_cast<uint32_t>(ld) + w.in_row;
  };
  const auto fetch = [&](Row &w, uint32_t r, bool live) {
    uint32_t outer = live ? r : 0, head = 0;
    if (a.inner > 1) {
      const uint32_t whole = outer / static_cast<uint32_t>(a.inner);
      head = outer - whole * a.inner, outer = whole;
    }
    w.outer = outer;
    w.in_row = head * static_cast<uint32_t>(a.width) + l * VEC;
    w.factor = a.res_scale;
    if (a.gate_kind == MOE_GATE_ROW && live) {
      float2 z[1] = {make_float2(bf16_to_f32(a.gate[outer * a.gate_ld + head]), 0.0f)};
      activate(z, a.gate_act);
      w.factor *= z[0].x;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * step;
      w.x[i] = w.z[i] = w.r[i] = W{};
      if (live && c < n) {  // a row's threads leave its work together
        w.x[i] = *reinterpret_cast<const W *>(a.x + at(w, a.x_ld) + c);
        if (element) w.z[i] = *reinterpret_cast<const W *>(a.gate + at(w, a.gate_ld) + c);
        if (a.resid_in) w.r[i] = *reinterpret_cast<const W *>(a.resid_in + at(w, a.resid_in_ld) + c);
      }
    }
  };
  // a channel's factors: the same for every row
  const auto channel = [&](const moe_bf16 *p, int i) {
    W w{};
    if (p && i * step < n) w = *reinterpret_cast<const W *>(p + l * VEC + i * step);
    return w;
  };
  const bool by_channel = a.gate_kind == MOE_GATE_CHANNEL;
  W post[NV], pre[NV], gate[NV];
  constexpr bool kKeep = NV == 1;
  if constexpr (kKeep) {
    post[0] = channel(a.gamma_post, 0), pre[0] = channel(a.gamma_pre, 0);
    gate[0] = channel(by_channel ? a.gate : nullptr, 0);
  }
  const float mean = 1.0f / static_cast<float>(a.width);

  const uint32_t rows = static_cast<uint32_t>(a.rows), stride = gridDim.x * per;
  // whole blocks go on together (the sums are formed by all their threads)
  uint32_t first = blockIdx.x * per;
  const uint32_t mine = CTA ? 0 : threadIdx.x >> shift;
  Row row;
  if (kKeep) fetch(row, first + mine, first + mine < rows);
  for (int turn = 0; first < rows; turn ^= 1) {
    if (!kKeep) fetch(row, first + mine, first + mine < rows);
    const Row cur = row;
    const int left = first + mine < rows ? n : 0;
    // (row counts and strides stay below 2^31, so this sum does not wrap)
    first += stride;
    if (kKeep && first < rows) fetch(row, first + mine, first + mine < rows);
    float2 y[NV][kP], ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack(cur.x[i], y[i]);
#pragma unroll
      for (int j = 0; j < kP; ++j) ss = fma2(y[i][j], y[i][j], ss);
    }
    float inv = 1.0f;
    if (a.gamma_post) inv = rsqrtf(fmaf(row_sum<CTA>(ss.x + ss.y, lanes, tmp[turn][0]), mean, a.eps));
    ss = both(0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * step;
      if (c < left) {
        float2 w[kP];
        if (a.gamma_post) {
          if constexpr (!kKeep) post[i] = channel(a.gamma_post, i);
          unpack(post[i], w);
#pragma unroll
          for (int j = 0; j < kP; ++j) y[i][j] = mul2(y[i][j], mul2(w[j], both(inv)));
        }
        if (element || by_channel) {
          if constexpr (!kKeep) gate[i] = channel(by_channel ? a.gate : nullptr, i);
          unpack(element ? cur.z[i] : gate[i], w);
          activate(w, a.gate_act);
#pragma unroll
          for (int j = 0; j < kP; ++j) y[i][j] = mul2(y[i][j], w[j]);
        }
        if (a.resid_in) {
          unpack(cur.r[i], w);
#pragma unroll
          for (int j = 0; j < kP; ++j) y[i][j] = fma2(both(cur.factor), y[i][j], w[j]);
        } else {
#pragma unroll
          for (int j = 0; j < kP; ++j) y[i][j] = mul2(both(cur.factor), y[i][j]);
        }
        // one rounding to bf16; the next norm reads the rounded residual
        W out;
        pack(y[i], out);
        if (a.resid_out) *reinterpret_cast<W *>(a.resid_out + at(cur, a.resid_out_ld) + c) = out;
        unpack(out, y[i]);
#pragma unroll
        for (int j = 0; j < kP; ++j) ss = fma2(y[i][j], y[i][j], ss);
      }
    }
    if (a.x_next) {
      inv = rsqrtf(fmaf(row_sum<CTA>(ss.x + ss.y, lanes, tmp[turn][1]), mean, a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * step;
        if (c < left) {
          float2 w[kP];
          if constexpr (!kKeep) pre[i] = channel(a.gamma_pre, i);
          unpack(pre[i], w);
#pragma unroll
          for (int j = 0; j < kP; ++j) w[j] = mul2(y[i][j], mul2(w[j], both(inv)));
          W out;
          pack(w, out);
          *reinterpret_cast<W *>(a.x_next + at(cur, a.x_next_ld) + c) = out;
        }
      }
    }
  }
}

template <int VEC, int NV, bool CTA, int MOST>
cudaError_t launch(const moe_norm_args &a, int threads, int shift, cudaStream_t s) {
  const int64_t per = CTA ? 1 : threads >> shift;  // rows of a block at a time
  const int64_t most = static_cast<int64_t>(tc_sm_count()) * (kSmThreads<VEC, NV, MOST> / threads);
  const int64_t blocks = (a.rows + per - 1) / per;
  return launch_early(norm_gate_kernel<VEC, NV, CTA, MOST>,
                      dim3(static_cast<unsigned>(blocks < most ? blocks : most)), threads, 0, s, a,
                      shift);
}

// Up to 32 groups of VEC values: part of a warp per row; more: a block per
// row, one group per thread while the block can be that wide.
template <int VEC>
cudaError_t route(const moe_norm_args &a, cudaStream_t s) {
  const int groups = (a.width + VEC - 1) / VEC;
  if (groups <= 32) {
    int shift = 0;
    while ((1 << shift) < groups) ++shift;
    return launch<VEC, 1, false, kRowThreads>(a, kRowThreads, shift, s);
  }
  if (groups <= 256) return launch<VEC, 1, true, 256>(a, (groups + 31) / 32 * 32, 0, s);
  if (groups <= 1024) return launch<VEC, 1, true, 1024>(a, (groups + 31) / 32 * 32, 0, s);
  if (groups <= 2048) return launch<VEC, 2, true, 1024>(a, ((groups + 1) / 2 + 31) / 32 * 32, 0, s);
  if constexpr (VEC <= 2)
    if (groups <= 8192) return launch<VEC, 8, true, 1024>(a, 1024, 0, s);
  if constexpr (VEC == 1) return launch<VEC, 16, true, 1024>(a, 1024, 0, s);
  return cudaErrorInvalidValue;  // not reached: width <= 16384
}

}  // namespace

cudaError_t launch_norm_gate_residual(const moe_norm_args &args, int vec, cudaStream_t s) {
  moe_norm_args a = args;
  // heads of whole rows one after another are plain rows
  const int64_t w = int64_t(a.inner) * a.width;
  if (a.inner > 1 && a.x_ld == w && (!a.resid_in || a.resid_in_ld == w) &&
      (!a.resid_out || a.resid_out_ld == w) && (!a.x_next || a.x_next_ld == w) &&
      (a.gate_kind != MOE_GATE_ELEMENT || a.gate_ld == w) &&
      (a.gate_kind != MOE_GATE_ROW || a.gate_ld == a.inner)) {
    a.inner = 1;
    a.x_ld = a.resid_in_ld = a.resid_out_ld = a.x_next_ld = a.width;
    a.gate_ld = a.gate_kind == MOE_GATE_ROW ? 1 : a.width;
  }
  return vec == 8 ? route<8>(a, s) : vec == 2 ? route<2>(a, s) : route<1>(a, s);
}

}  // namespace moe
