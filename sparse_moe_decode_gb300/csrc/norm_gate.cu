// norm_gate.cu -- the norm after a block, its gate, the scaled residual add
// and the norm before the next block, one pass over each row:
//   y = a act(gate) rms(x) g_post + resid,  r = bf16(y),  n = bf16(rms(r) g_pre).
// Bound by memory: x, resid and an element gate are read once and r and n
// written once; a row's values stay in registers between the two norms.
#include <cuda_runtime.h>

#include "common.cuh"
#include "mixer.h"

namespace moe {
namespace {

// exp's argument is rounded once: a relative error of the sigmoid of 2^-21 up
// to |z| = 8 and of |z| 2^-24 beyond, far below the one rounding to bf16.
__device__ __forceinline__ float act(float z, int kind) {
  if (kind == MOE_ACT_IDENTITY) return z;
  const float s = __fdividef(1.0f, 1.0f + __expf(-z));
  return kind == MOE_ACT_SILU ? z * s : s;
}

// VEC consecutive bf16.
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

__device__ __forceinline__ void unpack(uint4 w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
}
__device__ __forceinline__ void unpack(uint32_t w, float (&v)[2]) {
  v[0] = bf16_lo(w), v[1] = bf16_hi(w);
}
__device__ __forceinline__ void unpack(uint16_t w, float (&v)[1]) { v[0] = bf16_to_f32(w); }

__device__ __forceinline__ uint32_t pair(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
  return make_uint4(pair(v[0], v[1]), pair(v[2], v[3]), pair(v[4], v[5]), pair(v[6], v[7]));
}
__device__ __forceinline__ uint32_t pack(const float (&v)[2]) { return pair(v[0], v[1]); }
__device__ __forceinline__ uint16_t pack(const float (&v)[1]) {
  return static_cast<uint16_t>(pair(v[0], 0.0f));
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

// `1 << shift` threads of a warp (or, CTA, the whole block) share a row,
// thread l the groups of VEC values l, l + lanes, ... (NV of them at most).
// Everything a thread reads is asked for before the first sum needs it.
template <int VEC, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : kRowThreads)
norm_gate_kernel(moe_norm_args a, int shift) {
  using W = typename Bits<VEC>::T;
  __shared__ float tmp[2][32];
  const uint32_t r = CTA ? blockIdx.x : (blockIdx.x * (kRowThreads >> shift)) + (threadIdx.x >> shift);
  const int l = CTA ? threadIdx.x : threadIdx.x & ((1 << shift) - 1);
  const int lanes = CTA ? blockDim.x : 1 << shift;
  const bool live = r < a.rows;  // a row's threads leave its work together
  uint32_t outer = 0, head = 0;
  if (live) {
    outer = r;
    if (a.inner > 1) outer = r / static_cast<uint32_t>(a.inner), head = r - outer * a.inner;
  }
  const int64_t in_row = static_cast<int64_t>(head) * a.width + l * VEC;
  const int n = live ? a.width - l * VEC : 0;  // values from this thread's first on
  const int step = lanes * VEC;
  const moe_bf16 *x = a.x + outer * a.x_ld + in_row;
  const bool element = a.gate_kind == MOE_GATE_ELEMENT;
  const moe_bf16 *gate = nullptr;
  if (element) gate = a.gate + outer * a.gate_ld + in_row;
  if (a.gate_kind == MOE_GATE_CHANNEL) gate = a.gate + l * VEC;
  const moe_bf16 *resid = a.resid_in ? a.resid_in + outer * a.resid_in_ld + in_row : nullptr;
  W xw[NV], zw[NV] = {}, rw[NV] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * step;
    if (c < n) {
      xw[i] = *reinterpret_cast<const W *>(x + c);
      if (gate) zw[i] = *reinterpret_cast<const W *>(gate + c);
      if (resid) rw[i] = *reinterpret_cast<const W *>(resid + c);
    }
  }
  float factor = a.res_scale;
  if (a.gate_kind == MOE_GATE_ROW && live)
    factor *= act(bf16_to_f32(a.gate[outer * a.gate_ld + head]), a.gate_act);
  float y[NV][VEC];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i * step < n) {
      unpack(xw[i], y[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
    }
  }
  float inv = 1.0f;
  if (a.gamma_post) inv = 1.0f / sqrtf(row_sum<CTA>(ss, lanes, tmp[0]) / a.width + a.eps);
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * step;
    if (c < n) {
      float w[VEC];
      if (a.gamma_post) {
        unpack(*reinterpret_cast<const W *>(a.gamma_post + l * VEC + c), w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[i][j] *= inv * w[j];
      }
      if (gate) {
        unpack(zw[i], w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[i][j] *= act(w[j], a.gate_act);
      }
      unpack(rw[i], w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[i][j] = resid ? fmaf(factor, y[i][j], w[j]) : factor * y[i][j];
      // one rounding to bf16; the next norm reads the rounded residual
      const W out = pack(y[i]);
      if (a.resid_out) *reinterpret_cast<W *>(a.resid_out + outer * a.resid_out_ld + in_row + c) = out;
      unpack(out, y[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
    }
  }
  if (a.x_next) {
    inv = 1.0f / sqrtf(row_sum<CTA>(ss, lanes, tmp[1]) / a.width + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * step;
      if (c < n) {
        float w[VEC];
        unpack(*reinterpret_cast<const W *>(a.gamma_pre + l * VEC + c), w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = y[i][j] * inv * w[j];
        *reinterpret_cast<W *>(a.x_next + outer * a.x_next_ld + in_row + c) = pack(w);
      }
    }
  }
}

template <int VEC, int NV, bool CTA>
cudaError_t launch(const moe_norm_args &a, int threads, int shift, cudaStream_t s) {
  const int64_t per = CTA ? 1 : threads >> shift;  // rows of a block
  norm_gate_kernel<VEC, NV, CTA>
      <<<static_cast<unsigned>((a.rows + per - 1) / per), threads, 0, s>>>(a, shift);
  return cudaGetLastError();
}

// Up to 32 groups of VEC values: part of a warp per row; more: a block per
// row, one group per thread while the block can be that wide.
template <int VEC>
cudaError_t route(const moe_norm_args &a, cudaStream_t s) {
  const int groups = (a.width + VEC - 1) / VEC;
  if (groups <= 32) {
    int shift = 0;
    while ((1 << shift) < groups) ++shift;
    return launch<VEC, 1, false>(a, kRowThreads, shift, s);
  }
  if (groups <= 1024) return launch<VEC, 1, true>(a, (groups + 31) / 32 * 32, 0, s);
  if (groups <= 2048) return launch<VEC, 2, true>(a, ((groups + 1) / 2 + 31) / 32 * 32, 0, s);
  if constexpr (VEC <= 2)
    if (groups <= 8192) return launch<VEC, 8, true>(a, 1024, 0, s);
  if constexpr (VEC == 1) return launch<VEC, 16, true>(a, 1024, 0, s);
  return cudaErrorInvalidValue;  // not reached: width <= 16384
}

}  // namespace

cudaError_t launch_norm_gate_residual(const moe_norm_args &a, int vec, cudaStream_t s) {
  return vec == 8 ? route<8>(a, s) : vec == 2 ? route<2>(a, s) : route<1>(a, s);
}

}  // namespace moe
