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

__device__ __forceinline__ float act(float z, int kind) {
  if (kind == MOE_ACT_IDENTITY) return z;
  const float s = 1.0f / (1.0f + expf(-z));
  return kind == MOE_ACT_SILU ? z * s : s;
}

// VEC consecutive bf16 as fp32.
template <int VEC>
__device__ __forceinline__ void load(const moe_bf16 *p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(u[i]), v[2 * i + 1] = bf16_hi(u[i]);
  } else {
    v[0] = bf16_to_f32(*p);
  }
}

template <int VEC>
__device__ __forceinline__ void store(moe_bf16 *p, const float (&v)[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    *p = f32_to_bf16(v[0]);
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
    const int warps = blockDim.x >> 5;
    __syncthreads();  // the previous sum's readers are done with tmp
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.0f;
    for (int w = 0; w < warps; ++w) r += tmp[w];
    return r;
  }
}

// `lanes` threads share a row, thread l the groups of VEC values l, l +
// lanes, ... (NV of them at most).
template <int VEC, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? 1024 : 256) norm_gate_kernel(moe_norm_args a, int lanes) {
  __shared__ float tmp[32];
  const int64_t id = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int64_t r = CTA ? blockIdx.x : id / lanes;
  const int l = CTA ? threadIdx.x : static_cast<int>(id % lanes);
  const bool live = r < a.rows;  // whole groups of lanes leave the row's work together
  const int64_t outer = live ? r / a.inner : 0;
  const int head = live ? static_cast<int>(r % a.inner) : 0;
  const int64_t in_row = static_cast<int64_t>(head) * a.width;
  const int n = live ? a.width : 0;
  const int step = lanes * VEC;
  float y[NV][VEC];
  float ss = 0.0f;
  const moe_bf16 *x = a.x + outer * a.x_ld + in_row;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = l * VEC + i * step;
    if (c < n) {
      load<VEC>(x + c, y[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(y[i][j], y[i][j], ss);
    }
  }
  if (a.gamma_post) {
    const float inv = 1.0f / sqrtf(row_sum<CTA>(ss, lanes, tmp) / a.width + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = l * VEC + i * step;
      if (c < n) {
        float w[VEC];
        load<VEC>(a.gamma_post + c, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[i][j] = y[i][j] * inv * w[j];
      }
    }
  }
  float factor = a.res_scale;
  if (a.gate_kind == MOE_GATE_ROW && live)
    factor *= act(bf16_to_f32(a.gate[outer * a.gate_ld + head]), a.gate_act);
  ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = l * VEC + i * step;
    if (c < n) {
      if (a.gate_kind == MOE_GATE_CHANNEL || a.gate_kind == MOE_GATE_ELEMENT) {
        float z[VEC];
        load<VEC>(a.gate_kind == MOE_GATE_CHANNEL ? a.gate + c
                                                  : a.gate + outer * a.gate_ld + in_row + c, z);
#pragma unroll
        for (int j = 0; j < VEC; ++j) y[i][j] *= act(z[j], a.gate_act);
      }
      float res[VEC] = {};
      if (a.resid_in) load<VEC>(a.resid_in + outer * a.resid_in_ld + in_row + c, res);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        // one rounding to bf16; the next norm reads the rounded residual
        y[i][j] = bf16_to_f32(f32_to_bf16(fmaf(factor, y[i][j], res[j])));
        ss = fmaf(y[i][j], y[i][j], ss);
      }
      if (a.resid_out) store<VEC>(a.resid_out + outer * a.resid_out_ld + in_row + c, y[i]);
    }
  }
  if (a.x_next) {
    const float inv = 1.0f / sqrtf(row_sum<CTA>(ss, lanes, tmp) / a.width + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = l * VEC + i * step;
      if (c < n) {
        float w[VEC];
        load<VEC>(a.gamma_pre + c, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) w[j] = y[i][j] * inv * w[j];
        store<VEC>(a.x_next + outer * a.x_next_ld + in_row + c, w);
      }
    }
  }
}

template <int VEC, int NV, bool CTA>
cudaError_t launch(const moe_norm_args &a, int lanes, cudaStream_t s) {
  const int threads = CTA ? lanes : 256;
  const int64_t grid = CTA ? a.rows : (a.rows * lanes + threads - 1) / threads;
  norm_gate_kernel<VEC, NV, CTA><<<static_cast<unsigned>(grid), threads, 0, s>>>(a, lanes);
  return cudaGetLastError();
}

template <int VEC>
cudaError_t route(const moe_norm_args &a, cudaStream_t s) {
  const int groups = (a.width + VEC - 1) / VEC;  // groups of VEC values in a row
  if (groups <= 32) {
    int lanes = 1;
    while (lanes < groups) lanes *= 2;
    return launch<VEC, 1, false>(a, lanes, s);
  }
  if (groups <= 64) return launch<VEC, 2, false>(a, 32, s);
  if (groups <= 128) return launch<VEC, 4, false>(a, 32, s);
  if (groups <= 256) return launch<VEC, 8, false>(a, 32, s);
  if (groups <= 1024) return launch<VEC, 4, true>(a, 256, s);
  if (groups <= 4096) return launch<VEC, 4, true>(a, 1024, s);
  if constexpr (VEC == 1) return launch<VEC, 16, true>(a, 1024, s);
  return cudaErrorInvalidValue;  // not reached: width <= 16384
}

}  // namespace

cudaError_t launch_norm_gate_residual(const moe_norm_args &a, bool vec8, cudaStream_t s) {
  return vec8 ? route<8>(a, s) : route<1>(a, s);
}

}  // namespace moe
