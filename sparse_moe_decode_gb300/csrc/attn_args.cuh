// attn_args.cuh -- what the attention kernels share: their arguments, the
// unfinished tiles' sums in the workspace, conversions of cached codes.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_sched.cuh"
#include "pair.cuh"

namespace moe {

// Unfinished tiles: block b's part 2 b is of the tile that the block did not
// begin, part 2 b + 1 of the one that it began and did not finish.
struct AttnParts {
  AttnOpen *open;  // [blocks]
  float2 *ml;      // [2 blocks][rows]: maximum (in powers of two) and total
  float *sums;     // [2 blocks][head_dim / 4][rows][4]: rows lie side by side
  int rows;        // of a tile
  // four columns from d on of a part's row
  __device__ __forceinline__ float *at(int64_t part, int head_dim, int d, int row) const {
    return sums + ((part * (head_dim / 4) + d / 4) * rows + row) * 4;
  }
};

struct AttnArgs {
  const moe_bf16 *q;
  moe_bf16 *out;
  int64_t q_ld, out_ld;
  const float *k_scale, *v_scale;
  AttnParts parts;
  float scale_log2;  // scale * log2(e)
  int least_share;
  int q_copy;  // q's tiles come by TMA
  unsigned long long budget;
};

__device__ __forceinline__ float attn_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The power of two at or below x, in [2^-110, 2^126], and its inverse.
__device__ __forceinline__ float pow2_floor(float x) {
  const uint32_t e = __float_as_uint(x) & 0x7F800000u;
  return __uint_as_float(min(max(e, (127u - 110u) << 23), (127u + 126u) << 23));
}
__device__ __forceinline__ float pow2_inverse(float p) {
  return __uint_as_float((254u << 23) - __float_as_uint(p));
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(v));
  return r;
}

// Four codes as fp16, exactly: bytes 0, 1 and 2, 3.
template <int KV>
__device__ __forceinline__ void codes_to_f16x2(uint32_t v, uint32_t &lo, uint32_t &hi) {
  if (KV == MOE_KV_INT8) {
    i8x4_to_f16x2(v, lo, hi);
  } else {
    lo = e4m3x2_to_f16x2(v);
    hi = e4m3x2_to_f16x2(v >> 16);
  }
}
// Bytes 0, 2 and 1, 3.
template <int KV>
__device__ __forceinline__ void codes_to_f16x2_apart(uint32_t v, uint32_t &even, uint32_t &odd) {
  codes_to_f16x2<KV>(__byte_perm(v, 0, 0x3120), even, odd);
}

}  // namespace moe
