// attn_tc_launch.cuh -- the launch of attn_tc_kernel for one cache type.
#pragma once

#include "attn_launch.h"
#include "attn_tc.cuh"
#include "kernels.h"

namespace moe {

template <int D, int KV>
cudaError_t launch_tc(const AttnLaunch &x) {
  using S = TcShape<D, KV>;
  const auto kernel = attn_tc_kernel<D, KV>;
  static bool attr[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    // the registers that its warps pass to one another are there at launch
    cudaFuncAttributes have;
    const cudaError_t f = cudaFuncGetAttributes(&have, kernel);
    if (f != cudaSuccess) return f;
    if (S::kSoftRegs && have.numRegs < S::kRegs) return cudaErrorLaunchOutOfResources;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  CUtensorMap tk, tv, tq;
  const int size = S::kBytes ? 1 : 2;
  const int kb = x.page < 128 ? x.page : 128, vb = x.page < S::kVKeys ? x.page : S::kVKeys;
  if (!attn_tc_map(&tk, x.k, D, size, x.cache_rows, kb, 1) ||
      !attn_tc_map(&tv, x.v, D, size, x.cache_rows, vb, S::kChunks))
    return cudaErrorInvalidValue;
  AttnArgs p = x.args;
  p.parts.rows = S::kR;
  // A query tile as whole tokens' groups of heads: one box.  (A negative or zero
  // scale enters through q: with a bf16 cache that has to pass through registers.)
  const int group = x.batch.group;
  p.q_copy = (group & (group - 1)) == 0 && (S::kBytes || p.scale_log2 > 0.0f);
  if (p.q_copy) {
    const uint64_t dims[3] = {D, static_cast<uint64_t>(group) * x.batch.kv_heads,
                              static_cast<uint64_t>(x.batch.N)};
    const uint64_t strides[2] = {D * 2, static_cast<uint64_t>(p.q_ld) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(group), 128u / group};
    if (!tc_make_map3(&tq, p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, strides, box))
      return cudaErrorInvalidValue;
  } else {
    tq = tk;  // (not used)
  }
  int grid = tc_sm_count();
  if (grid > kTcMaxCtas) grid = kTcMaxCtas;
  const cudaError_t e =
      launch_early(kernel, dim3(grid), S::kThreads, S::kSmem, x.stream, tk, tv, tq, x.batch, x.range, p);
  if (e != cudaSuccess) return e;
  return launch_attn_combine(x.batch, p, D, grid, x.stream);
}

template <int KV>
cudaError_t launch_tc_kv(const AttnLaunch &x, int d) {
  return d == 64 ? launch_tc<64, KV>(x) : d == 128 ? launch_tc<128, KV>(x) : launch_tc<256, KV>(x);
}

}  // namespace moe
