// attn_stream_launch.cuh -- the launch of attn_stream_kernel for one cache type.
#pragma once

#include "attn_launch.h"
#include "attn_stream.cuh"
#include "kernels.h"

namespace moe {

template <int D, int KV>
cudaError_t launch_stream(const AttnLaunch &x) {
  using S = StreamShape<D, KV>;
  const auto kernel = attn_stream_kernel<D, KV>;
  static bool attr[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr[dev] = true;
  }
  CUtensorMap tk, tv;
  if (!attn_map(&tk, x.k, D, S::kBytes ? 1 : 2, x.cache_rows, 64 < x.page ? 64 : x.page) ||
      !attn_map(&tv, x.v, D, S::kBytes ? 1 : 2, x.cache_rows, 64 < x.page ? 64 : x.page))
    return cudaErrorInvalidValue;
  AttnArgs p = x.args;
  p.parts.rows = S::kR;
  int grid = tc_sm_count() * S::kBlocks;
  if (grid > kStreamMaxCtas) grid = kStreamMaxCtas;
  const cudaError_t e = launch_early(kernel, dim3(grid), S::kThreads, S::kSmem, x.stream, tk, tv,
                                     x.batch, x.range, p);
  if (e != cudaSuccess) return e;
  return launch_attn_combine(x.batch, p, D, grid, x.stream);
}

template <int KV>
cudaError_t launch_stream_kv(const AttnLaunch &x, int d) {
  return d == 64    ? launch_stream<64, KV>(x)
         : d == 128 ? launch_stream<128, KV>(x)
                    : launch_stream<256, KV>(x);
}

}  // namespace moe
