// attn_launch.h -- what passes between the choice of an attention kernel and
// the files that hold the kernels of each cache type (internal).
#pragma once

#include <cuda.h>

#include "attn_args.cuh"

namespace moe {

struct AttnLaunch {
  const void *k, *v;
  int64_t cache_rows;  // pages * kv_heads * page
  int page;
  AttnBatch batch;
  AttnRange range;
  AttnArgs args;
  cudaStream_t stream;
};

// The cache's rows of d elements of `size` bytes as lines of 128 bytes: a box
// is `box` positions of one page and head, all their columns.
bool attn_map(CUtensorMap *m, const void *base, int d, int size, int64_t rows, int box);

// The same rows as columns of 64 elements (128 bytes with the swizzle, or 64
// of codes as they lie): a box is `box` positions by `cols` of them.
bool attn_tc_map(CUtensorMap *m, const void *base, int d, int size, int64_t rows, int box, int cols);

cudaError_t launch_tc_bf16(const AttnLaunch &x, int d);
cudaError_t launch_tc_int8(const AttnLaunch &x, int d);
cudaError_t launch_tc_e4m3(const AttnLaunch &x, int d);

cudaError_t launch_stream_bf16(const AttnLaunch &x, int d);
cudaError_t launch_stream_int8(const AttnLaunch &x, int d);
cudaError_t launch_stream_e4m3(const AttnLaunch &x, int d);

// Joins the tiles that the `blocks` blocks of the kernel before it left apart.
cudaError_t launch_attn_combine(const AttnBatch &a, const AttnArgs &p, int d, int blocks,
                                cudaStream_t s);

}  // namespace moe
