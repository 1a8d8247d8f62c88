// attn_stream_bf16.cu -- attn_stream_kernel over a cache of bf16.
#include "attn_stream_launch.cuh"

namespace moe {

cudaError_t launch_stream_bf16(const AttnLaunch &x, int d) {
  return launch_stream_kv<MOE_KV_BF16>(x, d);
}

}  // namespace moe
