// attn_stream_int8.cu -- attn_stream_kernel over a cache of int8.
#include "attn_stream_launch.cuh"

namespace moe {

cudaError_t launch_stream_int8(const AttnLaunch &x, int d) {
  return launch_stream_kv<MOE_KV_INT8>(x, d);
}

}  // namespace moe
