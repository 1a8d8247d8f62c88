// attn_stream_e4m3.cu -- attn_stream_kernel over a cache of e4m3.
#include "attn_stream_launch.cuh"

namespace moe {

cudaError_t launch_stream_e4m3(const AttnLaunch &x, int d) {
  return launch_stream_kv<MOE_KV_E4M3>(x, d);
}

}  // namespace moe
