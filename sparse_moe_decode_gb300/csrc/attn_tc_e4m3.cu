// attn_tc_e4m3.cu -- attn_tc_kernel over a cache of e4m3.
#include "attn_tc_launch.cuh"

namespace moe {

cudaError_t launch_tc_e4m3(const AttnLaunch &x, int d) { return launch_tc_kv<MOE_KV_E4M3>(x, d); }

}  // namespace moe
