// attn_tc_int8.cu -- attn_tc_kernel over a cache of int8.
#include "attn_tc_launch.cuh"

namespace moe {

cudaError_t launch_tc_int8(const AttnLaunch &x, int d) { return launch_tc_kv<MOE_KV_INT8>(x, d); }

}  // namespace moe
