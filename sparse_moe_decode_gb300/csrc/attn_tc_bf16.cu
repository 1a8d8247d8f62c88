// attn_tc_bf16.cu -- attn_tc_kernel over a cache of bf16.
#include "attn_tc_launch.cuh"

namespace moe {

cudaError_t launch_tc_bf16(const AttnLaunch &x, int d) { return launch_tc_kv<MOE_KV_BF16>(x, d); }

}  // namespace moe
