// kk_tree_attn_kv8's kernels for 128 and 256 dims (kk_attn_kv8.cuh): a unit of their own, to compile beside.
#include "kk_attn_kv8.cuh"

namespace kk {

AttnPlan attn_kv8_plan_wide(const KCache& kc, int rows) {
  return kc.D == 128 ? plan_d<128>(rows) : plan_d<256>(rows);
}

cudaError_t launch_attn_kv8_wide(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  return a.kc.D == 128 ? go_d<128>(a, pl, s) : a.kc.D == 256 ? go_d<256>(a, pl, s) : cudaErrorNotSupported;
}

}  // namespace kk
