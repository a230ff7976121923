// kk_tree_attn_kv8's kernels for 32 and 64 dims (kk_attn_kv8.cuh), and their choice.
#include "kk_attn_kv8.cuh"

namespace kk {

AttnPlan attn_kv8_plan_wide(const KCache& kc, int rows);
cudaError_t launch_attn_kv8_wide(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s);

AttnPlan attn_kv8_plan(const KCache& kc, int rows) {
  return kc.D == 32 ? plan_d<32>(rows) : kc.D == 64 ? plan_d<64>(rows) : attn_kv8_plan_wide(kc, rows);
}

cudaError_t launch_attn_kv8(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  return a.kc.D == 32 ? go_d<32>(a, pl, s) : a.kc.D == 64 ? go_d<64>(a, pl, s) : launch_attn_kv8_wide(a, pl, s);
}

}  // namespace kk
