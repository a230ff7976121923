// kk_tree_attn's tensor-memory kernel (kk_attn_tc.cuh) on bf16 caches.
#include "kk_attn_tc.cuh"

namespace kk {
namespace {

template <int D>
cudaError_t go(AttnArgs a, cudaStream_t s) {
  CUtensorMap tk, tv;
  const int tb = tile_piece(a.kc.bs, kTK);
  if (!encode_tile_map(a.kc, a.layer, tb, &tk) || !encode_tile_map(a.vc, a.layer, tb, &tv)) return cudaErrorNotSupported;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_tc_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, false>::kSmem);
  if (e != cudaSuccess) return e;
  a.skip_tile = take_skip_tile();
  attn_tc_kernel<D, false><<<a.grid, tc_threads<false>(), Cfg<D, false>::kSmem, s>>>(tk, tv, a, tb);
  return cudaGetLastError();
}

}  // namespace

bool attn_tc_suits(const KCache& kc) { return (kc.D == 64 || kc.D == 128) && tile_layout_suits(kc); }

AttnPlan attn_tc_plan() { return AttnPlan{AttnPlan::kTc, 256, kTK, sm_count()}; }

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) {
  return a.kc.D == 64 ? go<64>(a, s) : go<128>(a, s);
}

}  // namespace kk
