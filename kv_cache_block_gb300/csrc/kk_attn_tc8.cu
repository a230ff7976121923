// kk_tree_attn_kv8's tensor-memory kernel (kk_attn_tc.cuh) for many query rows.
#include "kk_attn_tc.cuh"

namespace kk {
namespace {

template <int D>
cudaError_t go(AttnArgs a, cudaStream_t s) {
  const cudaError_t e =
      cudaFuncSetAttribute(attn_tc_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, true>::kSmem);
  if (e != cudaSuccess) return e;
  a.skip_tile = take_skip_tile();
  const CUtensorMap none = {};  // nothing is copied by TMA
  attn_tc_kernel<D, true><<<a.grid, tc_threads<true>(), Cfg<D, true>::kSmem, s>>>(none, none, a, 1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc8(const AttnArgs& a, cudaStream_t s) { return a.kc.D == 64 ? go<64>(a, s) : go<128>(a, s); }

}  // namespace kk
