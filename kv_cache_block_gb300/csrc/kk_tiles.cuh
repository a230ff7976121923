// What the tensor-core kernels over a paged cache share: waits of whole warps,
// and the TMA view of one layer's pages.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kk_attn.cuh"
#include "kk_tcgen05.cuh"

namespace kk {

// A value all lanes hold, as one the compiler knows to be uniform (the warp-wide
// reduction's result lives in a uniform register, a shuffle's does not): what
// issues copies and MMAs takes its operands from there.
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __reduce_or_sync(kFull, x); }
__device__ __forceinline__ int uni(int x) { return (int)__reduce_or_sync(kFull, (unsigned)x); }

// Waits for a barrier's phase with the whole warp; gives up (false) past the
// limit or when another role has given up, and tells the others. All lanes leave
// the loop at once: what the warp does next takes its addresses from uniform
// registers and must not be reached by some lanes before the others.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const AttnArgs& a, volatile int* stop) {
  uint32_t n = 0;
  uint64_t t0 = 0;
  while (!__all_sync(kFull, mbar_try_wait(bar, parity))) {
    if ((++n & 63u) != 0) continue;  // the timer is slow to read
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    const bool late = now - t0 > a.wait_ns;
    if (__any_sync(kFull, late || *stop)) {
      if (late) {
        *stop = 1;
        flag_error(a.err, kErrTimeout);
      }
      __syncwarp();
      return false;
    }
  }
  return true;
}

// 4-D map of one layer: 64 dims x `tb` tokens of a (token, head, page) cache.
inline bool encode_tile_map(const KCache& kc, int layer, int tb, CUtensorMap* tm) {
  auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (!encode) return false;
  const long long ext[3] = {kc.bs, kc.H, kc.num_pages}, st[3] = {kc.sT * 2, kc.sH * 2, kc.sP * 2};
  cuuint64_t dims[4] = {(cuuint64_t)kc.D, 0, 0, 0}, strides[3];
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = (cuuint64_t)ext[i];
    strides[i] = ext[i] == 1 ? (cuuint64_t)kc.D * 2 : (cuuint64_t)st[i];
  }
  const cuuint32_t box[4] = {64, (cuuint32_t)tb, 1, 1}, es[4] = {1, 1, 1, 1};
  void* at = const_cast<uint16_t*>(static_cast<const uint16_t*>(kc.base) + layer * kc.sL);
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, at, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens of a TMA box: the largest divisor of both the block and the tile.
inline int tile_piece(int bs, int tile) {
  int a = bs, b = tile;
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// Whether a bf16 cache's pages can be loaded so: whole 8-row swizzle groups in a
// block, and strides a tensor map takes.
inline bool tile_layout_suits(const KCache& kc) {
  if (kc.dtype != 1 || kc.D % 64 != 0 || kc.bs % 8 != 0) return false;
  const long long ext[3] = {kc.bs, kc.H, kc.num_pages}, st[3] = {kc.sT, kc.sH, kc.sP};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && (st[i] < 8 || st[i] * 2 >= (1ll << 40))) return false;
  return true;
}

}  // namespace kk
