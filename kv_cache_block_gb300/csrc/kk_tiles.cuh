// What the tensor-core kernels over a paged cache share: waits of whole warps,
// and the TMA view of one layer's pages.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kk_attn.cuh"
#include "kk_tcgen05.cuh"

namespace kk {

// ---- tensor cores, beyond kk_tcgen05.cuh ---------------------------------------
// Rows of 128 bytes in the 128-byte swizzle (as desc_kmajor_sw128's) as an
// MN-major operand, whose rows run along the contracted axis: 8-row groups 1024 bytes apart (stride byte offset), the next 64
// elements of a row `chunk` bytes on (leading byte offset).
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr, uint32_t chunk) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(chunk >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescBMajorMN = 1u << 16;  // instruction descriptor: B is MN-major

// mma_bf16 with the descriptors' low words (the address field moves with them)
// and their shared high word; and with A in TMEM (bf16, two per column, a row
// per lane). A whole warp keeps these operands uniform and one elected lane
// issues.
__device__ __forceinline__ void mma_bf16_lo(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t hi, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t hi,
                                               uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Loads 8 consecutive columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}
// Stores 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Makes this thread's writes to shared memory visible to TMA and the tensor cores.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 4-D tiled load, as tma_load_5d.
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int c0, int c1, int c2, int c3,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}


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
