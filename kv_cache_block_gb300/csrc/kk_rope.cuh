// Arguments of kk_qk_norm_rope's kernel.
#pragma once
#include <algorithm>

#include "kk_internal.h"

namespace kk {

struct RopeRows {  // [node][head][D], element strides
  void* base;
  long long sn, sh;
};
struct RopeArgs {
  int f32, nodes, Hq, H, D;
  RopeRows q, k, v_rows, q_out, k_out;
  bool v;  // Values are written to vc
  const void *q_weight, *k_weight;
  float eps;
  const int* positions;
  const float* inv_freq;
  int rd, half;  // rotary dims; pairs (i, i + rd / 2), else (2i, 2i + 1)
  float rope_scale;
  // the caches' slots (kc null: none); bt.offsets null: no table
  void *kc, *vc;
  long long kL, kP, kH, kT, vL, vP, vH, vT;
  int bs, num_pages, layer;
  Table bt;
  const int* token_off;
  int* err;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s);

}  // namespace kk
