// Arguments of kk_kv8_write's kernel.
#pragma once
#include <algorithm>

#include "kk_internal.h"

namespace kk {

struct Write8Side {  // Keys or Values
  const void* src;
  long long sl, sn, sh;  // element strides of the new tokens: layer, node, head
  void* codes;
  long long dL, dP, dH, dT;
  float* scale;
};
struct Write8Args {
  KCache kc;  // sizes
  Table bt;
  Write8Side side[2];
  int sides;
  int f32;
  int layer, layers;
  const int* token_off;
  int max_new, num_nodes;
  int* err;
};
cudaError_t launch_kv8_write(const Write8Args& a, cudaStream_t s);

}  // namespace kk
