// What the attention kernels that stream tokens through per-warp rings share: a
// 64-token tile in equal shares of its warps.
#pragma once
#include "kk_attn.cuh"

namespace kk {

constexpr int kRingTK = 64;

// A lane's token of the tile the warp loads next.
struct Tok {
  const char *k, *v;
  bool ok;
};

template <int ES, int TOK>
__device__ __forceinline__ Tok find_token(const AttnArgs& a, int r, const AttnReq& rq, int h, int t, int w, int lane) {
  Tok x;
  const int l = lane & (TOK - 1);
  if (t < rq.tiles_c) {
    TokenAt at;
    x.ok = token_at(a, r, rq, t * kRingTK + w * TOK + l, true, &at);
    x.k = static_cast<const char*>(a.kc.base) +
          (a.layer * a.kc.sL + at.page * a.kc.sP + h * a.kc.sH + at.tok * a.kc.sT) * ES;
    x.v = static_cast<const char*>(a.vc.base) +
          (a.layer * a.vc.sL + at.page * a.vc.sP + h * a.vc.sH + at.tok * a.vc.sT) * ES;
  } else {
    const int j = (t - rq.tiles_c) * kRingTK + w * TOK + l;
    x.ok = a.dk && t < rq.tiles && j < rq.n;
    x.k = static_cast<const char*>(x.ok ? a.dk : a.q);
    x.v = x.k;
    if (x.ok) {
      x.k += ((long long)(rq.node0 + j) * a.dk_sn + h * a.dk_sh) * ES;
      x.v = static_cast<const char*>(a.dv) + ((long long)(rq.node0 + j) * a.dv_sn + h * a.dv_sh) * ES;
    }
  }
  return x;
}

}  // namespace kk
