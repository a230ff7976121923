// Work division shared by the attention kernels over a paged cache.
//
// A query row of request r and KV head h is (node i, query head h*G + g) at
// row i*G + g; rows are taken in tiles of M. An item is (r, h, row tile); its
// tokens are cut into tiles of TK: those of the cached tokens first, then those
// of the drafted nodes. Each (item, tile) is one unit of work, numbered request
// by request, and every CTA of G (the grid, or fewer when there are fewer units)
// takes total / G of them in order, the first total % G CTAs one more: the SMs
// stay level whatever the lengths are, without any work list from the
// host. An item inside one CTA's range is written out by that CTA; an item
// that ranges cut leaves one partial result per CTA (running maximum, sum and
// accumulator) in the workspace, at most two per CTA (its first and its last
// item), which the combine kernel adds up in CTA order: the same split gives
// the same bits.
#pragma once
#include "kk_device.cuh"

namespace kk {

struct AttnArgs {
  KCache kc, vc;
  Table bt;
  int layer;
  const int* sel_pages;  // selected blocks (nullable): [R][selK]
  const int* sel_logical;
  const int* sel_count;
  int selK;
  const int* node_off;  // [R+1], or null: max_nodes of every request
  int max_nodes, total_nodes;
  const uint32_t* mask;  // [total_nodes][mask_words], or null: j <= i
  int mask_words;
  const void *dk, *dv;  // drafted Keys and Values (nullable)
  long long dk_sn, dk_sh, dv_sn, dv_sh;
  const void* q;
  long long q_sn, q_sh;
  int Hq, G;
  float scale_log2;  // scale * log2(e)
  void* out;         // [total_nodes][Hq][D]
  float* lse;        // [total_nodes][Hq] or null
  int4* cuts;        // [R * H * mt_max]: the CTAs that share an item (see note_cut; twin only)
  int mt_max;        // row tiles of a request, at most
  float* ws;
  int grid;  // CTAs of the main kernel
  int twin;  // row tiles are pairs of M/2 rows; an odd last one is a single (kk_attn_tc.cu)
  // attention mass only
  const float* row_w;
  const int* row_lens;
  const int* old_lens;
  float decay;
  const float* mass_in;
  float* mass_out;
  // 8-bit caches only: [L][num_pages][H]
  const float* k_scale;
  const float* v_scale;
  unsigned long long wait_ns;
  long long skip_tile;  // failure-detection tests: CTA 0 waits for 16 bytes more than this Key tile has (-1: none)
  int* err;
};

// How a call runs: which kernel, its row and token tiles, its grid.
struct AttnPlan {
  enum Kind { kF32, kMma, kTc, kKv8 };
  Kind kind;
  int M, TK, grid;
};
// kk_attn_mma.cu (bf16; wide: 32 rows a tile instead of 16 where D is 32 or 128)
AttnPlan attn_mma_plan(const KCache& kc, bool wide);
cudaError_t launch_attn_mma(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s);
// kk_attn_f32.cu (float32; rows: query rows of a request and KV head, at most)
AttnPlan attn_f32_plan(const KCache& kc, int rows);
cudaError_t launch_attn_f32(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s);
// kk_attn_kv8.cu (e4m3 with scales)
AttnPlan attn_kv8_plan(const KCache& kc, int rows);
cudaError_t launch_attn_kv8(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s);
// kk_attn_tc.cu (bf16, D 64 or 128, both caches of layouts it suits)
bool attn_tc_suits(const KCache& kc);
AttnPlan attn_tc_plan();
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s);
// kk_attn_tc8.cu (e4m3 with scales, D 64 or 128, any layout)
inline bool attn_tc8_suits(const KCache& kc) { return kc.D == 64 || kc.D == 128; }
cudaError_t launch_attn_tc8(const AttnArgs& a, cudaStream_t s);

// kk_mass_tc.cu (bf16, D 64, 128 or 256, a layout it suits)
bool mass_tc_suits(const KCache& kc);
cudaError_t launch_mass_tc(const AttnArgs& a, cudaStream_t s);

struct AttnReq {
  int node0, n;      // first node, nodes
  int off, T;        // table start, cached tokens
  int ctx;           // token slots to visit: T, or block_size * selected blocks
  int mt, odd;       // row tiles; the last one is a single of M/2 rows
  int tiles_c, tiles;  // token tiles: cached, all (at least 1 when there are nodes)
};

// Request r's sizes; bad metadata leaves it without cached tokens (or nodes).
__device__ __forceinline__ AttnReq load_req(const AttnArgs& a, int r, int M, int TK, bool report) {
  AttnReq q;
  bool ok = true;
  q.node0 = a.node_off ? a.node_off[r] : r * a.max_nodes;
  const int n1 = a.node_off ? a.node_off[r + 1] : q.node0 + a.max_nodes;
  q.n = n1 - q.node0;
  if (q.node0 < 0 || n1 > a.total_nodes || q.n < 0 || q.n > a.max_nodes) {
    ok = false;
    q.n = 0;
    q.node0 = 0;
  }
  q.off = a.bt.offsets[r];
  const int nb = a.bt.offsets[r + 1] - q.off;
  q.T = a.bt.seq_lens[r];
  if (q.T < 0 || q.T > kMaxTokens || nb < 0 || nb > a.bt.max_blocks || nb != (int)(((unsigned)q.T + (unsigned)a.kc.bs - 1u) / (unsigned)a.kc.bs)) {
    ok = false;
    q.T = 0;
  }
  long long ctx = q.T;
  if (a.sel_pages) {
    const int c = a.sel_count[r];
    if (c < 0 || c > a.selK) ok = false;
    ctx = (c < 0 || c > a.selK || q.T == 0) ? 0 : (long long)c * a.kc.bs;
    if (ctx > kMaxTokens) {
      ok = false;
      ctx = 0;
    }
  }
  q.ctx = (int)ctx;
  q.mt = (q.n * a.G + M - 1) / M;
  q.odd = a.twin && q.n > 0 && q.n * a.G - (q.mt - 1) * M <= M / 2;
  q.tiles_c = (int)(((unsigned)q.ctx + (unsigned)TK - 1u) / (unsigned)TK);
  q.tiles = q.tiles_c + (a.dk ? (q.n + TK - 1) / TK : 0);
  if (q.tiles == 0) q.tiles = 1;
  if (a.mass_out) {  // attention mass: the unit is a token tile of one KV head, whatever its rows
    q.mt = 1;
    q.tiles = q.tiles_c;
  }
  if (report && !ok) flag_error(a.err, kErrBadIndex);
  return q;
}
__device__ __forceinline__ long long req_units(const AttnArgs& a, const AttnReq& q) {
  return (long long)a.kc.H * ((long long)(q.mt - q.odd) * q.tiles + q.odd * ((q.tiles + 1) / 2));
}

// a / b of non-negative numbers; in 32 bits, a tenth of the time, where they fit.
__device__ __forceinline__ long long udiv(long long a, long long b) {
  if (((unsigned long long)a | (unsigned long long)b) >> 32) return a / b;
  return (long long)((unsigned)a / (unsigned)b);
}
// The CTAs' ranges over `total` units.
struct Split {
  long long q;  // units of a CTA, and one more in the first `rem` CTAs
  int rem, G;
};
__device__ __forceinline__ Split make_split(long long total, int grid) {
  Split s;
  s.G = (int)min((long long)grid, total);
  s.q = s.G > 0 ? udiv(total, s.G) : 0;
  s.rem = (int)(total - s.q * s.G);
  return s;
}
__device__ __forceinline__ long long split_start(const Split& s, int c) { return c * s.q + min(c, s.rem); }
__device__ __forceinline__ int split_owner(const Split& s, long long u) {
  const long long big = (s.q + 1) * s.rem;
  return (int)(u < big ? udiv(u, s.q + 1) : s.rem + udiv(u - big, s.q));
}

// Units that a CTA has done before it comes to unit u, and those of its range.
__device__ __forceinline__ int split_time(const Split& s, long long u, int* range) {
  const long long big = (s.q + 1) * s.rem;
  *range = (int)(u < big ? s.q + 1 : s.q);
  const long long v = u < big ? u : u - big;
  return (int)(v - udiv(v, *range) * *range);
}

// An item: KV head, row tile, whether it is a single, its first unit inside
// the request and its number of units (a single's unit is two token tiles);
// [t0, t1): the units of a range that starts inside it.
struct ItemAt {
  int h, mt, units, t0, t1;
  bool single;
  long long start;
};
__device__ __forceinline__ ItemAt item_of(const AttnReq& q, int h, int mt) {
  ItemAt x;
  const int pairs = q.mt - q.odd, half = (q.tiles + 1) / 2;
  x.h = h;
  x.mt = mt;
  x.single = mt >= pairs;
  x.units = x.single ? half : q.tiles;
  x.start = h * ((long long)pairs * q.tiles + q.odd * half) + (long long)mt * q.tiles;
  x.t0 = x.t1 = 0;
  return x;
}
__device__ __forceinline__ ItemAt item_at(const AttnReq& q, long long local) {
  const long long per = (long long)(q.mt - q.odd) * q.tiles + q.odd * ((q.tiles + 1) / 2);
  const int h = (int)udiv(local, per);
  ItemAt x = item_of(q, h, min((int)udiv(local - h * per, q.tiles), q.mt - 1));
  x.t0 = (int)(local - x.start);
  return x;
}

// Element offset (without head and layer) of token slot v of a request in the
// K and V caches; false when the slot holds no valid token. `report`: tell
// a page out of range.
struct TokenAt {
  int page, tok;
};
__device__ __forceinline__ bool token_at(const AttnArgs& a, int r, const AttnReq& q, int v, bool report, TokenAt* t) {
  t->page = 0;
  t->tok = 0;
  if (v >= q.ctx) return false;
  const int bs = a.kc.bs, b = v / bs, o = v - b * bs;
  int page;
  if (a.sel_pages) {
    const int logical = a.sel_logical[(long long)r * a.selK + b];
    page = a.sel_pages[(long long)r * a.selK + b];
    if (logical < 0 || (long long)logical * bs >= q.T) {
      if (report) flag_error(a.err, kErrBadIndex);
      return false;
    }
    if ((long long)logical * bs + o >= q.T) return false;
  } else {
    page = a.bt.pages[q.off + b];
  }
  if (page < 0 || page >= a.kc.num_pages) {
    if (report) flag_error(a.err, kErrBadIndex);
    return false;
  }
  t->page = page;
  t->tok = o;
  return true;
}

// A CTA's place in the work: request `r` whose units start at `base`, and the
// range [u0, u1) of all units. Called by NT threads (a multiple of 32, at most
// 1024); `sh` is NT/32 + 4 long longs of shared memory.
struct AttnPlace {
  long long u0, u1, base, total;
  int r;
};
template <int NT>
__device__ __forceinline__ AttnPlace find_place(const AttnArgs& a, int cta, int M, int TK, long long* sh, int tid) {
  const int R = a.bt.R, per = (R + NT - 1) / NT;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += req_units(a, load_req(a, r, M, TK, cta == 0));
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kFull, incl, o);
    if ((tid & 31) >= o) incl += x;
  }
  if ((tid & 31) == 31) sh[tid >> 5] = incl;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    if (w < (tid >> 5)) before += sh[w];
    total += sh[w];
  }
  long long lo = before + incl - mine;
  AttnPlace p;
  p.total = total;
  const Split sp = make_split(total, a.grid);
  p.u0 = cta < sp.G ? split_start(sp, cta) : total;
  p.u1 = cta < sp.G ? split_start(sp, cta + 1) : total;
  long long* found = sh + NT / 32;
  if (p.u0 < p.u1 && lo <= p.u0 && p.u0 < lo + mine) {
    int r = r0;
    for (; r < r1; ++r) {
      const long long n = req_units(a, load_req(a, r, M, TK, false));
      if (p.u0 < lo + n) break;
      lo += n;
    }
    found[0] = r;
    found[1] = lo;
  }
  __syncthreads();
  p.r = p.u0 < p.u1 ? (int)found[0] : 0;
  p.base = p.u0 < p.u1 ? found[1] : 0;
  __syncthreads();
  return p;
}

// Partial results: a slot (two per CTA, and a third where row tiles come in
// pairs) holds M*D accumulators, then M running maxima (log2 domain) and M sums.
__device__ __forceinline__ float* partial_slot(const AttnArgs& a, int cta, int which, int M, int D) {
  return a.ws + (size_t)((a.twin ? 3 : 2) * cta + which) * M * (D + 2);
}

// For the tensor-memory kernel's combine: the CTA that holds an item's first unit notes itself
// and its slot (0 where the item starts its range), the one that holds the last
// unit notes itself: (first CTA, its slot, last CTA).
__device__ __forceinline__ void note_cut(const AttnArgs& a, int cta, int r, const ItemAt& it, bool starts) {
  int* c = reinterpret_cast<int*>(a.cuts + ((long long)r * a.kc.H + it.h) * a.mt_max + it.mt);
  if (it.t0 == 0) {
    c[0] = cta;
    c[1] = starts ? 0 : 1;
  }
  if (it.t1 == it.units) c[2] = cta;
}

// 1 / sum and lse of a row with running maximum m (log2 domain) and sum l; a
// row that saw nothing is 0 with lse -inf.
__device__ __forceinline__ float row_inv(float l) { return l > 0.f || l != l ? 1.f / l : 0.f; }
__device__ __forceinline__ float row_lse(float m, float l) {
  return l > 0.f || l != l ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// 16-byte asynchronous copies; one that is not `real` reads nothing and writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x; results below the normal range are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two floats as bf16, each rounded once to nearest.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <typename T>
__device__ __forceinline__ void store_elem(void* p, long long i, float v);
template <>
__device__ __forceinline__ void store_elem<float>(void* p, long long i, float v) {
  static_cast<float*>(p)[i] = v;
}
template <>
__device__ __forceinline__ void store_elem<bf16_t>(void* p, long long i, float v) {
  uint16_t h;  // one rounding to nearest, the cache's own type
  asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
  static_cast<uint16_t*>(p)[i] = h;
}

// Whether node i may see drafted node j (both inside the request).
__device__ __forceinline__ bool sees(const AttnArgs& a, const AttnReq& q, int i, int j) {
  if (!a.mask) return j <= i;
  return (a.mask[(long long)(q.node0 + i) * a.mask_words + (j >> 5)] >> (j & 31)) & 1u;
}

}  // namespace kk
