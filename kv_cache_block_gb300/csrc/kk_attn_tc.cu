// kk_tree_attn on bf16 caches with many query rows per KV head (a draft tree,
// a piece of a prompt): bound by the tensor cores and the exponentials.
//
// One CTA per SM with two streams, A and B, each a 128-row tile with its own
// scores S (128 TMEM columns) and accumulator O (D columns). Warps 0-3 are
// A's softmax, warps 4-7 B's (a thread owns a row), warp 8 issues every MMA
// (tcgen05), warps 9-11 load. While one stream's softmax runs, the tensor cores
// work for the other:
//   S_x = Q_x K^T    both operands in shared memory
//   P_x = exp2(S_x * c - m_x)  written over S_x as bf16, the A operand
//   O_x += P_x V     P from TMEM, V from shared memory as it lies (MN-major)
// MMAs of one thread run in order, so S_x of the next tile may follow P_x V at
// once. The maximum a row's weights are taken against moves only when the true
// one has risen past it by 2^8: until then the weights stay below 2^8, which
// costs bf16 nothing, and O need not be rescaled.
//
// An item is a pair of row tiles (both streams take every token tile) or, for
// the last tile of an odd number, a single one (the streams take alternate
// token tiles and leave two partial results): either way a unit of work is two
// tile products, and both streams are busy.
//
// Full tiles of tokens come by TMA (one box per page piece and 64 dims, 128-byte
// swizzle). Tiles with a place that holds no token (the end of a request, a
// partial selected block, a bad page) and tiles of drafted nodes are copied by
// the loader warps, zeros for what is not there: a weight of zero must not meet
// what such a place holds.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>

#include "kk_attn.cuh"
#include "kk_pdl.cuh"
#include "kk_tcgen05.cuh"

namespace kk {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kLoaders = 96;
constexpr int kTK = 128;
constexpr int kMeta = 8;  // ring of per-tile notes from the loaders to the softmax warps
constexpr int kTmemCols = 512;
constexpr float kRise = 8.f;

// Notes on a tile for the softmax warps: which places hold a token, the drafted
// tile it is (-1: cached tokens), and whether a drafted Value is not finite.
struct TileNote {
  uint32_t live[4];
  int draft;
  int odd;
};

template <int D>
struct Cfg {
  static constexpr int NC = D / 64;           // 64-dim chunks
  static constexpr int ST = D == 64 ? 4 : 2;  // stages of K and of V
  static constexpr int kChunk = 128 * 128;    // bytes of a chunk of 128 rows
  static constexpr int kTile = NC * kChunk;   // bytes of 128 rows
  static constexpr int kSmem = 2 * kTile + 2 * ST * kTile + 1024;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t note[kMeta];
  uint64_t drain;
};

// Waits for a barrier's phase; gives up (false) past the limit or when another
// role has given up, and tells the others.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const AttnArgs& a, volatile int* stop) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*stop) return false;
    if (globaltimer_ns() - t0 > a.wait_ns) {
      *stop = 1;
      flag_error(a.err, kErrTimeout);
      return false;
    }
  }
  return true;
}

// An item's place in a CTA's range.
struct Work {
  AttnReq rq;
  ItemAt at;
  int r, row0, rows;  // rows of the item (at most 256)
  int first, tiles;   // token tiles [first, first + tiles)
};
// The item that holds unit u; advances (r, base) past finished requests.
__device__ __forceinline__ Work work_at(const AttnArgs& a, const AttnPlace& pl, long long u, int* r, long long* base) {
  Work w;
  for (;;) {
    w.rq = load_req(a, *r, 256, kTK, false);
    const long long n = req_units(a, w.rq);
    if (u < *base + n) break;
    *base += n;
    ++*r;
  }
  w.r = *r;
  w.at = item_at(w.rq, u - *base);
  w.at.t1 = (int)min((long long)w.at.units, w.at.t0 + (pl.u1 - u));
  w.row0 = w.at.mt * 256;
  w.rows = min(w.at.single ? 128 : 256, w.rq.n * a.G - w.row0);
  w.first = w.at.single ? 2 * w.at.t0 : w.at.t0;
  w.tiles = (w.at.single ? min(2 * w.at.t1, w.rq.tiles) : w.at.t1) - w.first;
  return w;
}

// Takes out what is not finite among eight bf16 values; true if there was any.
__device__ __forceinline__ bool drop_nonfinite(uint4* x) {
  uint32_t* y = reinterpret_cast<uint32_t*>(x);
  bool hit = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((y[e] & 0x7F800000u) == 0x7F800000u) y[e] &= 0x0000FFFFu, hit = true;
    if ((y[e] & 0x00007F80u) == 0x00007F80u) y[e] &= 0xFFFF0000u, hit = true;
  }
  return hit;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const AttnArgs a,
                   const int tb) {
  using C = Cfg<D>;
  constexpr int NC = C::NC, ST = C::ST;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* s_q = smem;
  unsigned char* s_k = s_q + 2 * C::kTile;
  unsigned char* s_v = s_k + ST * C::kTile;
  __shared__ Bars b;
  __shared__ TileNote s_note[kMeta];
  __shared__ long long s_place[kThreads / 32 + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_stop;
  volatile int* stop = &s_stop;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(&b.q_full, 1);
    mbar_init(&b.q_empty, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.k_full[i], 1);
      mbar_init(&b.k_empty[i], 1);
      mbar_init(&b.v_full[i], 1);
      mbar_init(&b.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.p_full[i], 4);
      mbar_init(&b.o_full[i], 1);
      mbar_init(&b.o_empty[i], 4);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&b.note[i], 1);
    mbar_init(&b.drain, 1);
    s_stop = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  const AttnPlace pl = find_place<kThreads>(a, blockIdx.x, 256, kTK, s_place, tid);  // holds block barriers
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int r = pl.r;
  long long base = pl.base;

  // Registers: 168 a thread at launch; the softmax warps hold a row of scores.
  // 2 * 208 + 88 = 3 * 168, so every request is met from what the others return.
  if (warp < 8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");

  if (warp < 8) {
    // ---- softmax: stream x, row `row` of its tile -----------------------------
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_at + x * 128, o_at = tmem + lane_at + 256 + x * 128;
    // scale 0 still has to leave hidden places at -inf: the smallest normal number stands for it
    const float c = fmaxf(fabsf(a.scale_log2), FLT_MIN);
    uint32_t seen = 0, notes = 0, items = 0;  // S tiles of this stream, tiles of the CTA, items
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      const Work w = work_at(a, pl, u, &r, &base);
      const int sub = w.at.single ? 0 : x;  // row tile of the stream
      const int steps = w.at.single ? (w.tiles + 1 - x) / 2 : w.tiles;
      const int rows = w.rows - sub * 128;
      const bool busy = (warp & 3) * 32 < rows;  // this warp has rows at all
      const int qrow = w.row0 + sub * 128 + row;
      const int node = min(qrow / a.G, w.rq.n - 1);
      float m_ref = -INFINITY, l = 0.f;  // in units of S
      uint32_t odd = 0;
      for (int i = 0; i < steps; ++i) {
        const uint32_t no = notes + (w.at.single ? 2 * i + x : i);
        const TileNote* note = &s_note[no % kMeta];
        alive = wait(&b.note[no % kMeta], (no / kMeta) & 1, a, stop) && wait(&b.s_full[x], seen & 1, a, stop);
        ++seen;
        alive = __all_sync(kFull, alive);
        if (!alive) break;
        tc_fence_after();
        if (busy) {
          uint32_t s[4][32];
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32(s_at + k * 32, s[k]);
          uint32_t live[4] = {note->live[0], note->live[1], note->live[2], note->live[3]};
          const int draft = note->draft;
          if (draft >= 0) {
            if (note->odd) odd |= 1u << draft;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int j0 = draft * kTK + k * 32;
              uint32_t see = 0xFFFFFFFFu;
              if (!a.mask)
                see = node < j0 ? 0u : node - j0 >= 31 ? 0xFFFFFFFFu : (2u << (node - j0)) - 1u;
              else if (draft * 4 + k < a.mask_words)
                see = a.mask[(long long)(w.rq.node0 + node) * a.mask_words + draft * 4 + k];
              live[k] &= see;
            }
          }
          tmem_wait_ld();
          if ((live[0] & live[1] & live[2] & live[3]) != 0xFFFFFFFFu) {
            // selected, whatever a hidden place holds
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((live[k] >> e) & 1u)) s[k][e] = 0xFF800000u;
          }
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mx[k] = __uint_as_float(s[k][0]);
#pragma unroll
            for (int e = 1; e < 32; ++e) mx[k] = fmaxf(mx[k], __uint_as_float(s[k][e]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const bool first = i == 0;
          const bool rise = first || (top - m_ref) * c > kRise || (m_ref == -INFINITY && top > m_ref);
          if (__any_sync(kFull, rise)) {
            float al = 1.f;
            if (rise) {
              const float m2 = fmaxf(m_ref, top);
              al = m_ref == -INFINITY ? 0.f : ex2((m_ref - m2) * c);
              m_ref = m2;
              l *= al;
            }
            if (!first) {  // S of this tile is complete, so is every product into O before it
#pragma unroll 1
              for (int k = 0; k < D / 32; ++k) {
                uint32_t o[32];
                tmem_ld32(o_at + k * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                tmem_st32(o_at + k * 32, o);
              }
            }
          }
          const float mc = m_ref == -INFINITY ? 0.f : m_ref * c;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            uint32_t p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float p0 = ex2(__uint_as_float(s[k + e / 16][(2 * e) % 32]) * c - mc);
              const float p1 = ex2(__uint_as_float(s[k + e / 16][(2 * e + 1) % 32]) * c - mc);
              sum[e & 3] += p0 + p1;
              p[e] = pack_bf16(p0, p1);  // the weights' one rounding
            }
            tmem_st32(s_at + k * 16, p);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.p_full[x]);
      }
      notes += w.tiles;
      // ---- the item's end: O and the row's maximum and sum
      if (alive && steps > 0) alive = __all_sync(kFull, wait(&b.o_full[x], items & 1, a, stop));
      if (!alive) break;
      tc_fence_after();
      const bool whole = !w.at.single && w.at.t0 == 0 && w.at.t1 == w.at.units;
      const bool mine = row < rows;
      const float inv = row_inv(l), ml2 = m_ref == -INFINITY ? -INFINITY : m_ref * c;
      const int prow = x * 128 + row;  // row of the partial slot (both streams of a single item leave one)
      float* part = partial_slot(a, blockIdx.x, u == pl.u0 ? 0 : 1, 256, D);
      const long long at = (long long)(w.rq.node0 + qrow / a.G) * a.Hq + w.at.h * a.G + qrow % a.G;
      if (busy) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          if (steps > 0) {
            tmem_ld32(o_at + k * 32, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (mine) {
            if (odd) {  // drafted Values that are not finite, for the nodes that see them
              for (int j = 0; j < w.rq.n; ++j) {
                if (!((odd >> (j >> 7)) & 1u) || !sees(a, w.rq, node, j)) continue;
                const uint16_t* v = static_cast<const uint16_t*>(a.dv) + (w.rq.node0 + j) * a.dv_sn + w.at.h * a.dv_sh;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const uint32_t y = v[k * 32 + e];
                  if ((y & 0x7F80u) == 0x7F80u)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(y << 16));
                }
              }
            }
            if (whole) {
              uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + k * 32);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int f = 0; f < 4; ++f)
                  y[f] =
                      pack_bf16(__uint_as_float(o[e * 8 + f * 2]) * inv, __uint_as_float(o[e * 8 + f * 2 + 1]) * inv);
                out[e] = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else {
              uint4* out = reinterpret_cast<uint4*>(part + (size_t)prow * D + k * 32);
#pragma unroll
              for (int e = 0; e < 8; ++e) out[e] = make_uint4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
            }
          }
          __syncwarp();
        }
        if (mine) {
          if (whole) {
            if (a.lse) a.lse[at] = row_lse(ml2, l);
          } else {
            part[256 * D + prow] = ml2;
            part[256 * D + 256 + prow] = l;
          }
        }
      }
      if (steps > 0) {
        ++items;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.o_empty[x]);
      }
      u += w.at.t1 - w.at.t0;
    }
  } else if (warp == kMmaWarp) {
    // ---- every MMA, by one thread ---------------------------------------------
    if (lane == 0) {
      constexpr uint32_t idqk = idesc_bf16_f32(128, 128), idpv = idesc_bf16_f32(128, D) | kIdescBMajorMN;
      uint32_t kc = 0, vc = 0, nitem = 0, pc[2] = {0, 0}, oc[2] = {0, 0};
      bool alive = true, any = false;
      for (long long u = pl.u0; u < pl.u1 && alive;) {
        const Work w = work_at(a, pl, u, &r, &base);
        const bool single = w.at.single;
        const int steps[2] = {single ? (w.tiles + 1) / 2 : w.tiles, single ? w.tiles / 2 : w.tiles};
        alive = wait(&b.q_full, nitem & 1, a, stop);
        if (!alive) break;
        any = true;
        // S_x of its next tile; K is let go behind its last reader
        auto qk = [&](int x) {
          const bool fresh = single || x == 0;
          const uint32_t st = (fresh ? kc : kc - 1) % ST;
          if (fresh) {
            if (!wait(&b.k_full[st], (kc / ST) & 1, a, stop)) return false;
            ++kc;
          }
          tc_fence_after();
          const uint32_t q0 = smem_u32(s_q) + (single ? 0 : x) * C::kTile, k0 = smem_u32(s_k) + st * C::kTile;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * C::kChunk + (k % 4) * 32;
            mma_bf16(tmem + x * 128, desc_kmajor_sw128(q0 + off), desc_kmajor_sw128(k0 + off), idqk, k > 0);
          }
          mma_commit(&b.s_full[x]);
          if (single || x == 1) mma_commit(&b.k_empty[st]);
          return true;
        };
        auto pv = [&](int x, bool first) {
          const bool fresh = single || x == 0;
          const uint32_t st = (fresh ? vc : vc - 1) % ST;
          if (!wait(&b.p_full[x], pc[x] & 1, a, stop)) return false;
          ++pc[x];
          if (fresh) {
            if (!wait(&b.v_full[st], (vc / ST) & 1, a, stop)) return false;
            ++vc;
          }
          // O is read out before the next item writes it
          if (first && oc[x] > 0 && !wait(&b.o_empty[x], (oc[x] - 1) & 1, a, stop)) return false;
          tc_fence_after();
          const uint32_t v0 = smem_u32(s_v) + st * C::kTile;
#pragma unroll
          for (int k = 0; k < kTK / 16; ++k)
            mma_bf16_ts(tmem + 256 + x * 128, tmem + x * 128 + k * 8, desc_mnmajor_sw128(v0 + k * 2048, C::kChunk), idpv,
                        !(first && k == 0));
          if (single || x == 1) mma_commit(&b.v_empty[st]);
          return true;
        };
        for (int x = 0; x < 2 && alive; ++x)
          if (steps[x] > 0) alive = qk(x);
        for (int i = 0; i < steps[0] && alive; ++i) {
          if (i == steps[0] - 1) mma_commit(&b.q_empty);  // every S of the item is on its way
          for (int x = 0; x < 2 && alive; ++x) {
            if (i >= steps[x]) continue;
            alive = pv(x, i == 0);
            if (!alive) break;
            if (i + 1 < steps[x]) {
              alive = qk(x);
            } else {
              mma_commit(&b.o_full[x]);
              ++oc[x];
            }
          }
        }
        ++nitem;
        u += w.at.t1 - w.at.t0;
      }
      if (any) {  // nothing may be in flight when TMEM and shared memory go
        mma_commit(&b.drain);
        mbar_wait_bounded(&b.drain, 0, a.wait_ns);
      }
    }
    __syncwarp();
  } else {
    // ---- loaders: three warps that stay in step (they leave together) ------------
    const int lt = tid - kLoadWarp * 32;
    const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale turns the queries' signs
    const int npiece = kTK / tb;                                  // page pieces of a tile
    uint32_t cnt = 0, nitem = 0;
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1;) {
      const Work w = work_at(a, pl, u, &r, &base);
      const int h = w.at.h, nsub = w.at.single ? 1 : 2;
      if (alive && nitem > 0) alive = wait(&b.q_empty, (nitem - 1) & 1, a, stop);
      alive = !named_sync_or(1, kLoaders, !alive);
      if (!alive) break;
      for (int i = lt; i < nsub * 128 * (D / 8); i += kLoaders) {
        const int m = i / (D / 8), c8 = i % (D / 8), qrow = w.row0 + m;
        uint4 y = make_uint4(0, 0, 0, 0);
        if (m < w.rows) {
          y = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (w.rq.node0 + qrow / a.G) * a.q_sn +
                                              (long long)(h * a.G + qrow % a.G) * a.q_sh + c8 * 8);
          y.x ^= flip;
          y.y ^= flip;
          y.z ^= flip;
          y.w ^= flip;
        }
        *reinterpret_cast<uint4*>(s_q + (m >> 7) * C::kTile + (c8 >> 3) * C::kChunk + (m & 127) * 128 +
                                  (((c8 & 7) ^ (m & 7)) << 4)) = y;
      }
      fence_async_smem();
      named_sync(1, kLoaders);
      if (lt == 0) mbar_arrive(&b.q_full);
      ++nitem;
      for (int i = 0; i < w.tiles; ++i, ++cnt) {
        const int t = w.first + i;
        const uint32_t st = cnt % ST, ph = ((cnt / ST) & 1) ^ 1;
        TileNote* note = &s_note[cnt % kMeta];
        const bool draft = t >= w.rq.tiles_c;
        // a piece is a run of tb tokens in one page (tb divides the block size)
        int page = 0, tok = 0;
        bool full = true;
        if (!draft && lane < npiece) {
          TokenAt at;
          const int v = t * kTK + lane * tb;
          full = token_at(a, w.r, w.rq, v + tb - 1, false, &at) && token_at(a, w.r, w.rq, v, false, &at);
          page = at.page;
          tok = at.tok;
        }
        full = __all_sync(kFull, full) && !draft;
        alive = alive && wait(&b.k_empty[st], ph, a, stop);
        alive = !named_sync_or(1, kLoaders, !alive);
        if (!alive) break;
        if (full) {
          if (warp == kLoadWarp) {
            if (lane == 0) {
              note->live[0] = note->live[1] = note->live[2] = note->live[3] = 0xFFFFFFFFu;
              note->draft = -1;
              note->odd = 0;
              mbar_arrive(&b.note[cnt % kMeta]);
              mbar_arrive_expect_tx(&b.k_full[st], C::kTile);
            }
            __syncwarp();
            if (lane < npiece) {
#pragma unroll
              for (int c = 0; c < NC; ++c)
                tma_load_4d(s_k + st * C::kTile + c * C::kChunk + lane * tb * 128, &tmk, c * 64, tok, h, page,
                            &b.k_full[st]);
            }
            alive = __all_sync(kFull, wait(&b.v_empty[st], ph, a, stop));
            if (alive) {
              if (lane == 0) mbar_arrive_expect_tx(&b.v_full[st], C::kTile);
              __syncwarp();
              if (lane < npiece) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                  tma_load_4d(s_v + st * C::kTile + c * C::kChunk + lane * tb * 128, &tmv, c * 64, tok, h, page,
                              &b.v_full[st]);
              }
            }
          }
          continue;
        }
        // copied by the 96 threads
        alive = wait(&b.v_empty[st], ph, a, stop);
        alive = !named_sync_or(1, kLoaders, !alive);
        if (!alive) break;
        bool hit = false;
        for (int j = lt; j < kTK * (D / 8); j += kLoaders) {
          const int m = j / (D / 8), c8 = j % (D / 8);
          uint4 ky = make_uint4(0, 0, 0, 0), vy = ky;
          if (!draft) {
            TokenAt at;
            if (token_at(a, w.r, w.rq, t * kTK + m, false, &at)) {
              ky = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.kc.base) + a.layer * a.kc.sL +
                                                   at.page * a.kc.sP + h * a.kc.sH + at.tok * a.kc.sT + c8 * 8);
              vy = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.vc.base) + a.layer * a.vc.sL +
                                                   at.page * a.vc.sP + h * a.vc.sH + at.tok * a.vc.sT + c8 * 8);
            }
          } else {
            const int n = (t - w.rq.tiles_c) * kTK + m;
            if (a.dk && n < w.rq.n) {
              ky = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dk) + (w.rq.node0 + n) * a.dk_sn +
                                                   h * a.dk_sh + c8 * 8);
              vy = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dv) + (w.rq.node0 + n) * a.dv_sn +
                                                   h * a.dv_sh + c8 * 8);
              hit |= drop_nonfinite(&vy);  // added back to the nodes that see it at the end
            }
          }
          const uint32_t off = st * C::kTile + (c8 >> 3) * C::kChunk + m * 128 + (((c8 & 7) ^ (m & 7)) << 4);
          *reinterpret_cast<uint4*>(s_k + off) = ky;
          *reinterpret_cast<uint4*>(s_v + off) = vy;
        }
        fence_async_smem();
        hit = named_sync_or(1, kLoaders, hit);
        if (warp == kLoadWarp) {
          uint32_t live[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            TokenAt at;
            const int n = (t - w.rq.tiles_c) * kTK + k * 32 + lane;
            const bool ok = draft ? a.dk && n < w.rq.n : token_at(a, w.r, w.rq, t * kTK + k * 32 + lane, true, &at);
            live[k] = __ballot_sync(kFull, ok);
          }
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < 4; ++k) note->live[k] = live[k];
            note->draft = draft ? t - w.rq.tiles_c : -1;
            note->odd = hit;
            mbar_arrive(&b.note[cnt % kMeta]);
            mbar_arrive(&b.k_full[st]);
            mbar_arrive(&b.v_full[st]);
          }
          __syncwarp();
        }
      }
      u += w.at.t1 - w.at.t0;
    }
    // copies in flight end before the CTA does (on the ordinary way they were all waited for)
    if (*stop && warp == kLoadWarp && lane == 0)
      for (uint32_t i = cnt > ST ? cnt - ST : 0; i <= cnt; ++i) {
        mbar_wait_bounded(&b.k_full[i % ST], (i / ST) & 1, a.wait_ns);
        mbar_wait_bounded(&b.v_full[i % ST], (i / ST) & 1, a.wait_ns);
      }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// 4-D map of one layer: 64 dims x `tb` tokens of a (token, head, page) cache.
bool encode_map(const KCache& kc, int layer, int tb, CUtensorMap* tm) {
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

int piece(int bs) {  // tokens of a TMA box: the largest divisor of both the block and the tile
  int a = bs, b = kTK;
  while (b) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

template <int D>
cudaError_t go(const AttnArgs& a, cudaStream_t s) {
  CUtensorMap tk, tv;
  const int tb = piece(a.kc.bs);
  if (!encode_map(a.kc, a.layer, tb, &tk) || !encode_map(a.vc, a.layer, tb, &tv)) return cudaErrorNotSupported;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<D><<<a.grid, kThreads, Cfg<D>::kSmem, s>>>(tk, tv, a, tb);
  return cudaGetLastError();
}

}  // namespace

bool attn_tc_suits(const KCache& kc) {
  if (kc.dtype != 1 || (kc.D != 64 && kc.D != 128) || kc.bs % 8 != 0) return false;
  const long long ext[3] = {kc.bs, kc.H, kc.num_pages}, st[3] = {kc.sT, kc.sH, kc.sP};
  for (int i = 0; i < 3; ++i)
    if (ext[i] > 1 && (st[i] < 8 || st[i] * 2 >= (1ll << 40))) return false;
  return true;
}

AttnPlan attn_tc_plan() { return AttnPlan{AttnPlan::kTc, 256, kTK, sm_count()}; }

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) {
  return a.kc.D == 64 ? go<64>(a, s) : go<128>(a, s);
}

}  // namespace kk
