// kk_tree_attn on bf16 caches with many query rows per KV head (a draft tree,
// a piece of a prompt): bound by the tensor cores and the exponentials.
//
// One CTA per SM with two streams, A and B, each a 128-row tile with its own
// accumulator O (D columns of TMEM) and two score buffers S of 64 tokens. Warps
// 0-3 are A's softmax, warps 4-7 B's (a thread owns a row), warp 8 issues A's
// MMAs (tcgen05) and warp 9 B's, warp 10 loads:
//   S_x = Q_x K^T    both operands in shared memory
//   P_x = exp2(S_x * c - m_x)  written over S_x as bf16, the A operand
//   O_x += P_x V     P from TMEM, V from shared memory as it lies (MN-major)
// MMAs of one thread run in order, so the scores two steps on follow P_x V into
// its buffer at once, and the softmax of the next step finds its scores ready.
// The maximum a row's weights are taken against moves only when the true one has
// risen past it by 2^8: until then the weights stay below 2^8, which costs bf16
// nothing, and O need not be rescaled.
//
// An item is a pair of row tiles (both streams take every token) or, for the
// last tile of an odd number, a single one (A takes the first 64 tokens of every
// 128-token tile, B the others, and they leave two partial results): either way
// both streams are busy, every tile is read by both, and a unit of work (one
// tile of a pair, two of a single) is four steps of 64 tokens.
//
// Full tiles of tokens come by TMA (one box per page piece and 64 dims, 128-byte
// swizzle), K of a tile ahead of V of the tile before; where the pages lie is
// looked up a tile ahead. Tiles with a place that holds no token (the end of a
// request, a partial selected block, a bad page) and tiles of drafted nodes are
// copied by the loader's lanes, zeros for what is not there: a weight of zero
// must not meet what such a place holds.
//
// Measured, D = 128, groups of 7: 8 requests of 32768 tokens and 64 nodes 214 us,
// 1.12 PF/s (36 nodes 1.01, groups of 8 and 64 nodes 1.25: whole row tiles);
// lengths from half of that up and 32 to 64 nodes, 164 us for 125 GF and 384 MB.
// The tensor cores are busy 53 % of the time: a step of 64 tokens takes both
// streams about 1900 cycles for 1280 of products, the rest is one thread waiting
// for barriers and issuing 24 instructions; 520 MB come from DRAM (1.28 GB from
// L2), 77 % of a copy's time for them. A call costs about 20 us before its first
// and after its last step (places, queries, the join).
#include <cuda.h>

#include <cfloat>

#include "kk_attn.cuh"
#include "kk_pdl.cuh"
#include "kk_tiles.cuh"

namespace kk {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kLoadWarp = 10;
constexpr int kTK = 128;
constexpr int kMeta = 8;  // ring of per-tile notes from the loader to the softmax warps
// Ring of per-item notes of drafted Values, more than the stages of V: with items of
// one tile, V of the item VS items on needs only this item's last product, which is also
// what lets its notes be read; V of the one after that waits for the read (o_empty).
constexpr int kOdd = 8;
constexpr int kTmemCols = 512;
constexpr float kRise = 8.f;

// Notes on a tile for the softmax warps: which places hold a token, and the
// drafted tile it is (-1: cached tokens).
struct TileNote {
  uint32_t live[4];
  int draft;
};

template <int D>
struct Cfg {
  static constexpr int NC = D / 64;           // 64-dim chunks
  static constexpr int KS = D == 64 ? 4 : 3;  // stages of K
  static constexpr int VS = D == 64 ? 4 : 2;  // stages of V
  static constexpr int kChunk = 128 * 128;    // bytes of 64 dims of 128 rows
  static constexpr int kTile = NC * kChunk;
  static constexpr int kSmem = (2 + KS + VS) * kTile + 1024;
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2][2], p_full[2][2];  // [stream][buffer]
  uint64_t pv_done[2], o_full[2], o_empty[2];
  uint64_t hand_full, hand_empty;  // stream B's part of a single item for stream A
  uint64_t note[kMeta];
  uint64_t drain;
};

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
  constexpr int NC = C::NC, KS = C::KS, VS = C::VS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* s_q = smem;
  unsigned char* s_k = s_q + 2 * C::kTile;
  unsigned char* s_v = s_k + KS * C::kTile;
  __shared__ Bars b;
  __shared__ TileNote s_note[kMeta];
  static_assert(kOdd > VS + 1);
  __shared__ int s_odd[kOdd][kMaxNodes / kTK];  // by item: a drafted tile has a Value that is not finite
  __shared__ long long s_place[kThreads / 32 + 4];
  __shared__ uint32_t s_tmem;
  __shared__ int s_stop;
  volatile int* stop = &s_stop;
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    mbar_init(&b.q_full, 8);
    mbar_init(&b.q_empty, 2);  // both streams
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.k_full[i], 1);
      mbar_init(&b.k_empty[i], 2);  // both streams
      mbar_init(&b.v_full[i], 1);
      mbar_init(&b.v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) {
        mbar_init(&b.s_full[i][j], 1);
        mbar_init(&b.p_full[i][j], 4);
      }
      mbar_init(&b.pv_done[i], 1);
      mbar_init(&b.o_full[i], 1);
      mbar_init(&b.o_empty[i], 4);
    }
    mbar_init(&b.hand_full, 4);
    mbar_init(&b.hand_empty, 4);
    for (int i = 0; i < kMeta; ++i) mbar_init(&b.note[i], 1);
    mbar_init(&b.drain, 2);
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
  const uint32_t tmem = uni(s_tmem);
  int r = pl.r;
  long long base = pl.base;

  if (warp < 8) {
    // ---- softmax: stream x, row `row` of its tile -----------------------------
    const int x = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_at + x * 128, o_at = tmem + lane_at + 256 + x * 128;
    // scale 0 still has to leave hidden places at -inf: the smallest normal number stands for it
    const float c = fmaxf(fabsf(a.scale_log2), FLT_MIN);
    uint32_t seen = 0, notes = 0, items = 0, hands = 0;  // steps, tiles, items; singles handed over
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      const Work w = work_at(a, pl, u, &r, &base);
      const bool single = uni((int)w.at.single);
      const int tiles = uni(w.tiles);
      if (tid == 0) note_cut(a, blockIdx.x, r, w.at, u == pl.u0);
      __syncwarp();
      const int sub = single ? 0 : x;  // row tile of the stream
      const int steps = single ? tiles : 2 * tiles;
      const int rows = uni(w.rows) - sub * 128;
      const bool busy = (warp & 3) * 32 < rows;  // this warp has rows at all
      const int qrow = w.row0 + sub * 128 + row;
      const int node = min(qrow / a.G, w.rq.n - 1);
      // The stream's queries, a row a thread (a single item's stream B reads A's).
      // A negative scale turns their signs; rows that do not exist are zero.
      if (items > 0) {
        alive = warp_wait(&b.q_empty, (items - 1) & 1, a, stop);
        if (!alive) break;
      }
      if (!single || x == 0) {
        const bool real = row < rows;
        const uint16_t* qp = static_cast<const uint16_t*>(a.q);
        if (real) qp += (w.rq.node0 + qrow / a.G) * a.q_sn + (long long)(w.at.h * a.G + qrow % a.G) * a.q_sh;
        const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
          uint4 y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            y[e] = real ? *reinterpret_cast<const uint4*>(qp + (c0 + e) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(s_q + sub * C::kTile + (c0 / 8) * C::kChunk + row * 128 +
                                      ((e ^ (row & 7)) << 4)) =
                make_uint4(y[e].x ^ flip, y[e].y ^ flip, y[e].z ^ flip, y[e].w ^ flip);
        }
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&b.q_full);
      __syncwarp();
      float m_ref = -INFINITY, l = 0.f;  // in units of S
      uint32_t dtile = 0;                // drafted tiles taken
      for (int i = 0; i < steps; ++i, ++seen) {
        const uint32_t no = notes + (single ? i : i >> 1);
        const int half = single ? x : i & 1;  // 64 tokens of the tile
        const TileNote* note = &s_note[no % kMeta];
        const uint32_t buf = seen & 1, sp = s_at + buf * 64;
        alive = warp_wait(&b.note[no % kMeta], (no / kMeta) & 1, a, stop) &&
                warp_wait(&b.s_full[x][buf], (seen >> 1) & 1, a, stop);
        if (!alive) break;
        tc_fence_after();
        if (busy) {
          uint32_t s[2][32];
          tmem_ld32(sp, s[0]);
          tmem_ld32(sp + 32, s[1]);
          uint32_t live[2] = {note->live[half * 2], note->live[half * 2 + 1]};
          const int draft = note->draft;
          if (draft >= 0) {
            dtile |= 1u << draft;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int word = draft * 4 + half * 2 + k, j0 = word * 32;
              uint32_t see = 0xFFFFFFFFu;
              if (!a.mask)
                see = node < j0 ? 0u : node - j0 >= 31 ? 0xFFFFFFFFu : (2u << (node - j0)) - 1u;
              else if (word < a.mask_words)
                see = a.mask[(long long)(w.rq.node0 + node) * a.mask_words + word];
              live[k] &= see;
            }
          }
          __syncwarp();
          tmem_wait_ld();
          if ((live[0] & live[1]) != 0xFFFFFFFFu) {
            // selected, whatever a hidden place holds
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!((live[k] >> e) & 1u)) s[k][e] = 0xFF800000u;
          }
          __syncwarp();
          float mx[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mx[k] = __uint_as_float(s[k >> 1][(k & 1) * 16]);
#pragma unroll
            for (int e = 1; e < 16; ++e) mx[k] = fmaxf(mx[k], __uint_as_float(s[k >> 1][(k & 1) * 16 + e]));
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
            __syncwarp();
            if (!first) {
              // every product into O so far (this stream's step before) has to be in
              if (!warp_wait(&b.pv_done[x], (seen - 1) & 1, a, stop)) al = 0.f;  // given up: the result is void
              tc_fence_after();
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
          uint32_t p[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2(__uint_as_float(s[e / 16][(2 * e) % 32]) * c - mc);
            const float p1 = ex2(__uint_as_float(s[e / 16][(2 * e + 1) % 32]) * c - mc);
            sum[e & 3] += p0 + p1;
            p[e] = pack_bf16(p0, p1);  // the weights' one rounding
          }
          tmem_st32(sp, p);
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.p_full[x][buf]);
        __syncwarp();
      }
      notes += tiles;
      // ---- the item's end: O and the row's maximum and sum
      if (alive) alive = warp_wait(&b.o_full[x], items & 1, a, stop);
      if (!alive) break;
      tc_fence_after();
      uint32_t odd = 0;
      for (int d = 0; d < kMaxNodes / kTK; ++d)
        if ((dtile >> d) & 1u) odd |= s_odd[items % kOdd][d] ? 1u << d : 0u;
      // An item that is this CTA's alone is written out here; of a single one,
      // stream B first hands its part to stream A through the CTA's third slot.
      const bool whole = w.at.t0 == 0 && w.at.t1 == w.at.units;
      const bool give = whole && single && x == 1, take = whole && single && x == 0;
      if (give && hands > 0) alive = warp_wait(&b.hand_empty, (hands - 1) & 1, a, stop);
      if (take) alive = warp_wait(&b.hand_full, hands & 1, a, stop);
      if (!alive) break;
      const bool mine = row < rows;
      const int prow = x * 128 + row;  // row of the partial slot (both streams of a single item leave one)
      float* part = partial_slot(a, blockIdx.x, whole ? 2 : u == pl.u0 ? 0 : 1, 256, D);
      const long long at = (long long)(w.rq.node0 + qrow / a.G) * a.Hq + w.at.h * a.G + qrow % a.G;
      float m2 = m_ref == -INFINITY ? -INFINITY : m_ref * c;
      float fa = 1.f, fb = 0.f;  // factors of this stream's and (take) the other's part
      if (take && mine) {
        const float mb = part[256 * D + 128 + row], lb = part[256 * D + 256 + 128 + row];
        const float mm = fmaxf(m2, mb), ref = mm == -INFINITY ? 0.f : mm;
        fa = ex2(m2 - ref);
        fb = ex2(mb - ref);
        l = l * fa + lb * fb;
        m2 = mm;
      }
      const float inv = row_inv(l);
      __syncwarp();
      if (busy) {
#pragma unroll 1
        for (int k = 0; k < D / 32; ++k) {
          uint32_t o[32];
          tmem_ld32(o_at + k * 32, o);
          tmem_wait_ld();
          if (mine) {
            // Drafted Values that are not finite, for the nodes that see them; of a single
            // item each stream's own half, since the other's may weigh nothing in the join.
            if (odd) {
              for (int j = 0; j < w.rq.n; ++j) {
                if (single && (j / 64 & 1) != x) continue;
                if (!((odd >> (j / kTK)) & 1u) || !sees(a, w.rq, node, j)) continue;
                const uint16_t* v = static_cast<const uint16_t*>(a.dv) + (w.rq.node0 + j) * a.dv_sn + w.at.h * a.dv_sh;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const uint32_t y = v[k * 32 + e];
                  if ((y & 0x7F80u) == 0x7F80u)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(y << 16));
                }
              }
            }
            if (take) {
              const float4* other = reinterpret_cast<const float4*>(part) + k * 8 * 256 + 128 + row;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 y = other[e * 256];
                o[e * 4] = __float_as_uint(__uint_as_float(o[e * 4]) * fa + y.x * fb);
                o[e * 4 + 1] = __float_as_uint(__uint_as_float(o[e * 4 + 1]) * fa + y.y * fb);
                o[e * 4 + 2] = __float_as_uint(__uint_as_float(o[e * 4 + 2]) * fa + y.z * fb);
                o[e * 4 + 3] = __float_as_uint(__uint_as_float(o[e * 4 + 3]) * fa + y.w * fb);
              }
            }
            if (whole && !give) {
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
              // four values of every row lie together: a warp's stores are contiguous
              uint4* out = reinterpret_cast<uint4*>(part) + k * 8 * 256 + prow;
#pragma unroll
              for (int e = 0; e < 8; ++e) out[e * 256] = make_uint4(o[e * 4], o[e * 4 + 1], o[e * 4 + 2], o[e * 4 + 3]);
            }
          }
          __syncwarp();
        }
        if (mine) {
          if (whole && !give) {
            if (a.lse) a.lse[at] = row_lse(m2, l);
          } else {
            part[256 * D + prow] = m2;
            part[256 * D + 256 + prow] = l;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b.o_empty[x]);
        if (give) mbar_arrive(&b.hand_full);
        if (take) mbar_arrive(&b.hand_empty);
      }
      __syncwarp();
      ++items;
      hands += give || take;
      u += w.at.t1 - w.at.t0;
    }
  } else if (warp < kLoadWarp) {
    // ---- MMAs of stream x: the warp stays together and one lane issues ---------
    // (one warp for both streams left the tensor cores idle half the time: waits,
    // commits and the issue itself take longer than 12 products of this size)
    constexpr uint32_t idqk = idesc_bf16_f32(128, 64), idpv = idesc_bf16_f32(128, D) | kIdescBMajorMN;
    const int x = warp - kMmaWarp;
    const uint64_t dq = desc_kmajor_sw128(smem_u32(s_q)), dk = desc_kmajor_sw128(smem_u32(s_k)),
                   dv = desc_mnmajor_sw128(smem_u32(s_v), C::kChunk);
    const uint32_t hi_k = (uint32_t)(dq >> 32), hi_v = (uint32_t)(dv >> 32);
    const uint32_t s_of = tmem + x * 128, o_to = tmem + 256 + x * 128;
    uint32_t cnt = 0, items = 0, qs = 0, ps = 0;  // tiles and items before; steps
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      const Work w = work_at(a, pl, u, &r, &base);
      const bool single = uni((int)w.at.single);
      const int tiles = uni(w.tiles);
      cnt = uni(cnt);
      items = uni(items);
      qs = uni(qs);
      ps = uni(ps);
      const int steps = single ? tiles : 2 * tiles;
      const uint32_t q0 = (uint32_t)dq + ((single ? 0 : x) * C::kTile >> 4);
      alive = warp_wait(&b.q_full, items & 1, a, stop);
      if (!alive) break;
      // scores of step j, 64 tokens; a tile is let go behind its last step
      auto qk = [&](int j) {
        const uint32_t no = cnt + (single ? j : j >> 1), st = no % KS;
        const int half = single ? x : j & 1;
        if ((single || !half) && !warp_wait(&b.k_full[st], (no / KS) & 1, a, stop)) return false;
        tc_fence_after();
        const uint32_t buf = qs++ & 1;
        const uint32_t k0 = (uint32_t)dk + ((st * C::kTile + half * (C::kChunk / 2)) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k / 4) * C::kChunk + (k % 4) * 32) >> 4;
            mma_bf16_lo(s_of + buf * 64, q0 + off, k0 + off, hi_k, idqk, k > 0);
          }
          mma_commit(&b.s_full[x][buf]);
          if (single || half) mma_commit(&b.k_empty[st]);
        }
        __syncwarp();
        return true;
      };
      auto pv = [&](int j) {
        const uint32_t no = cnt + (single ? j : j >> 1), st = no % VS;
        const int half = single ? x : j & 1;
        const uint32_t buf = ps & 1;
        if ((single || !half) && !warp_wait(&b.v_full[st], (no / VS) & 1, a, stop)) return false;
        // O is read out before the next item writes it
        if (j == 0 && items > 0 && !warp_wait(&b.o_empty[x], (items - 1) & 1, a, stop)) return false;
        if (!warp_wait(&b.p_full[x][buf], (ps >> 1) & 1, a, stop)) return false;
        ++ps;
        tc_fence_after();
        const uint32_t v0 = (uint32_t)dv + ((st * C::kTile + half * (C::kChunk / 2)) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16_ts_lo(o_to, s_of + buf * 64 + k * 8, v0 + (k * 2048 >> 4), hi_v, idpv, j > 0 || k > 0);
          mma_commit(&b.pv_done[x]);
          if (single || half) mma_commit(&b.v_empty[st]);
          if (j + 1 == steps) mma_commit(&b.o_full[x]);
        }
        __syncwarp();
        return true;
      };
      alive = qk(0) && (steps < 2 || qk(1));
      for (int j = 0; j < steps && alive; ++j) alive = pv(j) && (j + 2 >= steps || qk(j + 2));
      // every score of the item is in, or on its way
      if (elect_one()) mma_commit(&b.q_empty);
      __syncwarp();
      cnt += tiles;
      ++items;
      u += w.at.t1 - w.at.t0;
    }
    // nothing may be in flight when TMEM and shared memory go
    if (elect_one()) mma_commit(&b.drain);
    __syncwarp();
    mbar_wait_bounded(&b.drain, 0, a.wait_ns);
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ---- loader: the warp stays together and one lane issues the copies ------------
    const int npiece = kTK / tb;  // page pieces of a tile
    uint32_t cnt = 0, items = 0, sent[2] = {0, 0};  // tiles and items before; tiles of K and V sent
    const Split split = make_split(pl.total, a.grid);
    const uint32_t skip = blockIdx.x == 0 ? (uint32_t)a.skip_tile : ~0u;
    bool alive = true;
    // Where a tile's pieces lie: a piece is a run of tb tokens in one page (tb
    // divides the block size).
    struct Piece {
      int page, tok, logical;
    };
    // The order of an item's tiles. The first pair of row tiles goes through them
    // in order; where the others stand in their CTA's time they take the tile that
    // CTAs of the first pair have in hand then (a single, which does two tiles a
    // unit, those of two CTAs): K and V come from DRAM once, and from L2 for the
    // other row tiles (with every CTA in its own order the 64-node batch read 654 MB,
    // in this one 520; once each would be 384).
    int rot = 0, half = 0;  // rotation; tiles of the first of two runs (0: one run)
    auto place = [&](const Work& w, long long u) {
      const int units = w.at.single ? (w.tiles + 1) / 2 : w.tiles;
      half = w.at.single ? units : 0;
      rot = 0;
      if (w.at.mt > 0) {
        const long long ref = base + item_of(w.rq, w.at.h, 0).start + w.first;
        int range;
        const int d = (int)(u - pl.u0) - split_time(split, ref, &range);
        rot = d < 0 ? d + range : d;
        if (rot >= units || rot < 0) rot = 0;
      }
      rot = uni(rot);
      half = uni(half);
    };
    auto tile_of = [&](const Work& w, int i) {
      if (half == 0) {
        const int x = i + rot;
        return w.first + (x < w.tiles ? x : x - w.tiles);
      }
      // units j = rot, rot + 1, ...: tiles j and half + j; of an odd number, unit
      // half - 1 has no second tile
      if ((w.tiles & 1) && i > 2 * (half - 1 - rot)) ++i;
      int j = (i >> 1) + rot;
      if (j >= half) j -= half;
      return w.first + (i & 1) * half + j;
    };
    // What the tables say of a tile's pieces, read a tile ahead and not looked at
    // before the tile's turn, so that the loop does not wait for it.
    auto look = [&](const Work& w, int i) {
      Piece x{-1, 0, 0};
      const int t = tile_of(w, i), v = t * kTK + lane * tb;
      if (i < w.tiles && t < w.rq.tiles_c && lane < npiece && v + tb <= w.rq.ctx) {
        const int bk = (unsigned)v / (unsigned)a.kc.bs;
        x.tok = v - bk * a.kc.bs;
        if (a.sel_pages) {
          const long long at = (long long)w.r * a.selK + bk;
          x.logical = a.sel_logical[at];
          x.page = a.sel_pages[at];
        } else {
          x.page = a.bt.pages[w.rq.off + bk];
        }
      }
      __syncwarp();
      return x;
    };
    // Whether all of the tile's pieces hold tokens only.
    auto all_full = [&](const Work& w, const Piece& x) {
      bool ok = x.page >= 0 && x.page < a.kc.num_pages;
      if (a.sel_pages) ok = ok && x.logical >= 0 && (long long)x.logical * a.kc.bs + x.tok + tb <= w.rq.T;
      return __all_sync(kFull, ok || lane >= npiece);
    };
    // K (or V) of tile i of the item into its stage
    auto load = [&](const Work& w, int i, const Piece& pc, const bool val) {
      const int h = uni(w.at.h), t = tile_of(w, i);
      const uint32_t no = cnt + i, ns = val ? VS : KS, st = no % ns;
      TileNote* note = &s_note[no % kMeta];
      uint64_t *noted = &b.note[no % kMeta], *bar = val ? &b.v_full[st] : &b.k_full[st];
      unsigned char* dst = (val ? s_v : s_k) + st * C::kTile;
      if (!warp_wait(val ? &b.v_empty[st] : &b.k_empty[st], ((no / ns) & 1) ^ 1, a, stop)) return false;
      sent[val] = no + 1;
      if (t < w.rq.tiles_c && all_full(w, pc)) {
        if (elect_one()) {
          if (!val) {
            note->live[0] = note->live[1] = note->live[2] = note->live[3] = 0xFFFFFFFFu;
            note->draft = -1;
            mbar_arrive(noted);
          }
          mbar_arrive_expect_tx(bar, C::kTile + (!val && no == skip ? 16 : 0));
        }
        __syncwarp();
        for (int k = 0; k < npiece; ++k) {
          const int page = __shfl_sync(kFull, pc.page, k), tok = __shfl_sync(kFull, pc.tok, k);
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              tma_load_4d(dst + c * C::kChunk + k * tb * 128, val ? &tmv : &tmk, c * 64, tok, h, page, bar);
          }
          __syncwarp();
        }
        return true;
      }
      // copied, a row a lane, all copies in flight at once
      const bool draft = t >= w.rq.tiles_c;
      uint32_t live[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int m = k * 32 + lane, n = (t - w.rq.tiles_c) * kTK + m;
        const char* p = nullptr;
        TokenAt at;
        if (!draft && token_at(a, w.r, w.rq, t * kTK + m, true, &at)) {
          const KCache& kc = val ? a.vc : a.kc;
          p = static_cast<const char*>(kc.base) + (a.layer * kc.sL + at.page * kc.sP + h * kc.sH + at.tok * kc.sT) * 2;
        } else if (draft && a.dk && n < w.rq.n) {
          p = val ? static_cast<const char*>(a.dv) + ((w.rq.node0 + n) * a.dv_sn + h * a.dv_sh) * 2
                  : static_cast<const char*>(a.dk) + ((w.rq.node0 + n) * a.dk_sn + h * a.dk_sh) * 2;
        }
        const bool real = p != nullptr;
        live[k] = __ballot_sync(kFull, real);
        if (!real) p = static_cast<const char*>(a.q);
        const uint32_t to = smem_u32(dst) + m * 128;
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
          cp_async16(to + (j / 8) * C::kChunk + (((j & 7) ^ (m & 7)) << 4), p + (real ? j * 16 : 0), real);
      }
      cp_wait_all();
      bool hit = false;
      if (draft && val) {
        // a draft's Value that is not finite is added back at the end, to the nodes that see it
#pragma unroll 1
        for (int k = 0; k < 4 * (D / 8); ++k) {
          uint4* y = reinterpret_cast<uint4*>(dst + ((k & 3) * 32 + lane) * 128 + (k / 32) * C::kChunk +
                                              ((k >> 2 & 7) << 4));
          uint4 z = *y;
          if (drop_nonfinite(&z)) {
            *y = z;
            hit = true;
          }
        }
      }
      fence_async_smem();
      hit = __any_sync(kFull, hit);
      if (lane == 0) {
        if (val) {
          if (draft) s_odd[items % kOdd][t - w.rq.tiles_c] = hit;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) note->live[k] = live[k];
          note->draft = draft ? t - w.rq.tiles_c : -1;
          mbar_arrive(noted);
        }
        mbar_arrive(bar);
      }
      __syncwarp();
      return true;
    };
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      const Work w = work_at(a, pl, u, &r, &base);
      const int tiles = uni(w.tiles);
      place(w, u);
      Piece last = look(w, 0), cur = last, next = look(w, 1);
      for (int i = 0; i <= tiles && alive; ++i) {  // K of tile i, V of the tile before
        if (i < tiles) alive = load(w, i, cur, false);
        if (i > 0 && alive) alive = load(w, i - 1, last, true);
        last = cur;
        cur = next;
        next = look(w, i + 2);
      }
      cnt += tiles;
      ++items;
      u += w.at.t1 - w.at.t0;
    }
    // Copies in flight end before the CTA does. All of them were waited for unless
    // another role gives up, which it may do after this one has sent its last.
    if (lane == 0) {
      for (uint32_t i = sent[0] > KS ? sent[0] - KS : 0; i < sent[0]; ++i)
        mbar_wait_bounded(&b.k_full[i % KS], (i / KS) & 1, a.wait_ns);
      for (uint32_t i = sent[1] > VS ? sent[1] - VS : 0; i < sent[1]; ++i)
        mbar_wait_bounded(&b.v_full[i % VS], (i / VS) & 1, a.wait_ns);
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

template <int D>
cudaError_t go(AttnArgs a, cudaStream_t s) {
  CUtensorMap tk, tv;
  const int tb = tile_piece(a.kc.bs, kTK);
  if (!encode_tile_map(a.kc, a.layer, tb, &tk) || !encode_tile_map(a.vc, a.layer, tb, &tv)) return cudaErrorNotSupported;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  a.skip_tile = take_skip_tile();
  attn_tc_kernel<D><<<a.grid, kThreads, Cfg<D>::kSmem, s>>>(tk, tv, a, tb);
  return cudaGetLastError();
}

}  // namespace

bool attn_tc_suits(const KCache& kc) { return (kc.D == 64 || kc.D == 128) && tile_layout_suits(kc); }

AttnPlan attn_tc_plan() { return AttnPlan{AttnPlan::kTc, 256, kTK, sm_count()}; }

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s) {
  return a.kc.D == 64 ? go<64>(a, s) : go<128>(a, s);
}

}  // namespace kk
