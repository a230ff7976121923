// kk_attn_mass on bf16 caches: S^T = K Q^T on the tensor cores, a token a TMEM
// lane and a query row a column, so a token's sum over the rows stays in one
// thread. Bound by K's bytes for a decode token's rows, by the exponentials for
// many rows.
//
// Warps 0-3 and 4-7 are two epilogue groups that take alternate token tiles of
// 128; warp 8 issues the MMAs (128 tokens x up to 128 rows a job), warp 9 loads
// K by TMA into a ring. Each group has two score buffers of 128 columns: it sums
// one while the tensor cores fill the other, and the other group's meanwhile.
// The rows that count (weight not 0, lse not -inf) of a (request, KV head) are
// listed and their queries kept in shared memory for all its tiles, so nodes
// that were rejected cost nothing. A place that holds no token only spoils its
// own lane, which stores nothing.
//
// Measured, D = 128, groups of 7: one node, 8 requests of up to 32768 tokens (195
// MB) 41.4 us, 4.7 TB/s, about 12 of it before and after the stream of tiles (four
// times the tokens run at 6.3 TB/s); up to 64 causal nodes, 2 x 16384 tokens (9.7 GF,
// 38 M exponentials) 35 us, half of it start and end too: 2 x 65536 tokens and 64
// nodes take 99 us, 610 TF/s, two thirds of what 16 exponentials a clock and SM
// allow. Twice the epilogue warps, which halved a tile's rows, were slower (39 us).
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "kk_tiles.cuh"

namespace kk {
namespace {

constexpr int kThreads = 320;
constexpr int kEpi = 256;  // epilogue threads
constexpr int kMmaWarp = 8, kLoadWarp = 9;
constexpr int kTK = 128;
constexpr int kCols = 128;  // rows of a job
constexpr int kMaxRows = 1024;
constexpr int kStagesMax = 8;
constexpr int kSmemMax = 227 * 1024 - 1024 - 20 * 1024;  // next to the row list and the barriers

struct __align__(8) RowInfo {
  float w;  // weight
  int len;  // tokens the row sees
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[kStagesMax], k_empty[kStagesMax];
  uint64_t s_full[4], s_empty[4];
  uint64_t drain;
};

// kFew: at most 8 rows.
template <int D, bool kFew>
__global__ void __launch_bounds__(kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap tmk, const AttnArgs a, const int tb, const int row_begin,
                   const int row_end, const int rows_pad, const int NS) {
  constexpr int NC = D / 64;
  constexpr int kChunk = 128 * 128;  // bytes of 64 dims of a token tile
  constexpr int kTile = NC * kChunk;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* s_k = smem;
  unsigned char* s_q = s_k + NS * kTile;  // [64-dim chunk][rows_pad][128 bytes], 128-byte swizzle
  __shared__ Bars b;
  // Rows up to a whole group of 32 see nothing.
  __shared__ __align__(16) float s_b[kMaxRows + 32];  // -lse in the log2 domain
  __shared__ __align__(16) RowInfo s_row[kMaxRows + 32];
  __shared__ int s_least;  // tokens that every row sees, with a weight of 1 (0 where there is another)
  __shared__ long long s_place[kThreads / 32 + 4];
  __shared__ int s_cnt[kEpi / 32];
  __shared__ int s_rows;  // rows of the item that count
  __shared__ uint32_t s_tmem;
  __shared__ int s_stop;
  volatile int* stop = &s_stop;
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    mbar_init(&b.q_full, kEpi / 32);
    mbar_init(&b.q_empty, 1);
    for (int i = 0; i < kStagesMax; ++i) {
      mbar_init(&b.k_full[i], 1);
      mbar_init(&b.k_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&b.s_full[i], 1);
      mbar_init(&b.s_empty[i], 4);
    }
    mbar_init(&b.drain, 1);
    s_stop = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  const AttnPlace pl = find_place<kThreads>(a, blockIdx.x, 1, kTK, s_place, tid);  // holds block barriers
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, s_tmem, 0);
  int r = pl.r;
  long long base = pl.base;
  // The CTA's next item: (request, KV head) and its token tiles [t0, t1).
  auto next_item = [&](long long u, AttnReq* rq, ItemAt* at) {
    for (;;) {
      *rq = load_req(a, r, 1, kTK, false);
      const long long n = req_units(a, *rq);
      if (u < base + n) break;
      base += n;
      ++r;
    }
    *at = item_at(*rq, u - base);
    at->t1 = (int)min((long long)at->units, at->t0 + (pl.u1 - u));
  };

  if (warp < 8) {
    // ---- epilogue groups: token `row` of every other tile --------------------------
    const int g = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_at = (uint32_t)((warp & 3) * 32) << 16;
    uint32_t jobs = 0, items = 0;  // of this group; of the CTA
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1;) {
      AttnReq rq;
      ItemAt at;
      next_item(u, &rq, &at);
      const int h = at.h;
      // The MMAs of the item before are through and every warp is past its scores:
      // its queries and rows may go.
      if (alive && items > 0) alive = warp_wait(&b.q_empty, (items - 1) & 1, a, stop);
      ++items;
      alive = !named_sync_or(1, kEpi, !alive);
      if (!alive) break;
      if (tid == 0) s_least = 0x7fffffff;
      const int r0 = min(row_begin, rq.n * a.G), r1 = min(row_end, rq.n * a.G);
      constexpr int NX = kMaxRows / kEpi;  // rows a thread looks at
      float rw[NX], rl[NX];
      int rn[NX], len[NX];
#pragma unroll
      for (int y = 0; y < NX; ++y) {
        const int x = r0 + y * kEpi + tid;
        rw[y] = 0.f;
        if (x < r1) {
          rn[y] = rq.node0 + x / a.G;
          rw[y] = a.row_w ? a.row_w[rn[y]] : 1.f;
          rl[y] = a.lse[(long long)rn[y] * a.Hq + h * a.G + x % a.G];
          len[y] = a.row_lens ? a.row_lens[rn[y]] : rq.T;
        }
      }
      int have = 0;
#pragma unroll
      for (int y = 0; y < NX; ++y) {  // list the rows that count, in order
        if (r0 + y * kEpi >= r1) break;
        const bool on = rw[y] != 0.f && rl[y] != -INFINITY;
        const uint32_t m = __ballot_sync(kFull, on);
        if (lane == 0) s_cnt[warp] = __popc(m);
        named_sync(1, kEpi);
        int before = have, all = have;
        for (int k = 0; k < kEpi / 32; ++k) {
          if (k < warp) before += s_cnt[k];
          all += s_cnt[k];
        }
        if (on) {
          const int i = before + __popc(m & ((1u << lane) - 1u)), x = r0 + y * kEpi + tid;
          s_b[i] = -rl[y] * 1.44269504088896341f;
          s_row[i] = RowInfo{rw[y], len[y]};
          atomicMin(&s_least, rw[y] == 1.f ? len[y] : 0);
          const uint16_t* q =
              static_cast<const uint16_t*>(a.q) + rn[y] * a.q_sn + (long long)(h * a.G + x % a.G) * a.q_sh;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            cp_async16(smem_u32(s_q) + (c / 8) * rows_pad * 128 + i * 128 + (((c & 7) ^ (i & 7)) << 4), q + c * 8, true);
        }
        have = all;
        named_sync(1, kEpi);
      }
      if (tid < 32) {
        s_b[have + tid] = 0.f;
        s_row[have + tid] = RowInfo{0.f, 0};
      }
      if (tid == 0) s_rows = have;
      cp_wait_all();
      fence_async_smem();
      named_sync(1, kEpi);
      if (lane == 0) mbar_arrive(&b.q_full);
      __syncwarp();
      const int n = __shfl_sync(kFull, s_rows, 0);
      const int nch = (n + kCols - 1) / kCols;
      const int old = a.old_lens ? a.old_lens[r] : rq.T;
      const int least = __shfl_sync(kFull, s_least, 0);
      // A tile's token is looked up two tiles ahead and what it had is read one
      // tile ahead: two dependent loads that would else wait behind every tile.
      auto find = [&](int t) {  // the token's weight, or -1
        TokenAt tk;
        long long x = -1;
        if (t < at.t1 && token_at(a, r, rq, t * kTK + row, true, &tk))
          x = (((long long)a.layer * a.kc.num_pages + tk.page) * a.kc.H + h) * a.kc.bs + tk.tok;
        __syncwarp();
        return x;
      };
      auto had = [&](int t, long long x) {
        float y = 0.f;
        // a later pass over more rows adds to what the first one wrote
        if (x >= 0 && row_begin > 0)
          y = a.mass_out[x];
        else if (x >= 0 && a.mass_in && t * kTK + row < old)
          y = a.decay * a.mass_in[x];
        __syncwarp();
        return y;
      };
      long long x1 = find(at.t0 + g), x2 = find(at.t0 + g + 2);
      float had1 = had(at.t0 + g, x1);
      for (int t = at.t0 + g; t < at.t1 && alive; t += 2) {
        const int v = t * kTK + row;
        const long long x = x1;
        const float before = had1;
        had1 = had(t + 2, x2);
        x1 = x2;
        x2 = find(t + 4);
        float acc = 0.f;
        for (int c = 0; c < nch; ++c, ++jobs) {
          const uint32_t buf = g + 2 * (jobs & 1);
          alive = warp_wait(&b.s_full[buf], (jobs >> 1) & 1, a, stop);
          if (!alive) break;
          tc_fence_after();
          const int cols = min(kCols, n - c * kCols);
          const uint32_t at_col = tmem + lane_at + buf * kCols;
          const float4* rb = reinterpret_cast<const float4*>(s_b + c * kCols);
          const RowInfo* ri = s_row + c * kCols;
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          // What a row's values cost to read bounds this: shared memory gives a
          // clock's worth of a warp 4 bytes a lane, whoever shares them. So where
          // every row sees the whole tile with weight 1, only its lse is read.
          auto sum = [&](auto count, const uint32_t* s, int k) {
            constexpr int N = decltype(count)::value;
            if (N > 8 && (t + 1) * kTK <= least && k + N <= cols) {
#pragma unroll
              for (int e = 0; e < N; e += 4) {
                const float4 y = rb[(k + e) / 4];
                part[0] += ex2(__uint_as_float(s[e]) * a.scale_log2 + y.x);
                part[1] += ex2(__uint_as_float(s[e + 1]) * a.scale_log2 + y.y);
                part[2] += ex2(__uint_as_float(s[e + 2]) * a.scale_log2 + y.z);
                part[3] += ex2(__uint_as_float(s[e + 3]) * a.scale_log2 + y.w);
              }
              return;
            }
#pragma unroll
            for (int e = 0; e < N; e += 4) {
              const float4 b4 = rb[(k + e) / 4];
              const float bb[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const RowInfo y = ri[k + e + j];
                const float p = ex2(__uint_as_float(s[e + j]) * a.scale_log2 + bb[j]);
                part[j] += y.w * (v < y.len ? p : 0.f);  // selected: a hidden place may hold anything
              }
            }
          };
          if (kFew || cols <= 8) {
            uint32_t s0[8];
            tmem_ld8(at_col, s0);
            tmem_wait_ld();
            sum(std::integral_constant<int, 8>{}, s0, 0);
          } else if constexpr (!kFew) {
            uint32_t s0[32], s1[32];
            tmem_ld32(at_col, s0);
#pragma unroll 1
            for (int k = 0; k < cols; k += 64) {  // the next columns come while these are summed
              tmem_wait_ld();
              if (k + 32 < cols) tmem_ld32(at_col + k + 32, s1);
              sum(std::integral_constant<int, 32>{}, s0, k);
              if (k + 32 < cols) {
                tmem_wait_ld();
                if (k + 64 < cols) tmem_ld32(at_col + k + 64, s0);
                sum(std::integral_constant<int, 32>{}, s1, k + 32);
              }
            }
          }
          acc += (part[0] + part[1]) + (part[2] + part[3]);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&b.s_empty[buf]);
          __syncwarp();
        }
        if (x >= 0 && alive) a.mass_out[x] = before + acc;
        __syncwarp();
      }
      u += at.t1 - at.t0;
    }
  } else if (warp == kMmaWarp) {
    // ---- MMAs: the warp stays together and one lane issues -------------------------
    const uint64_t dk = desc_kmajor_sw128(smem_u32(s_k)), dq = desc_kmajor_sw128(smem_u32(s_q));
    const uint32_t hi = (uint32_t)(dk >> 32);
    uint32_t cnt = 0, items = 0, jobs[2] = {0, 0};
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      AttnReq rq;
      ItemAt at;
      next_item(u, &rq, &at);
      const int tiles = __shfl_sync(kFull, at.t1 - at.t0, 0);
      alive = warp_wait(&b.q_full, items & 1, a, stop);
      if (!alive) break;
      const int n = __shfl_sync(kFull, s_rows, 0), nch = (n + kCols - 1) / kCols;
      for (int i = 0; i < tiles && alive; i += 2) {
        const int two = min(2, tiles - i);
        for (int c = 0; c < max(nch, 1) && alive; ++c) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (g >= two || !alive) continue;
            const uint32_t no = cnt + i + g, st = no % NS;
            if (c == 0) alive = warp_wait(&b.k_full[st], (no / NS) & 1, a, stop);
            if (!alive) continue;
            if (nch > 0) {
              const uint32_t buf = g + 2 * (jobs[g] & 1);
              alive = warp_wait(&b.s_empty[buf], ((jobs[g] >> 1) & 1) ^ 1, a, stop);
              if (!alive) continue;
              ++jobs[g];
              tc_fence_after();
              const uint32_t id = idesc_bf16_f32(128, (min(kCols, n - c * kCols) + 15) & ~15);
              const uint32_t k0 = (uint32_t)dk + (st * kTile >> 4);
              const uint32_t q0 = (uint32_t)dq + (c * kCols * 128 >> 4), qc = rows_pad * 128 >> 4;
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                  mma_bf16_lo(tmem + buf * kCols, k0 + ((k / 4) * kChunk + (k % 4) * 32 >> 4),
                              q0 + (k / 4) * qc + ((k % 4) * 32 >> 4), hi, id, k > 0);
                mma_commit(&b.s_full[buf]);
                if (c == nch - 1) mma_commit(&b.k_empty[st]);
              }
            } else if (elect_one()) {
              mma_commit(&b.k_empty[st]);  // no row counts: the tile is let go unread
            }
            __syncwarp();
          }
        }
      }
      if (elect_one()) mma_commit(&b.q_empty);
      __syncwarp();
      cnt += tiles;
      ++items;
      u += at.t1 - at.t0;
    }
    // nothing may be in flight when TMEM and shared memory go
    if (elect_one()) mma_commit(&b.drain);
    __syncwarp();
    mbar_wait_bounded(&b.drain, 0, a.wait_ns);
    __syncwarp();
  } else {
    // ---- loader ----------------------------------------------------------------------
    const int npiece = kTK / tb;  // page pieces of a tile
    const uint32_t skip = blockIdx.x == 0 ? (uint32_t)a.skip_tile : ~0u;
    uint32_t cnt = 0, sent = 0;
    bool alive = true;
    for (long long u = pl.u0; u < pl.u1 && alive;) {
      AttnReq rq;
      ItemAt at;
      next_item(u, &rq, &at);
      const int tiles = __shfl_sync(kFull, at.t1 - at.t0, 0), h = __shfl_sync(kFull, at.h, 0);
      // Pieces that begin with a token are loaded (to the end of their page); the
      // rest of the tile keeps what it held. Looked up a tile ahead.
      auto look = [&](int i, TokenAt* x) {
        const bool on = i < tiles && lane < npiece && token_at(a, r, rq, (at.t0 + i) * kTK + lane * tb, false, x);
        __syncwarp();
        return on;
      };
      TokenAt cur, next;
      bool on = look(0, &cur);
      for (int i = 0; i < tiles; ++i) {
        const bool more = look(i + 1, &next);
        const uint32_t no = cnt + i, st = no % NS;
        alive = warp_wait(&b.k_empty[st], ((no / NS) & 1) ^ 1, a, stop);
        if (!alive) break;
        sent = no + 1;
        const uint32_t pieces = __ballot_sync(kFull, on);
        if (elect_one()) mbar_arrive_expect_tx(&b.k_full[st], __popc(pieces) * tb * D * 2 + (no == skip ? 16 : 0));
        __syncwarp();
        for (int k = 0; k < npiece; ++k) {
          const int page = __shfl_sync(kFull, cur.page, k), tok = __shfl_sync(kFull, cur.tok, k);
          if (((pieces >> k) & 1u) && elect_one()) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
              tma_load_4d(s_k + st * kTile + c * kChunk + k * tb * 128, &tmk, c * 64, tok, h, page, &b.k_full[st]);
          }
          __syncwarp();
        }
        cur = next;
        on = more;
      }
      cnt += tiles;
      u += at.t1 - at.t0;
    }
    // Copies in flight end before the CTA does. All of them were waited for unless
    // another role gives up, which it may do after this one has sent its last.
    if (lane == 0)
      for (uint32_t i = sent > (uint32_t)NS ? sent - NS : 0; i < sent; ++i)
        mbar_wait_bounded(&b.k_full[i % NS], (i / NS) & 1, a.wait_ns);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Rows of one pass: as many as leave room for at least two stages of K.
template <int D>
constexpr int max_rows() {
  return std::min(kMaxRows, (kSmemMax - 2 * 128 * D * 2) / (D * 2) / 16 * 16);
}

template <int D>
cudaError_t go(AttnArgs a, cudaStream_t s) {
  CUtensorMap tk;
  const int tb = tile_piece(a.kc.bs, kTK);
  if (!encode_tile_map(a.kc, a.layer, tb, &tk)) return cudaErrorNotSupported;
  a.grid = sm_count();
  const int rows = a.max_nodes * a.G;
  // Without the code of wider jobs a decode token's rows take 41.4 us instead of 42.8 (8 requests of up to 32768
  // tokens), 42.5 instead of 48 with caches flushed: less to fetch, 91 registers instead of 163.
  const auto k = rows <= 8 ? mass_tc_kernel<D, true> : mass_tc_kernel<D, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax + 1024);
  for (int b = 0; b < rows && e == cudaSuccess; b += max_rows<D>()) {
    const int pad = (std::min(rows - b, max_rows<D>()) + 15) & ~15;
    const int ns = std::min(kStagesMax, (kSmemMax - pad * D * 2) / (128 * D * 2));
    const int smem = ns * 128 * D * 2 + pad * D * 2 + 1024;
    a.skip_tile = take_skip_tile();
    k<<<a.grid, kThreads, smem, s>>>(tk, a, tb, b, b + max_rows<D>(), pad, ns);
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace

bool mass_tc_suits(const KCache& kc) { return tile_layout_suits(kc); }

cudaError_t launch_mass_tc(const AttnArgs& a, cudaStream_t s) {
  switch (a.kc.D) {
    case 64: return go<64>(a, s);
    case 128: return go<128>(a, s);
    case 256: return go<256>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace kk
