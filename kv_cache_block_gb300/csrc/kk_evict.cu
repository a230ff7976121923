// Eviction by accumulated attention weight, per (request, layer, KV head):
//  * evict_select_kernel: the first `sinks` tokens, the last `recent` ones and
//    the heaviest of the rest, `keep` in all, in ascending order (equal weights
//    to the lower index, NaN below everything);
//  * evict_move_kernel, evict_compact_kernel: their Keys, Values and weights
//    moved to slots 0 .. keep-1 of new pages, or of the request's own.
// Measured, 896 rows of 8192 bf16 tokens of 128 dims cut to 2048: the selection 41
// us (29 MB read once: bound by instructions, 78 % of the issue slots, and by equal
// weights meeting in one bin of a histogram), the move to new pages 287 us (1.87
// GB, 6.6 TB/s), in place 378.
#include <algorithm>
#include <cmath>

#include "kk_device.cuh"

namespace kk {
namespace {

// ---- selection -------------------------------------------------------------
constexpr int kBins = 2048;
// Weights of a row kept in shared memory (next to the histogram); longer rows
// are read again for each of the five passes.
constexpr int kMaxCached = 48 * 1024;

// Order of a weight as an unsigned integer (larger: heavier): -0 as +0, NaN 0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  return m != m ? 0u : f32_to_ordered(m + 0.f);
}

// One CTA of NT threads per (request, layer, head). The key of the (keep - sinks - recent)-th
// heaviest token of the middle is found digit by digit (11, 11 and 10 bits)
// from histograms in shared memory; then every warp counts the tokens of its
// share above it and equal to it, and, knowing the counts before its own, writes
// its kept tokens in order. Bound by instructions, so keys are taken four at a
// time (and read four at a time where the weights lie so, kVec = 4).
template <int NT, bool kCached, int kVec>
__global__ void __launch_bounds__(NT, 1536 / NT) evict_select_kernel(KCache kc, Table bt, const float* mass,
                                                                      int sinks, int recent, int keep, int* kept,
                                                                      int* new_lens, int* err) {
  extern __shared__ __align__(16) uint32_t s_key[];  // cached: the keys of the request's tokens
  __shared__ __align__(16) uint32_t s_hist[kBins];
  __shared__ uint32_t s_scan[NT / 32];
  __shared__ uint32_t s_digit, s_left;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int h = blockIdx.x % kc.H, l = (blockIdx.x / kc.H) % kc.L, r = blockIdx.x / (kc.H * kc.L);
  const int off = bt.offsets[r], nb = bt.offsets[r + 1] - off, bs = kc.bs;
  int T = bt.seq_lens[r];
  if (T < 0 || T > kMaxTokens || nb < 0 || nb > bt.max_blocks || nb != (int)(((unsigned)T + (unsigned)bs - 1u) / (unsigned)bs)) {
    if (tid == 0) flag_error(err, kErrBadIndex);
    T = 0;
  }
  int* out = kept + (long long)blockIdx.x * keep;
  const int n = min(T, keep);
  if (tid == 0 && l == 0 && h == 0 && new_lens) new_lens[r] = n;
  for (int i = n + tid; i < keep; i += NT) out[i] = -1;
  if (T <= keep) {
    for (int i = tid; i < n; i += NT) out[i] = i;
    return;
  }
  const int m0 = sinks, m1 = T - recent;  // the middle [m0, m1)
  const uint32_t want = (uint32_t)(keep - sinks - recent);
  for (int i = tid; i < sinks; i += NT) out[i] = i;
  for (int i = tid; i < recent; i += NT) out[keep - recent + i] = T - recent + i;
  if (want == 0) return;
  const float* mbase = mass + ((long long)l * kc.num_pages * kc.H + h) * bs;
  const long long page_stride = (long long)kc.H * bs;
  if (kCached) {
    // A thread keeps its place in the block and steps whole blocks: one division
    // in all. U pages are read, then U weights, so that the two dependent loads
    // cost two latencies a round.
    constexpr int U = kVec == 4 ? 4 : 8;
    const int row = bs / kVec;                                  // pieces of a block
    const int per = row < NT ? NT / row : 1;  // blocks a turn
    const int b0 = row < NT ? tid / row : 0, o0 = row < NT ? tid - b0 * row : tid;
    bool bad = false;
    if (b0 < per)
      for (int o = o0; o < row; o += NT)
        for (int b = m0 / bs + b0; b < nb; b += per * U) {
          int page[U];
          float wt[U][kVec];
#pragma unroll
          for (int u = 0; u < U; ++u) page[u] = b + u * per < nb ? bt.pages[off + b + u * per] : 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const bool good = page[u] >= 0 && page[u] < kc.num_pages;
            bad |= !good;
#pragma unroll
            for (int e = 0; e < kVec; ++e) wt[u][e] = NAN;  // a bad page ranks last
            if (b + u * per < nb && good) {
              // past the last token a page may hold anything: its keys are not looked at
              const float* p = mbase + page[u] * page_stride + o * kVec;
              if constexpr (kVec == 4) {
                const float4 x = *reinterpret_cast<const float4*>(p);
                wt[u][0] = x.x;
                wt[u][1] = x.y;
                wt[u][2] = x.z;
                wt[u][3] = x.w;
              } else {
                wt[u][0] = *p;
              }
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (b + u * per >= nb) break;
            uint32_t* to = s_key + (b + u * per) * bs + o * kVec;
            if constexpr (kVec == 4)
              *reinterpret_cast<uint4*>(to) =
                  make_uint4(mass_key(wt[u][0]), mass_key(wt[u][1]), mass_key(wt[u][2]), mass_key(wt[u][3]));
            else
              *to = mass_key(wt[u][0]);
          }
        }
    if (bad) flag_error(err, kErrBadIndex);
    __syncthreads();
  }
  // Keys of tokens 4 v .. 4 v + 3, and which of them are of the middle.
  struct Four {
    uint32_t k[4];
    uint32_t in;
  };
  auto four = [&](int v) {
    Four f;
    const int t = v * 4;
    f.in = 0xFu;
    if (t < m0 || t + 3 >= m1) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e < m0 || t + e >= m1) f.in &= ~(1u << e);
    }
    if (kCached) {
      const uint4 x = *reinterpret_cast<const uint4*>(s_key + t);
      f.k[0] = x.x;
      f.k[1] = x.y;
      f.k[2] = x.z;
      f.k[3] = x.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f.k[e] = 0;
        if (!((f.in >> e) & 1u)) continue;
        const int b = (t + e) / bs, page = bt.pages[off + b];
        if (page < 0 || page >= kc.num_pages)
          flag_error(err, kErrBadIndex);
        else
          f.k[e] = mass_key(mbase[page * page_stride + (t + e - b * bs)]);
      }
    }
    return f;
  };
  const int v0 = m0 / 4, v1 = (m1 + 3) / 4;
  uint32_t prefix = 0, left = want;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, bins = 1 << bits;
    const int up = shift;
    shift -= bits;
    for (int i = tid; i < bins; i += NT) s_hist[i] = 0;
    __syncthreads();
    for (int v = v0 + tid; v < v1; v += NT) {
      const Four f = four(v);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (((f.in >> e) & 1u) && (pass == 0 || (f.k[e] >> up) == prefix))
          atomicAdd(&s_hist[(f.k[e] >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // from the top bin down: the bin in which the `left`-th key lies
    constexpr int PER = kBins / NT;  // a multiple of 4
    uint32_t c[PER], sum = 0;
    const int low = bins - (tid + 1) * PER;  // the thread's bins, low + PER - 1 .. low
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (low >= 0) x = *reinterpret_cast<const uint4*>(&s_hist[low + PER - 4 - i]);
      c[i] = x.w;
      c[i + 1] = x.z;
      c[i + 2] = x.y;
      c[i + 3] = x.x;
      sum += (x.x + x.y) + (x.z + x.w);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[w] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int x = 0; x < w; ++x) before += s_scan[x];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (before < left && left <= before + c[i]) {
        s_digit = (uint32_t)(low + PER - 1 - i);
        s_left = left - before;
      }
      before += c[i];
    }
    __syncthreads();
    prefix = (prefix << bits) | s_digit;
    left = s_left;
    __syncthreads();
  }
  // `prefix` is the threshold key; the first `left` tokens equal to it stay. Counts
  // are kept as (above, equal) halves of 64 bits.
  const int seg = ((v1 - v0 + NT - 1) / NT) * 32;  // a warp's share
  const int a0 = min(v1, v0 + w * seg), a1 = min(v1, a0 + seg);
  __shared__ unsigned long long s_before[NT / 32];
  auto count = [&](const Four& f) {
    unsigned long long c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((f.in >> e) & 1u) c += f.k[e] > prefix ? 1ull : f.k[e] == prefix ? 1ull << 32 : 0ull;
    return c;
  };
  unsigned long long mine = 0;
  for (int v = a0 + lane; v < a1; v += 32) mine += count(four(v));
  const uint32_t gt = __reduce_add_sync(kFull, (uint32_t)mine), eq = __reduce_add_sync(kFull, (uint32_t)(mine >> 32));
  if (lane == 0) s_before[w] = ((unsigned long long)eq << 32) | gt;
  __syncthreads();
  unsigned long long done = 0;  // above and equal before this warp's
  for (int x = 0; x < w; ++x) done += s_before[x];
  for (int b = a0; b < a1; b += 32) {
    const int v = b + lane;
    Four f;
    f.in = 0;
    if (v < a1) f = four(v);
    const unsigned long long c = count(f);
    // a lane holds 4 at most, a warp 128: both counts in one word for the scan
    const uint32_t both = (uint32_t)c | (uint32_t)(c >> 32) << 16;
    uint32_t incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    const uint32_t all = __shfl_sync(kFull, incl, 31), ex = incl - both;
    uint32_t g = (uint32_t)done + (ex & 0xFFFFu), q = (uint32_t)(done >> 32) + (ex >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!((f.in >> e) & 1u)) continue;
      const bool above = f.k[e] > prefix, same = f.k[e] == prefix;
      if (above || (same && q < left)) out[sinks + g + min(q, left)] = v * 4 + e;
      g += above;
      q += same;
    }
    done += ((unsigned long long)(all >> 16) << 32) + (all & 0xFFFFu);
  }
}

// ---- move --------------------------------------------------------------------
struct MoveArgs {
  KCache kc, vc;
  Table bt;
  const int* kept;
  int keep, dst_blocks;
  const float* mass_in;
  float* mass_out;
  const int* dst_pages;  // [R][dst_blocks], or null: the request's own pages
  int* err;
  int items;  // rows of kept tokens: requests x layers x heads
};

// The sizes of the row of kept tokens that block x moves.
struct MoveRow {
  int h, l, r, off, T, n;
  bool ok;
};
__device__ __forceinline__ MoveRow move_row(const MoveArgs& a, int x, bool report) {
  MoveRow m;
  m.h = x % a.kc.H;
  m.l = (x / a.kc.H) % a.kc.L;
  m.r = x / (a.kc.H * a.kc.L);
  m.off = a.bt.offsets[m.r];
  const int nb = a.bt.offsets[m.r + 1] - m.off;
  m.T = a.bt.seq_lens[m.r];
  m.ok = !(m.T < 0 || m.T > kMaxTokens || nb < 0 || nb > a.bt.max_blocks ||
           nb != (int)(((unsigned)m.T + (unsigned)a.kc.bs - 1u) / (unsigned)a.kc.bs));
  if (!m.ok && report) flag_error(a.err, kErrBadIndex);
  m.n = m.ok ? min(m.T, a.keep) : 0;
  return m;
}
// Where slot i of the row comes from and goes to.
struct Move {
  int sp, st, dp, dt;
  bool ok;
};
__device__ __forceinline__ Move move_at(const MoveArgs& a, const MoveRow& m, const int* kept, int i) {
  Move x{0, 0, 0, 0, false};
  if (i >= m.n) return x;
  const int t = kept[i], bs = a.kc.bs;
  if (t < 0 || t >= m.T) {
    flag_error(a.err, kErrBadIndex);
    return x;
  }
  const int sb = t / bs, db = i / bs;
  x.st = t - sb * bs;
  x.dt = i - db * bs;
  x.sp = a.bt.pages[m.off + sb];
  x.dp = a.dst_pages ? a.dst_pages[(long long)m.r * a.dst_blocks + db] : a.bt.pages[m.off + db];
  if (x.sp < 0 || x.sp >= a.kc.num_pages || x.dp < 0 || x.dp >= a.kc.num_pages) {
    flag_error(a.err, kErrBadIndex);
    return x;
  }
  x.ok = true;
  return x;
}
__device__ __forceinline__ long long row_at(const KCache& c, const MoveRow& m, int page, int tok, int es) {
  return (m.l * c.sL + page * c.sP + m.h * c.sH + tok * c.sT) * es;
}
__device__ __forceinline__ uint4 ld16_once(const char* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

constexpr int kMoveThreads = 256;

// To other pages: a warp moves kRows kept tokens. Each lane finds one token's
// places; then P lanes copy a token's row of P 16-byte pieces, the rows' loads
// all in flight before the first store.
template <int P>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveArgs a) {
  constexpr int RI = 32 / P;           // rows of one instruction
  constexpr int kRows = 8 * RI < 32 ? 8 * RI : 32;
  constexpr int U = kRows / RI;        // loads in flight, for K and for V each
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, sub = lane / P, c = lane % P * 16;
  // the rows' first pieces, then their second ones, ... in one dimension of the grid, which has room for all
  const int piece = blockIdx.x / a.items, item = blockIdx.x - piece * a.items;
  const MoveRow m = move_row(a, item, piece == 0 && threadIdx.x == 0);
  const int i0 = (piece * (kMoveThreads / 32) + w) * kRows;
  if (i0 >= m.n) return;
  const int es = a.kc.dtype == 1 ? 2 : 4;
  const Move mv = lane < kRows ? move_at(a, m, a.kept + (long long)item * a.keep, i0 + lane) : Move{0, 0, 0, 0, false};
  const uint32_t ok = __ballot_sync(kFull, mv.ok);
  const bool has_v = a.vc.base != nullptr;
  const long long ks = row_at(a.kc, m, mv.sp, mv.st, es), kd = row_at(a.kc, m, mv.dp, mv.dt, es);
  const long long vs = row_at(a.vc, m, mv.sp, mv.st, es), vd = row_at(a.vc, m, mv.dp, mv.dt, es);
  const long long mi = ((long long)m.l * a.kc.num_pages * a.kc.H + m.h) * a.kc.bs;
  const long long mp = (long long)a.kc.H * a.kc.bs;
  float wt = 0.f;
  if (a.mass_in && mv.ok) wt = a.mass_in[mi + mv.sp * mp + mv.st];
  const char* kb = static_cast<const char*>(a.kc.base);
  const char* vb = static_cast<const char*>(a.vc.base);
  uint4 kx[U], vx[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = u * RI + sub;
    const long long s = __shfl_sync(kFull, ks, row), v = __shfl_sync(kFull, vs, row);
    const bool on = (ok >> row) & 1u;
    kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
    if (on) kx[u] = ld16_once(kb + s + c);
    if (on && has_v) vx[u] = ld16_once(vb + v + c);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int row = u * RI + sub;
    const long long d = __shfl_sync(kFull, kd, row), v = __shfl_sync(kFull, vd, row);
    if ((ok >> row) & 1u) {
      *reinterpret_cast<uint4*>(const_cast<char*>(kb) + d + c) = kx[u];
      if (has_v) *reinterpret_cast<uint4*>(const_cast<char*>(vb) + v + c) = vx[u];
    }
  }
  if (a.mass_in && mv.ok) a.mass_out[mi + mv.dp * mp + mv.dt] = wt;
}

// In place: a cluster per (request, layer, head) takes the slots in chunks. A
// chunk is read whole, by all its CTAs, before any of it is written, and since
// kept[i] >= i its writes never reach a source of a later chunk.
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const MoveArgs a, int P) {
  constexpr int U = 4;
  const int tid = threadIdx.x;
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int x = blockIdx.x / C;
  const MoveRow m = move_row(a, x, rank == 0 && tid == 0);
  const int es = a.kc.dtype == 1 ? 2 : 4;
  const int* kept = a.kept + (long long)x * a.keep;
  const int rows = kMoveThreads / P, per = rows * U * C;  // rows of a turn, of a chunk
  const int c = tid % P * 16, sub = tid / P;
  const char* kb = static_cast<const char*>(a.kc.base);
  const char* vb = static_cast<const char*>(a.vc.base);
  const long long mi = ((long long)m.l * a.kc.num_pages * a.kc.H + m.h) * a.kc.bs;
  const long long mp = (long long)a.kc.H * a.kc.bs;
  for (int b = 0; b < m.n; b += per) {
    uint4 kx[U], vx[U];
    Move mv[U];
    float wt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mv[u] = move_at(a, m, kept, b + (u * C + rank) * rows + sub);
      kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
      wt[u] = 0.f;
      if (mv[u].ok) {
        kx[u] = ld16_once(kb + row_at(a.kc, m, mv[u].sp, mv[u].st, es) + c);
        if (vb) vx[u] = ld16_once(vb + row_at(a.vc, m, mv[u].sp, mv[u].st, es) + c);
        if (a.mass_in && c == 0) wt[u] = a.mass_in[mi + mv[u].sp * mp + mv[u].st];
      }
    }
    cluster_arrive_release();  // every lane's loads have landed: their values are used below
    cluster_wait_acquire();
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (mv[u].ok) {
        *reinterpret_cast<uint4*>(const_cast<char*>(kb) + row_at(a.kc, m, mv[u].dp, mv[u].dt, es) + c) = kx[u];
        if (vb) *reinterpret_cast<uint4*>(const_cast<char*>(vb) + row_at(a.vc, m, mv[u].dp, mv[u].dt, es) + c) = vx[u];
        if (a.mass_in && c == 0) a.mass_out[mi + mv[u].dp * mp + mv[u].dt] = wt[u];
      }
  }
}

template <int P>
cudaError_t move_t(const MoveArgs& a, long long most, cudaStream_t s) {
  constexpr int kRows = 8 * (32 / P) < 32 ? 8 * (32 / P) : 32;
  const int per = kMoveThreads / 32 * kRows;
  const long long pieces = std::max((std::min<long long>(a.keep, most) + per - 1) / per, 1ll);  // one looks the tables over
  if (pieces * a.items > 0x7FFFFFFFll) return cudaErrorNotSupported;
  evict_move_kernel<P><<<(unsigned)(pieces * a.items), kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict_select(const KCache& kc, const Table& bt, const float* mass, int sinks, int recent, int keep,
                                int* kept, int* new_lens, int* err, cudaStream_t s) {
  const int grid = bt.R * kc.L * kc.H;
  const long long most = (long long)bt.max_blocks * kc.bs;  // tokens of a request
  // 896 rows of 8192 tokens, us: kept in shared memory 44 (one key at a time 50), read again 105
  if (most <= kMaxCached) {
    const bool vec = kc.bs % 4 == 0 && reinterpret_cast<uintptr_t>(mass) % 16 == 0;
    // Four warps a row where the steps between barriers are short, or where rows queue for an SM. 128 / 512
    // threads, us: 7168 rows of 512 tokens 53 / 117, 896 of 512 12.5 / 18.7, 192 of 512 8.4 / 10.5, 896 of 4096 25 /
    // 29, of 8192 50 / 41, 192 of 2048 12.5 / 10.5, 48 of 4096 15.6 / 10.4.
    const int nt = most <= 1024 || (most <= 4096 && grid > 3 * sm_count()) ? 128 : 512;
    const auto k = nt == 128 ? vec ? evict_select_kernel<128, true, 4> : evict_select_kernel<128, true, 1>
                   : vec     ? evict_select_kernel<512, true, 4>
                             : evict_select_kernel<512, true, 1>;
    const size_t smem = ((size_t)most + 3) / 4 * 16;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (e != cudaSuccess) return e;
    k<<<grid, nt, smem, s>>>(kc, bt, mass, sinks, recent, keep, kept, new_lens, err);
  } else {
    evict_select_kernel<512, false, 1><<<grid, 512, 0, s>>>(kc, bt, mass, sinks, recent, keep, kept, new_lens, err);
  }
  return cudaGetLastError();
}

cudaError_t launch_evict_compact(const KCache& kc, const KCache& vc, const Table& bt, const int* kept, int keep,
                                 const float* mass_in, float* mass_out, const int* dst_pages, int* err,
                                 cudaStream_t s) {
  const int items = bt.R * kc.L * kc.H;
  const MoveArgs a{kc, vc, bt, kept, keep, (keep - 1) / kc.bs + 1, mass_in, mass_out, dst_pages, err, items};
  const int P = kc.D * (kc.dtype == 1 ? 2 : 4) / 16;  // 16-byte pieces of a row
  const long long most = (long long)bt.max_blocks * kc.bs;  // tokens of a request
  if (dst_pages) switch (P) {
      case 4: return move_t<4>(a, most, s);
      case 8: return move_t<8>(a, most, s);
      case 16: return move_t<16>(a, most, s);
      case 32: return move_t<32>(a, most, s);
      default: return cudaErrorNotSupported;
    }
  // CTAs of a cluster: two, and up to eight when there are few rows. 2 / 4 / 8, us: 896 rows of 8192 tokens cut
  // to 2048 378 / 408 / 400 (one: 441), 7168 of 1024 to 512 739 / 772 / 830; 48 rows of 4093 cut to
  // 1024 42 / 25 / 17 (one: 76).
  int C = 2;
  while (C < 8 && (long long)items * C < 4ll * sm_count()) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * C));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_compact_kernel, a, P);
}

}  // namespace kk
