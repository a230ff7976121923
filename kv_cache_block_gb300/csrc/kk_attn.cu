// Attention of drafted nodes (one node: a decode token) over a paged cache,
//   out = sum_t e^(s_t - lse) v_t,  s_t = scale * q . k_t,  lse = log sum_t e^s_t
// over the cached tokens (or those of the selected blocks, "Key-Key Semantic
// Affinity" page §5.2 step 4: only they are loaded) and the drafted nodes a
// node may see. One pass over the tokens with a running maximum and sum per
// row; the work division is kk_attn.cuh's. The main kernels are in kk_attn_f32.cu
// (float32 caches), kk_attn_mma.cu (bf16, few rows) and kk_attn_tc.cu (bf16, many
// rows); this file chooses one and adds up the parts of the items that were cut.
#include <algorithm>

#include "kk_attn.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

// The CTAs [c0, c0 + n) whose partial results make up an item (n = 0: nothing
// to add up, or no rows from `row` of the tile on), and c0's slot: worked out
// again from the sizes while the main kernel still runs, so that nothing but
// the parts is read after it.
struct Cut {
  int c0, n, first, node0, rows;
};
template <int NT>
__device__ __forceinline__ Cut find_cut(const AttnArgs& a, int r, int h, int mt, int row, int M, int TK, int tid) {
  __shared__ long long s_sum[2][NT / 32];
  __shared__ Cut s_cut;
  long long before = 0, all = 0;
  for (int i = tid; i < a.bt.R; i += NT) {
    const long long n = req_units(a, load_req(a, i, M, TK, false));
    all += n;
    if (i < r) before += n;
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    all += __shfl_xor_sync(kFull, all, x);
    before += __shfl_xor_sync(kFull, before, x);
  }
  if ((tid & 31) == 0) {
    s_sum[0][tid >> 5] = before;
    s_sum[1][tid >> 5] = all;
  }
  __syncthreads();
  if (tid == 0) {  // one thread divides for the block
    before = all = 0;
    for (int x = 0; x < NT / 32; ++x) {
      before += s_sum[0][x];
      all += s_sum[1][x];
    }
    const AttnReq rq = load_req(a, r, M, TK, false);
    Cut c = {};
    if (mt < rq.mt && mt * M + row < rq.n * a.G) {
      const Split sp = make_split(all, a.grid);
      const ItemAt it = item_of(rq, h, mt);
      const long long lo = before + it.start;
      c.c0 = split_owner(sp, lo);
      c.n = split_owner(sp, lo + it.units - 1) - c.c0 + 1;
      c.first = split_start(sp, c.c0) == lo ? 0 : 1;  // c0's slot: its first item, or its last
      if (c.n == 1) c.n = 0;
      c.node0 = rq.node0;
      c.rows = rq.n * a.G;
    }
    s_cut = c;
  }
  __syncthreads();
  return s_cut;
}

// Block (item, row chunk): rows of one item's partial results, added up.
// Whole items were written by the main kernel. `wpr` of the eight warps share a
// row (more when few items are cut into many parts): each group of lanes that
// spans a row's D values adds every n-th part in CTA order, and the groups'
// sums are joined in order, so the result does not depend on timing.
constexpr int kCombineThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) attn_combine_kernel(const AttnArgs a, int M, int TK, int mt_max,
                                                                       int wpr) {
  constexpr int L = D / 4 < 32 ? D / 4 : 32;  // lanes of a row
  constexpr int V = D / (4 * L);              // float4 of a lane
  constexpr int NG = kCombineThreads / L;     // lane groups of the block
  __shared__ __align__(16) float s_acc[NG][D];
  __shared__ float s_m[NG], s_l[NG];
  const int tid = threadIdx.x;
  const int mt = blockIdx.x % mt_max, h = (blockIdx.x / mt_max) % a.kc.H, r = blockIdx.x / (mt_max * a.kc.H);
  const int rpb = kCombineThreads / 32 / wpr;  // rows of a block
  const Cut cut = find_cut<kCombineThreads>(a, r, h, mt, blockIdx.y * rpb, M, TK, tid);
  // Every block waits, those with nothing to join too: what the stream or a graph
  // runs next is ordered behind this kernel alone, and without a cut item nothing
  // else here would keep it from ending before the main kernel does.
  pdl_wait();
  const int parts = cut.n;
  if (parts == 0) return;
  const int grp = tid / L, ln = tid % L, gpr = NG / rpb;  // lane groups of a row
  const int row = mt * M + blockIdx.y * rpb + grp / gpr, gi = grp % gpr;
  const bool real = row < cut.rows;
  const int m = real ? row - mt * M : 0;
  float mm = -INFINITY, l = 0.f;
  float4 acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = gi; i < parts; i += gpr) {
    const float* part = partial_slot(a, cut.c0 + i, i == 0 ? cut.first : 0, M, D);
    const float pm = part[M * D + m], pl = part[M * D + M + m];
    const float m2 = fmaxf(mm, pm), ref = m2 == -INFINITY ? 0.f : m2;
    const float f = ex2(mm - ref), al = ex2(pm - ref);
    l = l * f + pl * al;
    mm = m2;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float4 x = *reinterpret_cast<const float4*>(part + m * D + (e * L + ln) * 4);
      acc[e].x = acc[e].x * f + x.x * al;
      acc[e].y = acc[e].y * f + x.y * al;
      acc[e].z = acc[e].z * f + x.z * al;
      acc[e].w = acc[e].w * f + x.w * al;
    }
  }
  if (gpr > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) *reinterpret_cast<float4*>(&s_acc[grp][(e * L + ln) * 4]) = acc[e];
    if (ln == 0) {
      s_m[grp] = mm;
      s_l[grp] = l;
    }
    __syncthreads();
    if (gi != 0) return;
    for (int x = 1; x < gpr; ++x) mm = fmaxf(mm, s_m[grp + x]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    l = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = 0; x < gpr; ++x) {
      const float al = ex2(s_m[grp + x] - ref);
      l += s_l[grp + x] * al;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float4 y = *reinterpret_cast<const float4*>(&s_acc[grp + x][(e * L + ln) * 4]);
        acc[e].x += y.x * al;
        acc[e].y += y.y * al;
        acc[e].z += y.z * al;
        acc[e].w += y.w * al;
      }
    }
  }
  if (!real) return;
  const float inv = row_inv(l);
  const long long at = (long long)(cut.node0 + row / a.G) * a.Hq + h * a.G + row % a.G;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const long long d = at * D + (e * L + ln) * 4;
    store_elem<T>(a.out, d, acc[e].x * inv);
    store_elem<T>(a.out, d + 1, acc[e].y * inv);
    store_elem<T>(a.out, d + 2, acc[e].z * inv);
    store_elem<T>(a.out, d + 3, acc[e].w * inv);
  }
  if (ln == 0 && a.lse) a.lse[at] = row_lse(mm, l);
}

// The same for the tensor-memory kernel's slots, [D/4][256 rows][4]: a lane is a
// row, a warp takes 8 of its values, and every load and store is whole sectors.
// A block has 32 rows x 32 values and, where few items are cut into many parts,
// `groups` of four warps that take every groups-th part and are joined in order.
// Eight parts are in flight a thread: with a row's 128 values in one block and
// four in flight, 18 parts took 11 us of latency.
constexpr int kTcCombineThreads = 128;

struct RowPart {  // a running result: eight values of one row
  float m, l;
  float4 acc[2];
};

template <int D, int groups>
__global__ void __launch_bounds__(kTcCombineThreads * groups)
    attn_combine_tc_kernel(const AttnArgs a, int TK, int mt_max) {
  constexpr int M = 256, U = 8;
  __shared__ RowPart s_part[groups > 1 ? groups - 1 : 1][kTcCombineThreads];
  const int tid = threadIdx.x % kTcCombineThreads, ln = tid & 31, w = tid >> 5;
  const int grp = threadIdx.x / kTcCombineThreads;
  const int mt = blockIdx.x % mt_max, h = (blockIdx.x / mt_max) % a.kc.H, r = blockIdx.x / (mt_max * a.kc.H);
  const AttnReq rq = load_req(a, r, M, TK, false);
  const int m = blockIdx.y * 32 + ln, row = mt * M + m, v4 = (blockIdx.z * 4 + w) * 2;  // first float4 of the row
  const bool real = mt < rq.mt && row < rq.n * a.G;
  pdl_wait();
  const int4 cut = a.cuts[blockIdx.x];
  // the block as one: no such item, or one written whole
  if (mt >= rq.mt || cut.z == cut.x) return;
  // A CTA that gave up a wait leaves the notes of its last items unwritten, and the
  // workspace held anything before: what is no possible note is not followed.
  if (cut.x < 0 || cut.z < cut.x || cut.z >= a.grid || (cut.y & ~1)) return;
  // a single's streams leave a part each, M/2 rows apart
  const int sh = mt >= rq.mt - rq.odd, parts = real ? (cut.z - cut.x + 1) << sh : 0;
  auto slot = [&](int i) { return partial_slot(a, cut.x + (i >> sh), i >> sh ? 0 : cut.y, M, D); };
  auto at_row = [&](int i) { return m + (i & sh) * (M / 2); };
  RowPart s = {-INFINITY, 0.f, {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)}};
  auto add = [&](float al, float l, const float4 (&x)[2]) {
    s.l += l * al;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      s.acc[e].x += x[e].x * al;
      s.acc[e].y += x[e].y * al;
      s.acc[e].z += x[e].z * al;
      s.acc[e].w += x[e].w * al;
    }
  };
  auto raise = [&](float m2) {  // the running results in terms of the maximum m2; the factor's reference
    const float ref = m2 == -INFINITY ? 0.f : m2, f = ex2(s.m - ref);
    s.m = m2;
    s.l *= f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
      s.acc[e] = make_float4(s.acc[e].x * f, s.acc[e].y * f, s.acc[e].z * f, s.acc[e].w * f);
    return ref;
  };
  for (int b = grp; b < parts; b += U * groups) {
    float pm[U], pl[U];
    float4 x[U][2];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int p = b + i * groups;
      const bool on = p < parts;
      const float* part = slot(on ? p : b);
      const int pr = at_row(on ? p : b);
      pm[i] = on ? part[M * D + pr] : -INFINITY;
      pl[i] = part[M * D + M + pr];
      x[i][0] = reinterpret_cast<const float4*>(part)[v4 * M + pr];
      x[i][1] = reinterpret_cast<const float4*>(part)[(v4 + 1) * M + pr];
    }
    float m2 = s.m;
#pragma unroll
    for (int i = 0; i < U; ++i) m2 = fmaxf(m2, pm[i]);
    const float ref = raise(m2);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (b + i * groups >= parts) break;
      add(ex2(pm[i] - ref), pl[i], x[i]);
    }
  }
  if constexpr (groups > 1) {
    if (grp) s_part[grp - 1][tid] = s;
    __syncthreads();
    if (grp) return;
    for (int g = 1; g < groups; ++g) {
      const RowPart o = s_part[g - 1][tid];
      const float ref = raise(fmaxf(s.m, o.m));
      add(ex2(o.m - ref), o.l, o.acc);
    }
  }
  if (!real) return;
  const float inv = row_inv(s.l);
  const long long at = (long long)(rq.node0 + row / a.G) * a.Hq + h * a.G + row % a.G;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at * D + v4 * 4) =
      make_uint4(pack_bf16(s.acc[0].x * inv, s.acc[0].y * inv), pack_bf16(s.acc[0].z * inv, s.acc[0].w * inv),
                 pack_bf16(s.acc[1].x * inv, s.acc[1].y * inv), pack_bf16(s.acc[1].z * inv, s.acc[1].w * inv));
  if (v4 == 0 && a.lse) a.lse[at] = row_lse(s.m, s.l);
}

// Launches a combine kernel so that it may start while the main kernel ends.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*k)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int D>
cudaError_t combine_tc(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  const int rows = a.max_nodes * a.G, mt_max = a.mt_max;
  const long long items = (long long)a.bt.R * a.kc.H * mt_max;
  const dim3 grid((unsigned)items, (unsigned)((std::min(pl.M, rows) + 31) / 32), (unsigned)(D / 32));
  // groups: about eight parts each (a single item leaves two a CTA) while the SMs hold every block. One request
  // of 32768 tokens: 62 -> 39 us (35 rows), 61 -> 49 (252 rows); where blocks of more groups would wait for room,
  // 8 x 2048 tokens and 252 rows, they took 47 us instead of 41.
  const long long blocks = (long long)grid.x * grid.y * grid.z;
  int groups = 1;
  while (groups < 4 && pl.grid * 2 / items > 8 * groups && blocks * groups * 2 <= 4 * sm_count())
    groups *= 2;
  auto go = [&](auto k) { return launch_dependent(k, grid, kTcCombineThreads * groups, s, a, pl.TK, mt_max); };
  return groups == 1   ? go(attn_combine_tc_kernel<D, 1>)
         : groups == 2 ? go(attn_combine_tc_kernel<D, 2>)
                       : go(attn_combine_tc_kernel<D, 4>);
}

template <typename T, int D>
cudaError_t combine_t(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  const int M = pl.M;
  const int mt_max = a.mt_max;
  const long long items = (long long)a.bt.R * a.kc.H * mt_max;
  // warps of a row: about four parts each when every CTA works on few items (one warp always: a million tokens
  // 379 us instead of 346, 8 x 32768 77 instead of 73, one of 1031 14.8 instead of 12.6; 32 selections the same)
  int wpr = 1;
  while (wpr < 8 && pl.grid / items > 4 * wpr) wpr *= 2;
  const int rows = min(M, a.max_nodes * a.G), rpb = kCombineThreads / 32 / wpr;
  return launch_dependent(attn_combine_kernel<T, D>, dim3((unsigned)items, (unsigned)((rows + rpb - 1) / rpb)),
                          kCombineThreads, s, a, M, pl.TK, mt_max, wpr);
}

// When the tensor-memory kernel is taken, where the caches' layouts suit it: it
// starts and ends slower than the mma kernel (23 against 15 us for 4 K cached
// tokens of all requests and KV heads), which reads the tokens once for every 16
// rows; so once tokens x (tiles of 16 rows - 1) pass 72 K. Measured with groups
// of 7 (mma / tensor memory, us), D = 128: 4 K x 5 20.7 / 23.1, 16 K x 1 20.5 /
// 22.9, 16 K x 3 24.8 / 23.7, 64 K x 1 28.7 / 31.0, 16 K x 5 26.9 / 24.9, 64 K x 3
// 37.4 / 33.0, 64 K x 5 46.9 / 37.2; D = 64: 64 K x 1 20.7 / 24.9, 16 K x 5 20.7 /
// 18.8, 64 K x 3 26.9 / 25.8, 64 K x 5 32.5 / 26.9. One tile of 16 rows: 1 M tokens
// 97.0 / 96.5 and 131 K 26.9 / 31.5 (D = 64: 57.4 / 65.8 and 20.7 / 28.9).
constexpr long long kTcWork = 72 << 10;
// From where the mma kernel's tiles have 32 rows (layouts that do not suit the
// other kernel): 512 K tokens of 128 dims and 28, 63, 91 rows 90 / 153 / 215 us
// against 100 / 176 / 252 with 16, but 64 K tokens 31 / 41 / 51 against 29 / 37 / 47;
// 1 M of 32 dims and 28, 63 rows 66 / 123 against 77 / 138. Never for 64 dims (512 K:
// 80 / 130 / 173 against 60 / 101 / 139).
constexpr long long kWideTokens = 256 << 10;

AttnPlan plan(const KCache& kc, const KCache& vc, int max_nodes, int G, long long tokens) {
  const int rows = max_nodes * G;
  if (kc.dtype != 1) return attn_f32_plan(kc, rows);
  if (tokens * ((rows - 1) / 16) >= kTcWork && attn_tc_suits(kc) && attn_tc_suits(vc)) return attn_tc_plan();
  return attn_mma_plan(kc, rows > 16 && tokens >= kWideTokens);
}

// Cached tokens of every request and KV head that a call reads, at most.
long long most_tokens(const AttnArgs& a) {
  const long long blocks = a.sel_pages ? std::min(a.selK, a.bt.max_blocks) : a.bt.max_blocks;
  return blocks * a.kc.bs * a.bt.R * a.kc.H;
}

size_t plan_bytes(const AttnPlan& pl, int D) {
  return (size_t)pl.grid * (pl.kind == AttnPlan::kTc ? 3 : 2) * pl.M * (D + 2) * sizeof(float);
}

// The notes on the items, in front of the partial results.
size_t cut_bytes(const AttnPlan& pl, int R, int H, int rows) {
  if (pl.kind != AttnPlan::kTc) return 0;
  return ((size_t)R * H * ((rows + pl.M - 1) / pl.M) * sizeof(int4) + 255) & ~size_t(255);
}

}  // namespace

size_t attn_workspace_bytes(const KCache& kc, int R, int max_nodes, int G) {
  // enough for any: which one runs also depends on the V cache's strides and the tokens
  const int rows = max_nodes * G;
  auto size = [&](const AttnPlan& pl) { return cut_bytes(pl, R, kc.H, rows) + plan_bytes(pl, kc.D); };
  if (kc.dtype != 1) return size(attn_f32_plan(kc, rows));
  const size_t n = size(attn_mma_plan(kc, false));
  if (rows <= 16) return n;
  const size_t m = std::max(n, size(attn_mma_plan(kc, true)));
  return attn_tc_suits(kc) ? std::max(m, size(attn_tc_plan())) : m;
}

cudaError_t launch_tree_attn(AttnArgs a, cudaStream_t s) {
  const AttnPlan pl = plan(a.kc, a.vc, a.max_nodes, a.G, most_tokens(a));
  a.grid = pl.grid;
  a.twin = pl.kind == AttnPlan::kTc;
  const int rows = a.max_nodes * a.G;
  a.mt_max = (rows + pl.M - 1) / pl.M;
  a.cuts = reinterpret_cast<int4*>(a.ws);
  a.ws = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + cut_bytes(pl, a.bt.R, a.kc.H, rows));
  const bool bf = a.kc.dtype == 1;
  cudaError_t e = cudaErrorNotSupported;
  if (pl.kind == AttnPlan::kTc) {
    e = launch_attn_tc(a, s);
  } else if (pl.kind == AttnPlan::kMma) {
    e = launch_attn_mma(a, pl, s);
  } else {
    e = launch_attn_f32(a, pl, s);
  }
  if (e != cudaSuccess) return e;
  if (pl.kind == AttnPlan::kTc) return a.kc.D == 64 ? combine_tc<64>(a, pl, s) : combine_tc<128>(a, pl, s);
  switch (a.kc.D) {
    case 32: return bf ? combine_t<bf16_t, 32>(a, pl, s) : combine_t<float, 32>(a, pl, s);
    case 64: return bf ? combine_t<bf16_t, 64>(a, pl, s) : combine_t<float, 64>(a, pl, s);
    case 128: return bf ? combine_t<bf16_t, 128>(a, pl, s) : combine_t<float, 128>(a, pl, s);
    default: return combine_t<bf16_t, 256>(a, pl, s);
  }
}

}  // namespace kk
