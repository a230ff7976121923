// kk_tree_attn on float32 caches, on the tensor cores: every operand x is cut
// into two tf32 numbers, x = hi + lo up to 2^-22 |x|, and a product is hi hi' +
// hi lo' + lo hi' (the dropped lo lo' is below 2^-22 of it), summed in float32.
// That keeps the products of float32 inputs within a few roundings of float32
// while M = 16 or 32 query rows share one read of K and V; on the CUDA cores 8
// rows shared it and a tile waited for uncoalesced rows.
//
// The structure is kk_attn_mma.cu's (a ring of 16-byte asynchronous copies per
// warp, no barrier between warps until an item ends), with m16n8k8 instructions
// and 8 tokens a warp: four warps of 16 tokens left each scheduler one warp and
// its chain of dependent products.
// Which of eight contracted positions holds which dim (or token) does not matter
// as long as both operands agree: it is chosen so that a lane reads 16 bytes of
// a row at once, and so that the scores' registers are the next product's.
// Measured, groups of 7, D = 64: one node, 8 x 8192 tokens and 2 heads (67 MB) 35
// us; 8 nodes, 2 x 4096 tokens 27 us, of which the main kernel 22, half its issue
// slots busy; on the CUDA cores 44 (8 nodes). 40 nodes, 8 x 8192: 26 TF/s of
// products (78 of tf32 instructions'), bound by the issue of cuts and products.
#include "kk_attn_ring.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTK = kRingTK, kTok = kTK / kWarps;  // tokens of a warp's share: one 8-column product
constexpr int kStages = 3;

// x's leading 11 bits as tf32, rounded to nearest.
__device__ __forceinline__ uint32_t tf32_of(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
struct Halves {
  uint32_t hi, lo;
};
__device__ __forceinline__ Halves split(float x) {
  Halves h;
  h.hi = tf32_of(x);
  h.lo = tf32_of(x - __uint_as_float(h.hi));
  return h;
}
// Whether x has no two halves: what tf32 rounds to infinity, infinities, NaN.
__device__ __forceinline__ bool no_halves(float x) { return (__float_as_uint(x) & 0x7FFFFFFFu) >= 0x7F7FF000u; }
__device__ __forceinline__ void mma1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The first half of a query's value: what would round to infinity is cut off
// instead, so that both halves together are the value, also for whole_dot.
__device__ __forceinline__ float query_half(float x) {
  return isfinite(x) && no_halves(x) ? __uint_as_float(__float_as_uint(x) & 0xFFFFE000u) : __uint_as_float(tf32_of(x));
}
// Byte offset of 16-byte piece c of row `row`: pieces are exchanged so that the
// rows 2q, 2q+1 (scores) and the rows of one parity (weights) that eight lanes
// read together fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  const int f = (((row >> 1) & 3) << 1) ^ ((row & 1) << 2);
  return row * D * 4 + ((c ^ f) << 4);
}

// q_m . k_t from the whole values.
template <int D>
__device__ __noinline__ float whole_dot(const unsigned char* qh, const unsigned char* ql, const unsigned char* k, int m,
                                        int t) {
  auto f4 = [](const unsigned char* p) { return *reinterpret_cast<const float4*>(p); };
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < D / 4; ++c) {
    const float4 y = f4(k + swz<D>(t, c)), x = f4(qh + swz<D>(m, c)), z = f4(ql + swz<D>(m, c));
    sum += (x.x + z.x) * y.x + (x.y + z.y) * y.y + (x.z + z.z) * y.z + (x.w + z.w) * y.w;
  }
  return sum;
}

template <int D>
__device__ __forceinline__ void load_tokens(uint32_t stage, const Tok& x, int lane) {
  constexpr int CH = D / 4, RI = 32 / CH;  // pieces of a row, rows per instruction
  const int c = lane % CH, sub = lane / CH;
  const uint32_t ok = __ballot_sync(kFull, x.ok);
#pragma unroll
  for (int i = 0; i < kTok / RI; ++i) {
    const int row = i * RI + sub;
    const char* k = reinterpret_cast<const char*>(__shfl_sync(kFull, (unsigned long long)x.k, row)) + c * 16;
    const char* v = reinterpret_cast<const char*>(__shfl_sync(kFull, (unsigned long long)x.v, row)) + c * 16;
    const uint32_t at = stage + swz<D>(row, c);
    cp_async16(at, k, (ok >> row) & 1);
    cp_async16(at + kTok * D * 4, v, (ok >> row) & 1);
  }
}

template <int D, int MR>
__host__ __device__ constexpr int f32_smem() {
  constexpr int ring = kWarps * kStages * kTok * D * 8, join = kWarps * MR * 16 * (D + 2) * 4;
  return (ring > join ? ring : join) + 2 * MR * 16 * D * 4;  // the queries' halves behind the ring
}

template <int D, int MR>
__global__ void __launch_bounds__(kThreads) attn_f32_kernel(const AttnArgs a) {
  constexpr int M = MR * 16, KS = D / 16, NT = D / 8;
  constexpr int kStage = kTok * D * 8;  // K, then V
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_place[kWarps + 4];
  __shared__ uint32_t s_ok[kWarps][kStages];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  unsigned char* qh = smem + f32_smem<D, MR>() - 2 * M * D * 4;
  unsigned char* ql = qh + M * D * 4;
  unsigned char* ring = smem + w * kStages * kStage;
  float* join = reinterpret_cast<float*>(smem);  // after an item: [warps][M][D], maxima, sums
  auto f4 = [](const unsigned char* p) { return *reinterpret_cast<const float4*>(p); };
  pdl_launch_dependents();
  const AttnPlace pl = find_place<kThreads>(a, blockIdx.x, M, kTK, s_place, tid);
  int r = pl.r;
  long long base = pl.base;
  for (long long u = pl.u0; u < pl.u1;) {
    const AttnReq rq = load_req(a, r, M, kTK, false);
    const long long units = req_units(a, rq);
    if (u >= base + units) {
      base += units;
      ++r;
      continue;
    }
    ItemAt it = item_at(rq, u - base);
    it.t1 = (int)min((long long)rq.tiles, it.t0 + (pl.u1 - u));
    const int t0 = it.t0, t1 = it.t1, h = it.h, row0 = it.mt * M;
    const int rows = min(M, rq.n * a.G - row0);
    // the first tiles' copies go out before the queries are read
    Tok nx = find_token<4, kTok>(a, r, rq, h, t0, w, lane);
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) {
      const bool on = t0 + st < t1;
      if (on) load_tokens<D>(smem_u32(ring) + st * kStage, nx, lane);
      cp_commit();
      const uint32_t ok = __ballot_sync(kFull, on && nx.ok) & 0xFFu;
      if (lane == 0) s_ok[w][st] = ok;
      nx = find_token<4, kTok>(a, r, rq, h, min(t0 + st + 1, t1 - 1), w, lane);
    }
    for (int i = tid; i < M * (D / 4); i += kThreads) {
      const int m = i / (D / 4), c = i - m * (D / 4), row = row0 + m;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m < rows)
        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (rq.node0 + row / a.G) * a.q_sn +
                                             (long long)(h * a.G + row % a.G) * a.q_sh + c * 4);
      const float4 y = make_float4(query_half(x.x), query_half(x.y), query_half(x.z), query_half(x.w));
      *reinterpret_cast<float4*>(qh + swz<D>(m, c)) = y;
      *reinterpret_cast<float4*>(ql + swz<D>(m, c)) = make_float4(isinf(x.x) ? 0.f : x.x - y.x, isinf(x.y) ? 0.f : x.y - y.y,
                                                                  isinf(x.z) ? 0.f : x.z - y.z, isinf(x.w) ? 0.f : x.w - y.w);
    }
    __syncthreads();

    float o[MR][NT][4], m_run[MR][2], l_run[MR][2];
#pragma unroll
    for (int mr = 0; mr < MR; ++mr) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mr][n][e] = 0.f;
      m_run[mr][0] = m_run[mr][1] = -INFINITY;
      l_run[mr][0] = l_run[mr][1] = 0.f;
    }
    int st = 0;
    for (int t = t0; t < t1; ++t) {
      cp_wait<kStages - 2>();
      __syncwarp();
      {  // refill the stage read in the last turn
        const int fs = st == 0 ? kStages - 1 : st - 1;
        const bool on = t + kStages - 1 < t1;
        if (on) load_tokens<D>(smem_u32(ring) + fs * kStage, nx, lane);
        cp_commit();
        const uint32_t ok = __ballot_sync(kFull, on && nx.ok) & 0xFFu;
        if (lane == 0) s_ok[w][fs] = ok;
        nx = find_token<4, kTok>(a, r, rq, h, min(t + kStages, t1 - 1), w, lane);
      }
      unsigned char* kst = ring + st * kStage;
      unsigned char* vst = kst + kTok * D * 4;
      const uint32_t live = s_ok[w][st];
      const bool draft = t >= rq.tiles_c;
      const int j0 = (t - rq.tiles_c) * kTK + w * kTok;  // a drafted tile's first node
      // scores of 8 tokens; the three kinds of product in sums of their own, three
      // chains instead of one
      float s[MR][4], c3[3][MR][4];
#pragma unroll
      for (int x = 0; x < 3; ++x)
#pragma unroll
        for (int mr = 0; mr < MR; ++mr)
#pragma unroll
          for (int e = 0; e < 4; ++e) c3[x][mr][e] = 0.f;
      // for many rows a loop whose code is fetched once (unrolled, instruction fetch
      // bound the short calls); one row tile needs the overlap of its few products
#pragma unroll(MR == 1 ? KS : 1)
      for (int ks = 0; ks < KS; ++ks) {
        const float4 kx = f4(kst + swz<D>(g, ks * 4 + q4));
        const Halves b[4] = {split(kx.x), split(kx.y), split(kx.z), split(kx.w)};
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
          const float4 h0 = f4(qh + swz<D>(mr * 16 + g, ks * 4 + q4)), h1 = f4(qh + swz<D>(mr * 16 + 8 + g, ks * 4 + q4));
          const float4 l0 = f4(ql + swz<D>(mr * 16 + g, ks * 4 + q4)), l1 = f4(ql + swz<D>(mr * 16 + 8 + g, ks * 4 + q4));
          const uint32_t ah[2][4] = {{__float_as_uint(h0.x), __float_as_uint(h1.x), __float_as_uint(h0.y), __float_as_uint(h1.y)},
                                     {__float_as_uint(h0.z), __float_as_uint(h1.z), __float_as_uint(h0.w), __float_as_uint(h1.w)}};
          const uint32_t al[2][4] = {{tf32_of(l0.x), tf32_of(l1.x), tf32_of(l0.y), tf32_of(l1.y)},
                                     {tf32_of(l0.z), tf32_of(l1.z), tf32_of(l0.w), tf32_of(l1.w)}};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma1688(c3[0][mr], al[x], b[2 * x].hi, b[2 * x + 1].hi);
            mma1688(c3[1][mr], ah[x], b[2 * x].lo, b[2 * x + 1].lo);
            mma1688(c3[2][mr], ah[x], b[2 * x].hi, b[2 * x + 1].hi);
          }
        }
      }
#pragma unroll
      for (int mr = 0; mr < MR; ++mr)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[mr][e] = (c3[0][mr][e] + c3[1][mr][e]) + c3[2][mr][e];
      // A Key without halves (infinite, or rounded to infinity) and an infinite query
      // leave NaN here: the scores are formed again from the whole values.
      bool nan = false;
#pragma unroll
      for (int mr = 0; mr < MR; ++mr)
#pragma unroll
        for (int e = 0; e < 4; ++e) nan |= s[mr][e] != s[mr][e];
      if (__any_sync(kFull, nan)) {
#pragma unroll
        for (int mr = 0; mr < MR; ++mr)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = mr * 16 + (e & 2 ? 8 : 0) + g, k = q4 * 2 + (e & 1);
            s[mr][e] = whole_dot<D>(qh, ql, kst, m, k);
          }
      }
      bool rise = false;
      float al[MR][2];
#pragma unroll
      for (int mr = 0; mr < MR; ++mr)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float mx = m_run[mr][hf];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = q4 * 2 + e;
            float& x = s[mr][hf * 2 + e];
            bool see = (live >> k) & 1;
            if (draft && see) {
              const int row = row0 + mr * 16 + hf * 8 + g;
              see = row < rq.n * a.G && sees(a, rq, row / a.G, j0 + k);
            }
            x = see ? x * a.scale_log2 : -INFINITY;  // selected, whatever a hidden place holds
            mx = fmaxf(mx, x);
          }
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
          const float ref = mx == -INFINITY ? 0.f : mx;
          al[mr][hf] = ex2(m_run[mr][hf] - ref);
          rise |= mx > m_run[mr][hf];
          m_run[mr][hf] = mx;
          const float p0 = ex2(s[mr][hf * 2] - ref), p1 = ex2(s[mr][hf * 2 + 1] - ref);
          s[mr][hf * 2] = p0;
          s[mr][hf * 2 + 1] = p1;
          l_run[mr][hf] = l_run[mr][hf] * al[mr][hf] + (p0 + p1);
        }
      if (__any_sync(kFull, rise)) {  // a maximum rarely rises after the first tiles
#pragma unroll
        for (int mr = 0; mr < MR; ++mr)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[mr][n][0] *= al[mr][0];
            o[mr][n][1] *= al[mr][0];
            o[mr][n][2] *= al[mr][1];
            o[mr][n][3] *= al[mr][1];
          }
      }
      // Values without halves (too large for tf32, infinite, NaN) are given to the rows
      // that see them here, and 0 stands for them in the products. A NaN alone among
      // cached tokens, which all rows see, goes the ordinary way. Looking for them
      // costs 0 to 6 % (64 dims, 40 nodes 341 -> 363 us).
      float top = 0.f;
      bool bad = false;
#pragma unroll
      for (int blk = 0; blk < D / 32; ++blk)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 v = f4(vst + swz<D>(q4 * 2 + k, blk * 8 + g));
          top = fmaxf(fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
          if (draft) bad |= v.x != v.x || v.y != v.y || v.z != v.z || v.w != v.w;
        }
      if (__any_sync(kFull, bad || no_halves(top))) {
#pragma unroll 1
        for (int k = 0; k < kTok; ++k) {
          float* x = reinterpret_cast<float*>(vst + k * D * 4);  // the token's row, its pieces in their own order
#pragma unroll
          for (int mr = 0; mr < MR; ++mr)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int row = row0 + mr * 16 + hf * 8 + g;
              const float p = __shfl_sync(kFull, k & 1 ? s[mr][hf * 2 + 1] : s[mr][hf * 2], (lane & ~3) | k >> 1);
              const bool sure = row < rq.n * a.G && (!draft || (j0 + k < rq.n && sees(a, rq, row / a.G, j0 + k)));
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const float y = x[(swz<D>(k, n / 4 * 8 + q4 * 2 + e) - k * D * 4) / 4 + n % 4];
                  if (sure && no_halves(y)) o[mr][n][hf * 2 + e] += isfinite(y) ? p * y : y;
                }
            }
          __syncwarp();
          for (int i = lane; i < D; i += 32)
            if (no_halves(x[i])) x[i] = 0.f;
        }
        __syncwarp();
      }
      // Position q4 of the contraction is token 2 q4, position q4 + 4 token 2 q4 + 1
      uint32_t ph[MR][4], pw[MR][4];
#pragma unroll
      for (int mr = 0; mr < MR; ++mr) {
        const Halves x0 = split(s[mr][0]), x1 = split(s[mr][2]), x2 = split(s[mr][1]), x3 = split(s[mr][3]);
        ph[mr][0] = x0.hi, ph[mr][1] = x1.hi, ph[mr][2] = x2.hi, ph[mr][3] = x3.hi;
        pw[mr][0] = x0.lo, pw[mr][1] = x1.lo, pw[mr][2] = x2.lo, pw[mr][3] = x3.lo;
      }
#pragma unroll
      for (int blk = 0; blk < D / 32; ++blk) {  // column n of product j is dim blk * 32 + 4 n + j
        const float4 v0 = f4(vst + swz<D>(q4 * 2, blk * 8 + g)), v1 = f4(vst + swz<D>(q4 * 2 + 1, blk * 8 + g));
        const Halves b0[4] = {split(v0.x), split(v0.y), split(v0.z), split(v0.w)};
        const Halves b1[4] = {split(v1.x), split(v1.y), split(v1.z), split(v1.w)};
#pragma unroll
        for (int k = 0; k < 3; ++k)  // each kind over all accumulators: no product waits for the one before
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int mr = 0; mr < MR; ++mr)
              mma1688(o[mr][blk * 4 + j], k == 0 ? pw[mr] : ph[mr], k == 1 ? b0[j].lo : b0[j].hi,
                      k == 1 ? b1[j].lo : b1[j].hi);
      }
      __syncwarp();
      st = st == kStages - 1 ? 0 : st + 1;
    }
    cp_wait<0>();
    __syncthreads();
    // the warps' shares, joined through the ring's memory
    float* jm = join + kWarps * M * D;
    float* jl = jm + kWarps * M;
#pragma unroll
    for (int mr = 0; mr < MR; ++mr)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int m = mr * 16 + hf * 8 + g;
        float l = l_run[mr][hf];
        l += __shfl_xor_sync(kFull, l, 1);
        l += __shfl_xor_sync(kFull, l, 2);
        if (q4 == 0) {
          jm[w * M + m] = m_run[mr][hf];
          jl[w * M + m] = l;
        }
#pragma unroll
        for (int blk = 0; blk < D / 32; ++blk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(join + (w * M + m) * D + blk * 32 + (q4 * 2 + e) * 4) =
                make_float4(o[mr][blk * 4][hf * 2 + e], o[mr][blk * 4 + 1][hf * 2 + e], o[mr][blk * 4 + 2][hf * 2 + e],
                            o[mr][blk * 4 + 3][hf * 2 + e]);
      }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == rq.tiles;
    float* part = partial_slot(a, blockIdx.x, u == pl.u0 ? 0 : 1, M, D);
    for (int i = tid; i < rows * (D / 4); i += kThreads) {
      const int m = i / (D / 4), d = (i - m * (D / 4)) * 4;
      float mm = jm[m];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) mm = fmaxf(mm, jm[x * M + m]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float f = ex2(jm[x * M + m] - ref);
        const float4 y = *reinterpret_cast<const float4*>(join + (x * M + m) * D + d);
        l += jl[x * M + m] * f;
        acc.x += y.x * f;
        acc.y += y.y * f;
        acc.z += y.z * f;
        acc.w += y.w * f;
      }
      if (whole) {
        const int row = row0 + m;
        const long long at = (long long)(rq.node0 + row / a.G) * a.Hq + h * a.G + row % a.G;
        const float inv = row_inv(l);
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at * D + d) =
            make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (d == 0 && a.lse) a.lse[at] = row_lse(mm, l);
      } else {
        *reinterpret_cast<float4*>(part + m * D + d) = acc;
        if (d == 0) {
          part[M * D + m] = mm;
          part[M * D + M + m] = l;
        }
      }
    }
    __syncthreads();
    u += t1 - t0;
  }
}

template <int D, int MR>
cudaError_t go(const AttnArgs& a, cudaStream_t s) {
  constexpr int smem = f32_smem<D, MR>();
  const cudaError_t e =
      cudaFuncSetAttribute(attn_f32_kernel<D, MR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_f32_kernel<D, MR><<<a.grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D, int MR>
AttnPlan plan_t() {
  const int per = 227 * 1024 / (f32_smem<D, MR>() + 1024 + 256);
  return AttnPlan{AttnPlan::kF32, MR * 16, kTK, sm_count() * (per < 1 ? 1 : per > 4 ? 4 : per)};
}

}  // namespace

// 16 rows a tile, 32 where rows of 128 dims make the reads dear. Groups of 7, us
// at 32 / 16 rows: D = 128, 8 x 8192 tokens and 28, 56, 280 rows 87 / 94, 146 / 167,
// 555 / 670 (2 x 4096: 28.9 / 26.9, 37.1 / 35.9, 92.5 / 103); D = 64 64 / 52, 105 / 88,
// 386 / 340 (64 rows: 89 at 56, 363 at 280): the more CTAs of an SM hide more.
AttnPlan attn_f32_plan(const KCache& kc, int rows) {
  if (kc.D == 128) return rows <= 16 ? plan_t<128, 1>() : plan_t<128, 2>();
  return kc.D == 32 ? plan_t<32, 1>() : plan_t<64, 1>();
}

cudaError_t launch_attn_f32(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  switch (a.kc.D) {
    case 32: return go<32, 1>(a, s);
    case 64: return go<64, 1>(a, s);
    case 128: return pl.M == 16 ? go<128, 1>(a, s) : go<128, 2>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace kk
