// kk_tree_attn on bf16 caches with few query rows per KV head (a decode token's
// group, a small draft): bound by the bytes of K and V.
//
// Four warps share an item's rows (M = 16 or 32) and take 16 tokens each of
// every 64-token tile. A warp streams its tokens' K and V rows through its own
// ring of shared-memory stages (16-byte asynchronous copies; a token that does
// not exist copies as zeros and reads nothing), multiplies with m16n8k16
// matrix instructions, and keeps its own running maximum, sum and accumulator:
// no barrier between warps until the item ends, so loads never wait for a
// neighbour. Two CTAs of three stages hold 128 KB in flight per SM at D = 128.
// Measured, D = 128, groups of 7, one node: 8 requests of up to 32768 tokens (378
// MB of K and V) 73 us with the join, 5.2 TB/s; a million tokens in pages of 16
// (2.1 GB) 343 us, 6.3 TB/s; 64 selected blocks of 128 tokens for each of 32
// requests (533 MB) 99 us, 5.4 TB/s. What is left: about 12 us of starting, first
// loads and join, and 230 registers, which hold an SM to two CTAs (72 % of DRAM's
// cycles busy, the instruction stream a third).
#include "kk_attn_ring.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTK = kRingTK, kTok = kTK / kWarps;  // tokens of a warp's share of a tile
constexpr int kStages = 3;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte piece c of row `row` in a tile of D-element rows:
// pieces are exchanged within 128 bytes so that eight rows' pieces of one
// column fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int c) {
  return D >= 64 ? row * D * 2 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

template <int D>
__device__ __forceinline__ void load_tokens(uint32_t stage, const Tok& x, int lane) {
  constexpr int CH = D / 8, RI = 32 / CH;  // pieces of a row, rows per instruction
  const int c = lane % CH, sub = lane / CH;
  const uint32_t ok = __ballot_sync(kFull, x.ok);
#pragma unroll
  for (int i = 0; i < kTok / RI; ++i) {
    const int row = i * RI + sub;
    const char* k = reinterpret_cast<const char*>(__shfl_sync(kFull, (unsigned long long)x.k, row)) + c * 16;
    const char* v = reinterpret_cast<const char*>(__shfl_sync(kFull, (unsigned long long)x.v, row)) + c * 16;
    const uint32_t at = stage + swz<D>(row, c);
    cp_async16(at, k, (ok >> row) & 1);
    cp_async16(at + kTok * D * 2, v, (ok >> row) & 1);
  }
}

template <int D, int MR>
__host__ __device__ constexpr int mma_smem() {
  constexpr int ring = kWarps * kStages * kTok * D * 4, join = kWarps * MR * 16 * (D + 2) * 4;
  return (ring > join ? ring : join) + MR * 16 * D * 2;
}

template <int D, int MR>
__global__ void __launch_bounds__(kThreads) attn_mma_kernel(const AttnArgs a) {
  constexpr int M = MR * 16, KS = D / 16, NT = D / 8;
  constexpr int kStage = kTok * D * 4;  // K, then V
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_place[kWarps + 4];
  __shared__ uint32_t s_ok[kWarps][kStages];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  unsigned char* qs = smem + mma_smem<D, MR>() - M * D * 2;
  const uint32_t q_at = smem_u32(qs), ring = smem_u32(smem) + w * kStages * kStage;
  float* join = reinterpret_cast<float*>(smem);  // after an item: [warps][M][D], maxima, sums
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
    Tok nx = find_token<2, kTok>(a, r, rq, h, t0, w, lane);
#pragma unroll
    for (int st = 0; st < kStages - 1; ++st) {
      const bool on = t0 + st < t1;
      if (on) load_tokens<D>(ring + st * kStage, nx, lane);
      cp_commit();
      const uint32_t ok = __ballot_sync(kFull, on && nx.ok) & 0xFFFFu;
      if (lane == 0) s_ok[w][st] = ok;
      nx = find_token<2, kTok>(a, r, rq, h, min(t0 + st + 1, t1 - 1), w, lane);
    }
    for (int i = tid; i < M * (D / 8); i += kThreads) {
      const int m = i / (D / 8), c = i - m * (D / 8), row = row0 + m;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (m < rows)
        x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (rq.node0 + row / a.G) * a.q_sn +
                                            (long long)(h * a.G + row % a.G) * a.q_sh + c * 8);
      *reinterpret_cast<uint4*>(qs + swz<D>(m, c)) = x;
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
        if (on) load_tokens<D>(ring + fs * kStage, nx, lane);
        cp_commit();
        const uint32_t ok = __ballot_sync(kFull, on && nx.ok) & 0xFFFFu;
        if (lane == 0) s_ok[w][fs] = ok;
        nx = find_token<2, kTok>(a, r, rq, h, min(t + kStages, t1 - 1), w, lane);
      }
      const uint32_t kst = ring + st * kStage, vst = kst + kTok * D * 2;
      const uint32_t live = s_ok[w][st];
      const bool draft = t >= rq.tiles_c;
      bool odd = false;
      if (draft) {
        // A drafted Value that is not finite must not meet the zero weights of
        // the nodes that do not see it: it is taken out here and given to the
        // nodes that do after the products.
#pragma unroll 1
        for (int i = lane; i < kTok * D / 8; i += 32) {
          unsigned char* p = smem + (vst - smem_u32(smem)) + i * 16;
          uint4 x = *reinterpret_cast<uint4*>(p);
          uint32_t* y = reinterpret_cast<uint32_t*>(&x);
          bool hit = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((y[e] & 0x7F800000u) == 0x7F800000u) y[e] &= 0x0000FFFFu, hit = true;
            if ((y[e] & 0x00007F80u) == 0x00007F80u) y[e] &= 0xFFFF0000u, hit = true;
          }
          if (hit) *reinterpret_cast<uint4*>(p) = x;
          odd |= hit;
        }
        odd = __any_sync(kFull, odd);
      }
      // scores of 16 tokens
      float s[MR][2][4];
#pragma unroll
      for (int mr = 0; mr < MR; ++mr)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mr][0][e] = s[mr][1][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t b[4];
        ldsm4(b, kst + swz<D>((lane & 7) + ((lane >> 4) << 3), ks * 2 + ((lane >> 3) & 1)));
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
          uint32_t x[4];
          ldsm4(x, q_at + swz<D>(mr * 16 + (lane & 15), ks * 2 + (lane >> 4)));
          mma16816(s[mr][0], x, b[0], b[1]);
          mma16816(s[mr][1], x, b[2], b[3]);
        }
      }
      uint32_t pa[MR][4];
      bool rise = false;
      float al[MR][2];
#pragma unroll
      for (int mr = 0; mr < MR; ++mr)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float mx = m_run[mr][hf];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = nt * 8 + q4 * 2 + e;
              float& x = s[mr][nt][hf * 2 + e];
              bool see = (live >> k) & 1;
              if (draft && see) {
                const int row = row0 + mr * 16 + hf * 8 + g;
                see = row < rq.n * a.G && sees(a, rq, row / a.G, (t - rq.tiles_c) * kTK + w * kTok + k);
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
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const float p0 = ex2(s[mr][nt][hf * 2] - ref), p1 = ex2(s[mr][nt][hf * 2 + 1] - ref);
            sum += p0 + p1;
            pa[mr][nt * 2 + hf] = pack_bf16(p0, p1);  // the weights' one rounding: bf16 feeds the product
          }
          l_run[mr][hf] = l_run[mr][hf] * al[mr][hf] + sum;
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
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b[4];
        ldsm4t(b, vst + swz<D>((lane & 7) + (((lane >> 3) & 1) << 3), n + (lane >> 4)));
#pragma unroll
        for (int mr = 0; mr < MR; ++mr) {
          mma16816(o[mr][n], pa[mr], b[0], b[1]);
          mma16816(o[mr][n + 1], pa[mr], b[2], b[3]);
        }
      }
      if (odd) {  // drafts that are not finite, for the nodes that see them
        const int j0 = (t - rq.tiles_c) * kTK + w * kTok;
        for (int k = 0; k < kTok && j0 + k < rq.n; ++k)
#pragma unroll
          for (int mr = 0; mr < MR; ++mr)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int row = row0 + mr * 16 + hf * 8 + g;
              if (row >= rq.n * a.G || !sees(a, rq, row / a.G, j0 + k)) continue;
              const uint16_t* v = static_cast<const uint16_t*>(a.dv) + (rq.node0 + j0 + k) * a.dv_sn + h * a.dv_sh;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t x = v[n * 8 + q4 * 2 + e];
                  if ((x & 0x7F80u) == 0x7F80u) o[mr][n][hf * 2 + e] += __uint_as_float(x << 16);
                }
            }
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
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<float2*>(join + (w * M + m) * D + n * 8 + q4 * 2) =
              make_float2(o[mr][n][hf * 2], o[mr][n][hf * 2 + 1]);
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
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + d) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
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
  constexpr int smem = mma_smem<D, MR>();
  const cudaError_t e =
      cudaFuncSetAttribute(attn_mma_kernel<D, MR>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_mma_kernel<D, MR><<<a.grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D>
AttnPlan plan_d(bool wide) {
  const bool two = wide && (D == 32 || D == 128);  // registers: the accumulator of 32 rows of 256 does not fit
  const int smem = two ? mma_smem<D, D == 32 || D == 128 ? 2 : 1>() : mma_smem<D, 1>();
  const int per = 227 * 1024 / (smem + 1024 + 256);
  return AttnPlan{AttnPlan::kMma, two ? 32 : 16, kTK, sm_count() * (per < 1 ? 1 : per > 4 ? 4 : per)};
}

}  // namespace

AttnPlan attn_mma_plan(const KCache& kc, bool wide) {
  switch (kc.D) {
    case 32: return plan_d<32>(wide);
    case 64: return plan_d<64>(wide);
    case 128: return plan_d<128>(wide);
    default: return plan_d<256>(wide);
  }
}

cudaError_t launch_attn_mma(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  switch (a.kc.D) {
    case 32: return pl.M == 16 ? go<32, 1>(a, s) : go<32, 2>(a, s);
    case 64: return go<64, 1>(a, s);
    case 128: return pl.M == 16 ? go<128, 1>(a, s) : go<128, 2>(a, s);
    case 256: return go<256, 1>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace kk
