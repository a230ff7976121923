// Attention mass: the weight every cached token received from a set of query
// rows whose lse is known,
//   mass_out = decay * mass_in + sum_i w_i sum_g [t < len_i] e^(s_igt - lse_ig)
// the score by which tokens are evicted. The products are formed again from
// the Keys (K is read once; the weights themselves are never stored). The work
// division is kk_attn.cuh's, with one unit per (request, KV head, token tile);
// a token's sum belongs to one thread, so there are no atomics. Here: float32
// caches, and bf16 ones whose layout no tensor map suits (kk_mass_tc.cu has the
// rest: 7 rows, up to 8 x 32768 tokens of 4 heads and 128 dims 41 us, with this
// kernel 86).
//
// A warp streams its Keys through its own two stages of shared memory, whole rows
// at a time (a thread that reads its own Key from memory touches a line for every
// 16 bytes: 316 us where this takes 149), and four lanes share each Key's dims.
// Measured, float32: 8 x 32768 tokens of 4 heads and 7 rows 149 us with 128 dims
// (546 MB, 3.7 TB/s), 77 with 64; 4 x 52780 of 64 dims and one row (54 MB) 17 us;
// 56 causal rows, 8 x 8192 tokens of 2 heads 57 us (64 dims) and 130 (128): bound by
// instructions, of which two thirds are the products'.
#include "kk_attn.cuh"

namespace kk {
namespace {

constexpr int kStages = 2;

// Sizes by a Key's bytes, so that three CTAs fit an SM (two on bf16 caches, whose
// Keys take more registers as they are widened): tokens of
// a tile, query rows staged at a time, and the Keys that four lanes share (a query
// value read from shared memory serves all of them; a CTA has a warp for every
// eight times as many).
template <typename T, int D>
struct Mass {
  static constexpr int kKey = D * elem_bytes<T>();
  static constexpr int kTK = kKey >= 512 ? 64 : 128;
  static constexpr int kRows = kKey >= 512 ? 16 : 32;
  static constexpr int kN = kKey >= 512 ? 2 : 4;
  static constexpr int kThreads = kTK / 8 / kN * 32;
  static constexpr int kCtas = kKey <= 128 ? 4 : elem_bytes<T>() == 4 ? 3 : 2;
  static constexpr int kSmem = kTK * kStages * kKey;
};
// Where 16-byte piece c of Key `row` lies in a warp's stage: two Keys next to one
// another in different halves of the banks.
template <int NV>
__device__ __forceinline__ int piece_at(int row, int c) {
  return (row * NV + (NV >= 8 ? c ^ (row & 1) * 4 : c)) * 16;
}

struct MassTok {  // a lane's token: its Key, where its mass lies, whether it exists
  const char* k;
  long long out;
  bool ok;
};

// Of four lanes' sums of N Keys, lane q's is Key q % N's.
template <int N>
__device__ __forceinline__ float own_sum(const float (&s)[N], int q) {
  const bool o1 = q & 1, o2 = q & 2;
  const float lo = (o1 ? s[1] : s[0]) + __shfl_xor_sync(kFull, o1 ? s[0] : s[1], 1);
  if constexpr (N == 2) return lo + __shfl_xor_sync(kFull, lo, 2);
  else {
    const float hi = (o1 ? s[3] : s[2]) + __shfl_xor_sync(kFull, o1 ? s[2] : s[3], 1);
    return (o2 ? hi : lo) + __shfl_xor_sync(kFull, o2 ? lo : hi, 2);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(Mass<T, D>::kThreads, Mass<T, D>::kCtas) mass_simt_kernel(const AttnArgs a) {
  constexpr int EPV = Vec16<T>::kElems;
  constexpr int ES = elem_bytes<T>();
  constexpr int NV = D / EPV;  // 16-byte pieces of a Key
  constexpr int PL = NV / 4;   // a lane's pieces of each of its Keys
  constexpr int kTK = Mass<T, D>::kTK, kRows = Mass<T, D>::kRows, kThreads = Mass<T, D>::kThreads;
  constexpr int N = Mass<T, D>::kN, kTok = 8 * N;
  constexpr int SB = kTok * NV * 16;  // a warp's stage
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(16) float s_q[kRows][D];
  __shared__ float s_lse[kRows], s_w[kRows];
  __shared__ int s_len[kRows];
  __shared__ long long s_place[kThreads / 32 + 4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * kStages * SB;
  // Four lanes share N Keys, rows g, g + 8, ... of the warp's; the lane's own, whose
  // sums it ends up with, is g + 8 (q % N).
  const int g = lane >> 2, q = lane & 3, own = warp * kTok + g + 8 * (q % N);
  const AttnPlace pl = find_place<kThreads>(a, blockIdx.x, 1, kTK, s_place, tid);
  int r = pl.r;
  long long base = pl.base;
  for (long long u = pl.u0; u < pl.u1;) {
    const AttnReq rq = load_req(a, r, 1, kTK, false);
    const long long units = req_units(a, rq);
    if (u >= base + units) {
      base += units;
      ++r;
      continue;
    }
    const int h = (int)udiv(u - base, rq.tiles), t0 = (int)(u - base - (long long)h * rq.tiles);
    const int t1 = (int)min((long long)rq.tiles, t0 + (pl.u1 - u));
    const int rows = rq.n * a.G, old = a.old_lens ? a.old_lens[r] : rq.T;

    // A token's page is read a tile before it is looked at, so that no warp waits for it.
    auto page_of = [&](int t) {
      const int v = t * kTK + own;
      return t < t1 && v < rq.T ? a.bt.pages[rq.off + v / a.kc.bs] : 0;
    };
    auto look = [&](int t, int page) {
      MassTok x = {static_cast<const char*>(a.kc.base), 0, false};
      const int v = t * kTK + own;
      if (t >= t1 || v >= rq.T) return x;
      if (page < 0 || page >= a.kc.num_pages) {
        flag_error(a.err, kErrBadIndex);
        return x;
      }
      const int tok = v % a.kc.bs;
      x.ok = true;
      x.k += (a.layer * a.kc.sL + page * a.kc.sP + h * a.kc.sH + tok * a.kc.sT) * ES;
      x.out = (((long long)a.layer * a.kc.num_pages + page) * a.kc.H + h) * a.kc.bs + tok;
      return x;
    };
    auto had = [&](const MassTok& x, int t) {  // a lane's token's weight so far
      return x.ok && a.mass_in && t * kTK + own < old ? a.decay * a.mass_in[x.out] : 0.f;
    };
    auto load = [&](const MassTok& x, int t) {  // the warp's Keys of tile t, whole rows at a time
      const uint32_t dst = smem_u32(ring + (t - t0) % kStages * SB);
      if (t < t1) {
#pragma unroll 8
        for (int i = lane; i < kTok * NV; i += 32) {
          const int row = i / NV, c = i % NV, from = (row & 7) * 4 + (row >> 3);
          const char* p = reinterpret_cast<const char*>(
              __shfl_sync(kFull, reinterpret_cast<unsigned long long>(x.k), from));
          cp_async16(dst + piece_at<NV>(row, c), p + c * 16, __shfl_sync(kFull, (int)x.ok, from));
        }
      }
      cp_commit();
    };
    auto stage_rows = [&](int b) {  // rows b .. b + kRows of the item, those past its last with weight 0
      const int nr = min(kRows, rows - b);
      __syncthreads();
      for (int i = tid; i < nr * D; i += kThreads) {
        const int m = i / D, d = i - m * D, row = b + m;
        const long long x = (rq.node0 + row / a.G) * a.q_sn + (long long)(h * a.G + row % a.G) * a.q_sh + d;
        s_q[m][d] = ES == 4 ? static_cast<const float*>(a.q)[x]
                            : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.q)[x] << 16);
      }
      if (tid < kRows) {
        s_w[tid] = 0.f;
        if (tid < nr) {
          const int row = b + tid, node = rq.node0 + row / a.G;
          const float l = a.lse[(long long)node * a.Hq + h * a.G + row % a.G];
          // a row that saw nothing gives nothing
          s_w[tid] = l == -INFINITY ? 0.f : a.row_w ? a.row_w[node] : 1.f;
          s_lse[tid] = l * 1.44269504088896341f;
          s_len[tid] = a.row_lens ? a.row_lens[node] : rq.T;
        }
      }
      __syncthreads();
    };

    MassTok x0 = look(t0, page_of(t0));
    int page1 = page_of(t0 + 1);
    load(x0, t0);
    float had0 = had(x0, t0);
    if (rows <= kRows) stage_rows(0);
    for (int t = t0; t < t1; ++t) {
      const MassTok x1 = look(t + 1, page1);
      page1 = page_of(t + 2);
      load(x1, t + 1);
      const float had1 = had(x1, t + 1);
      const int v = t * kTK + own;
      cp_wait<kStages - 1>();
      __syncwarp();
      uint4 k[N][PL];
      const unsigned char* st = ring + (t - t0) % kStages * SB;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int c = 0; c < PL; ++c)
          k[i][c] = *reinterpret_cast<const uint4*>(st + piece_at<NV>(g + 8 * i, q + 4 * c));
      __syncwarp();  // the next turn's copies may overwrite the stage
      float acc = 0.f;
      for (int b = 0; b < rows; b += kRows) {
        if (rows > kRows) stage_rows(b);
        const int nr = min(kRows, rows - b);
        float part = 0.f;
        for (int m = 0; m < nr; m += 4) {
          float s[4][N] = {};
#pragma unroll
          for (int c = 0; c < PL; ++c) {
            float x[N][EPV];
#pragma unroll
            for (int i = 0; i < N; ++i) Vec16<T>::unpack(k[i][c], x[i]);
#pragma unroll
            for (int e = 0; e < EPV; e += 4) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(&s_q[m + j][(q + 4 * c) * EPV + e]);
#pragma unroll
                for (int i = 0; i < N; ++i) s[j][i] += x[i][e] * y.x;
#pragma unroll
                for (int i = 0; i < N; ++i) s[j][i] += x[i][e + 1] * y.y;
#pragma unroll
                for (int i = 0; i < N; ++i) s[j][i] += x[i][e + 2] * y.z;
#pragma unroll
                for (int i = 0; i < N; ++i) s[j][i] += x[i][e + 3] * y.w;
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = own_sum(s[j], q), wt = s_w[m + j];
            if (wt != 0.f && v < s_len[m + j]) part += wt * exp2f(x * a.scale_log2 - s_lse[m + j]);
          }
        }
        acc += part;
      }
      if (x0.ok && q < N) a.mass_out[x0.out] = had0 + acc;
      x0 = x1;
      had0 = had1;
    }
    u += t1 - t0;
    __syncthreads();  // the rows' places are free, and every copy has landed
  }
}

template <typename T, int D>
cudaError_t simt_t(AttnArgs a, cudaStream_t s) {
  using M = Mass<T, D>;
  const cudaError_t e =
      cudaFuncSetAttribute(mass_simt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, M::kSmem);
  if (e != cudaSuccess) return e;
  a.grid = sm_count() * M::kCtas;
  mass_simt_kernel<T, D><<<a.grid, M::kThreads, M::kSmem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_mass(const AttnArgs& a, cudaStream_t s) {
  const bool bf = a.kc.dtype == 1;
  if (mass_tc_suits(a.kc)) return launch_mass_tc(a, s);
  switch (a.kc.D) {
    case 32: return bf ? simt_t<bf16_t, 32>(a, s) : simt_t<float, 32>(a, s);
    case 64: return bf ? simt_t<bf16_t, 64>(a, s) : simt_t<float, 64>(a, s);
    case 128: return bf ? simt_t<bf16_t, 128>(a, s) : simt_t<float, 128>(a, s);
    case 256: return bf ? simt_t<bf16_t, 256>(a, s) : cudaErrorNotSupported;
  }
  return cudaErrorNotSupported;
}

}  // namespace kk
