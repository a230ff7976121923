// Attention mass: the weight every cached token received from a set of query
// rows whose lse is known,
//   mass_out = decay * mass_in + sum_i w_i sum_g [t < len_i] e^(s_igt - lse_ig)
// the score by which tokens are evicted. The products are formed again from
// the Keys (K is read once; the weights themselves are never stored). The work
// division is kk_attn.cuh's, with one unit per (request, KV head, token tile);
// a token's sum belongs to one thread, so there are no atomics. Here: float32
// caches, and bf16 ones whose layout no tensor map suits (kk_mass_tc.cu has the
// rest: 7 rows, up to 8 x 32768 tokens of 4 heads and 128 dims 41 us, with this
// kernel 156). A thread reads its token's Key once for 16 rows: 4 x 52780 float32
// tokens of 64 dims and one row (54 MB) 23 us, 2.4 TB/s; 8 x 32768 of 4 heads and
// 128 dims and 7 rows (546 MB) 316 us, 1.7 TB/s.
#include "kk_attn.cuh"

namespace kk {
namespace {

constexpr int kThreads = 128;
constexpr int kTK = 128;
constexpr int kRows = 16;  // query rows staged at a time

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) mass_simt_kernel(const AttnArgs a) {
  constexpr int EPV = Vec16<T>::kElems;
  constexpr int ES = elem_bytes<T>();
  constexpr int NV = D / EPV;
  __shared__ __align__(16) float s_q[kRows][D];
  __shared__ float s_lse[kRows], s_w[kRows];
  __shared__ int s_len[kRows];
  __shared__ long long s_place[kThreads / 32 + 4];
  const int tid = threadIdx.x;
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
    const int h = (int)udiv(u - base, rq.tiles), t = (int)(u - base - (long long)h * rq.tiles);
    const int v = t * kTK + tid;
    TokenAt at;
    const bool ok = token_at(a, r, rq, v, true, &at);
    uint4 k[NV];
    if (ok) {
      const uint4* kp = reinterpret_cast<const uint4*>(
          static_cast<const char*>(a.kc.base) +
          (a.layer * a.kc.sL + at.page * a.kc.sP + h * a.kc.sH + at.tok * a.kc.sT) * ES);
#pragma unroll
      for (int c = 0; c < NV; ++c) k[c] = kp[c];
    } else {
#pragma unroll
      for (int c = 0; c < NV; ++c) k[c] = make_uint4(0, 0, 0, 0);
    }
    float acc = 0.f;
    const int rows = rq.n * a.G;
    for (int b = 0; b < rows; b += kRows) {
      const int nr = min(kRows, rows - b);
      __syncthreads();
      for (int i = tid; i < nr * D; i += kThreads) {
        const int m = i / D, d = i - m * D, row = b + m;
        const long long x = (rq.node0 + row / a.G) * a.q_sn + (long long)(h * a.G + row % a.G) * a.q_sh + d;
        s_q[m][d] = ES == 4 ? static_cast<const float*>(a.q)[x]
                            : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.q)[x] << 16);
      }
      if (tid < nr) {
        const int row = b + tid, node = rq.node0 + row / a.G;
        const float l = a.lse[(long long)node * a.Hq + h * a.G + row % a.G];
        // a row that saw nothing gives nothing
        s_w[tid] = l == -INFINITY ? 0.f : a.row_w ? a.row_w[node] : 1.f;
        s_lse[tid] = l * 1.44269504088896341f;
        s_len[tid] = a.row_lens ? a.row_lens[node] : rq.T;
      }
      __syncthreads();
      float part = 0.f;
      for (int m = 0; m < nr; ++m) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          float x[EPV];
          Vec16<T>::unpack(k[c], x);
#pragma unroll
          for (int e = 0; e < EPV; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(&s_q[m][c * EPV + e]);
            s += x[e] * y.x;
            s += x[e + 1] * y.y;
            s += x[e + 2] * y.z;
            s += x[e + 3] * y.w;
          }
        }
        const float wt = s_w[m];
        if (v < s_len[m] && wt != 0.f) part += wt * exp2f(s * a.scale_log2 - s_lse[m]);
      }
      acc += part;
    }
    if (ok) {
      const long long x = (((long long)a.layer * a.kc.num_pages + at.page) * a.kc.H + h) * a.kc.bs + at.tok;
      const bool had = !a.old_lens || v < a.old_lens[r];
      a.mass_out[x] = (had && a.mass_in ? a.decay * a.mass_in[x] : 0.f) + acc;
    }
    u += 1;
  }
}

template <typename T, int D>
cudaError_t simt_t(AttnArgs a, cudaStream_t s) {
  a.grid = sm_count() * 4;
  mass_simt_kernel<T, D><<<a.grid, kThreads, 0, s>>>(a);
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
