// kk_qk_norm_rope: RMS norm of every query and Key head, rotation by position,
// and the write of Keys and Values into their cache slots, in one pass; bound by
// the bytes of the heads (each read once and written once).
//
// A head's row is spread over D / (2 E) lanes (E elements in 16 bytes), each
// holding the two 16-byte pieces whose elements rotate with one another: pieces
// j and j + rotary_dim / (2 E) of pairs (i, i + rotary_dim / 2), or two
// neighbours where pairs are interleaved. Rows need no exchange but the sum of
// squares, a lane turns the same pairs in every head, and both pieces are read
// and written in whole sectors. Dims past rotary_dim go through untouched.
//
// The sine and cosine of a position are made once a block for all its heads. The
// angle p * f is reduced exactly: a block turns each f into f / (2 pi) modulo 1
// as a 64-bit fixed-point number (the product with 1 / (2 pi) in two float64
// parts), and p times that, modulo 2^64, is the angle in turns whatever p is. The
// top 32 bits go to sincospi; a float32 product p * f would be off by whole
// radians at the far positions of a long context, and float64 is slow here.
#include "kk_device.cuh"
#include "kk_rope.cuh"

namespace kk {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;
constexpr int kBatch = 8;  // nodes of a block, at most

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float* f);
template <>
__device__ __forceinline__ uint4 pack_vec<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack_vec<bf16_t>(const float* f) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// f / (2 pi) modulo 1, in units of 2^-64.
__device__ __forceinline__ unsigned long long turns_of(float f) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double x = f, p = x * kHi, q = fma(x, kHi, -p) + x * kLo;
  // the fraction of p is exact; q, its remainder, is tiny
  return (unsigned long long)((p - floor(p)) * 18446744073709551616.0) +
         (unsigned long long)(long long)rint(q * 18446744073709551616.0);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, int batch) {
  constexpr int E = Vec16<T>::kElems, LPR = D / (2 * E), RPW = 32 / LPR;  // lanes of a row, rows of a warp
  constexpr int ES = 16 / E;
  __shared__ unsigned long long s_turn[kMaxPairs];
  __shared__ float2 s_cs[kBatch][kMaxPairs];
  __shared__ long long s_slot[kBatch][2];  // byte offset of the node's slot in K and V, -1: none
  __shared__ int s_pos[kBatch];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int node0 = blockIdx.x * batch, nodes = min(batch, a.nodes - node0);
  const int pairs = a.rd / 2;
  if (tid < pairs) s_turn[tid] = turns_of(a.inv_freq[tid]);
  if (tid < nodes) {
    const int node = node0 + tid;
    int pos = node;
    long long ks = -1, vs = -1;
    if (a.bt.offsets) {
      int r = node, i = 0, n = 1;  // request, the node's number in it, its nodes
      bool ok = true;
      if (a.token_off) {
        int lo = 0, hi = a.bt.R;  // the last r with token_off[r] <= node
        while (hi - lo > 1) {
          const int m = (lo + hi) >> 1;
          if (a.token_off[m] <= node) lo = m;
          else hi = m;
        }
        r = lo;
        i = node - a.token_off[r];
        n = a.token_off[r + 1] - a.token_off[r];
        ok = i >= 0 && i < n;
      }
      const int off = a.bt.offsets[r], nb = a.bt.offsets[r + 1] - off, T1 = a.bt.seq_lens[r], bs = a.bs;
      ok = ok && T1 >= n && T1 <= kMaxTokens && nb >= 0 && nb <= a.bt.max_blocks &&
           nb == (int)(((unsigned)T1 + (unsigned)bs - 1u) / (unsigned)bs);
      pos = 0;
      if (ok) {
        pos = T1 - n + i;
        const int page = a.bt.pages[off + pos / bs], o = pos % bs;
        ok = page >= 0 && page < a.num_pages;
        if (ok) {
          ks = (a.layer * a.kL + page * a.kP + o * a.kT) * ES;
          vs = (a.layer * a.vL + page * a.vP + o * a.vT) * ES;
        }
      }
      if (!ok) flag_error(a.err, kErrBadIndex);
    }
    s_slot[tid][0] = ks;
    s_slot[tid][1] = vs;
    s_pos[tid] = a.positions ? a.positions[node] : pos;
  }
  __syncthreads();
  for (int i = tid; i < nodes * pairs; i += kThreads) {
    const int k = i / pairs, p = i - k * pairs;
    const unsigned long long turn = (unsigned long long)(long long)s_pos[k] * s_turn[p];
    float sn, cs;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
    s_cs[k][p] = make_float2(cs * a.rope_scale, sn * a.rope_scale);
  }
  __syncthreads();

  // the lane's two pieces of a row, and its first pair (none: past rotary_dim)
  const int j = lane % LPR, turned = a.rd / (2 * E);
  const bool rot = j < turned;
  const int p0 = a.half && rot ? j : 2 * j, p1 = a.half && rot ? j + turned : 2 * j + 1;
  const int heads = a.Hq + a.H + (a.v ? a.H : 0), per = (heads + gridDim.y - 1) / gridDim.y;
  const int h0 = blockIdx.y * per, h1 = min(heads, h0 + per);
  if (h0 >= h1) return;
  const int rows = nodes * (h1 - h0);
  const float inv_d = 1.f / D;
  for (int row = w * RPW + lane / LPR;; row += kWarps * RPW) {
    if (__all_sync(kFull, row >= rows)) break;
    const bool real = row < rows;
    const int k = real ? row / (h1 - h0) : 0, hh = real ? h0 + row - k * (h1 - h0) : h0, node = node0 + k;
    const int kind = hh < a.Hq ? 0 : hh < a.Hq + a.H ? 1 : 2, h = hh - (kind ? a.Hq : 0) - (kind == 2 ? a.H : 0);
    const RopeRows& x = kind == 0 ? a.q : kind == 1 ? a.k : a.v_rows;
    const char* from = static_cast<const char*>(x.base) + (node * x.sn + h * x.sh) * ES;
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    if (real) {
      u = *reinterpret_cast<const uint4*>(from + p0 * 16);
      v = *reinterpret_cast<const uint4*>(from + p1 * 16);
    }
    float f[2 * E];
    Vec16<T>::unpack(u, f);
    Vec16<T>::unpack(v, f + E);
    float ss = 0.f;
    if (a.q_weight || a.k_weight) {  // the same for all lanes: rows of a warp may be of different kinds
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) ss += f[e] * f[e];
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    }
    if (kind != 2) {
      const void* wt = kind ? a.k_weight : a.q_weight;
      if (wt) {
        float g[2 * E];
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const char*>(wt) + p0 * 16), g);
        Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const char*>(wt) + p1 * 16), g + E);
        const float s = rsqrtf(ss * inv_d + a.eps);
#pragma unroll
        for (int e = 0; e < 2 * E; ++e) f[e] = f[e] * s * g[e];
      }
      if (rot) {
        const float2* cs = s_cs[k] + j * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float2 t = cs[e];
          float* p = a.half ? f + e : f + 2 * e;
          float* q = a.half ? f + E + e : f + 2 * e + 1;
          const float y = *p, z = *q;
          *p = y * t.x - z * t.y;
          *q = z * t.x + y * t.y;
        }
      }
      u = pack_vec<T>(f);
      v = pack_vec<T>(f + E);
    }
    if (!real) continue;
    auto put = [&](char* to) {
      *reinterpret_cast<uint4*>(to + p0 * 16) = u;
      *reinterpret_cast<uint4*>(to + p1 * 16) = v;
    };
    if (kind == 0) put(static_cast<char*>(a.q_out.base) + (node * a.q_out.sn + h * a.q_out.sh) * ES);
    if (kind == 1 && a.k_out.base) put(static_cast<char*>(a.k_out.base) + (node * a.k_out.sn + h * a.k_out.sh) * ES);
    if (kind == 1 && a.kc && s_slot[k][0] >= 0) put(static_cast<char*>(a.kc) + s_slot[k][0] + h * a.kH * ES);
    if (kind == 2 && s_slot[k][1] >= 0) put(static_cast<char*>(a.vc) + s_slot[k][1] + h * a.vH * ES);
  }
}

template <typename T, int D>
cudaError_t go(const RopeArgs& a, cudaStream_t s) {
  const int sms = sm_count(), heads = a.Hq + 2 * a.H;
  // nodes of a block: as many as leave every SM several blocks; few nodes: their heads are spread over blocks
  int batch = kBatch;
  while (batch > 1 && (long long)((a.nodes + batch - 1) / batch) < 4ll * sms) batch >>= 1;
  constexpr int rows = kWarps * (32 / (D / (2 * Vec16<T>::kElems)));
  const int blocks = (a.nodes + batch - 1) / batch;
  int split = std::max(1, std::min((heads + rows - 1) / rows * batch, sms / blocks));
  split = std::min(split, heads);
  rope_kernel<T, D><<<dim3((unsigned)blocks, (unsigned)split), kThreads, 0, s>>>(a, batch);
  return cudaGetLastError();
}
template <typename T>
cudaError_t go_t(const RopeArgs& a, cudaStream_t s) {
  switch (a.D) {
    case 32: return go<T, 32>(a, s);
    case 64: return go<T, 64>(a, s);
    case 128: return go<T, 128>(a, s);
    case 256: return go<T, 256>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t s) {
  return a.f32 ? go_t<float>(a, s) : go_t<bf16_t>(a, s);
}

}  // namespace kk
