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
//
// Measured, 28 + 4 heads of 128 bf16 dims with the Values: 11.2 K nodes (207 MB) 39.4 us,
// 5.3 TB/s; one node of 8 requests 8.2 us (11 with the host). With blocks of 8
// nodes 62 (their look-ups and sines, a chain of latencies, came 3.4 times to an
// SM), with sines as they are numbered, four lanes to a bank, 46.
#include "kk_device.cuh"
#include "kk_f32x2.cuh"
#include "kk_pdl.cuh"
#include "kk_rope.cuh"

namespace kk {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 128;
constexpr int kBatch = 32;  // nodes of a block, at most

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

template <typename T, int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeArgs a, int batch) {
  constexpr int E = Vec16<T>::kElems, LPR = D / (2 * E), RPW = 32 / LPR;  // lanes of a row, rows of a warp
  constexpr int ES = 16 / E;
  __shared__ unsigned long long s_turn[kMaxPairs];
  // [nodes][E / 2][pairs / E]: the cosines and the sines of two pairs; the lanes of a row read neighbours
  extern __shared__ float4 s_cs[];
  __shared__ long long s_slot[kBatch][2];  // byte offset of the node's slot in K and V, -1: none
  __shared__ int s_pos[kBatch];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int node0 = blockIdx.x * batch, nodes = min(batch, a.nodes - node0);
  const int pairs = a.rd / 2;
  // The position and the cache slots of node node0 + k, by one thread: a chain of four or five loads.
  auto look_up = [&](int k) {
    const int node = node0 + k;
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
      if (!ok && blockIdx.y == 0) flag_error(a.err, kErrBadIndex);
    }
    s_slot[k][0] = ks;
    s_slot[k][1] = vs;
    return pos;
  };
  // Given positions need no table: the slots are looked up by the last warp while the others are at the queries.
  const bool late = a.positions != nullptr && a.Hq > 0;
  if (tid < pairs) s_turn[tid] = turns_of(a.inv_freq[tid]);
  if (tid < nodes) {
    const int pos = late ? 0 : look_up(tid);
    s_pos[tid] = a.positions ? a.positions[node0 + tid] : pos;
  }
  __syncthreads();
  for (int i = tid; i < nodes * pairs; i += kThreads) {
    const int k = i / pairs, p = i - k * pairs;
    const unsigned long long turn = (unsigned long long)(long long)s_pos[k] * s_turn[p];
    float sn, cs;
    sincospif((float)(int)(turn >> 32) * 0x1p-31f, &sn, &cs);
    float* to = reinterpret_cast<float*>(s_cs + k * (pairs / 2) + p % E / 2 * (pairs / E) + p / E) + (p & 1);
    to[0] = cs * a.rope_scale;
    to[2] = sn * a.rope_scale;
  }
  __syncthreads();
  if (late && w == kWarps - 1 && lane < nodes) look_up(lane);
  __syncwarp();

  // the lane's two pieces of a row, and its first pair (none: past rotary_dim)
  const int j = lane % LPR, turned = a.rd / (2 * E);
  const bool rot = j < turned;
  const int p0 = HALF && rot ? j : 2 * j, p1 = HALF && rot ? j + turned : 2 * j + 1;
  // A warp takes RPW heads of one node and one kind at a time, two such chunks together so that four loads a
  // lane are under way; queries first, then Keys, then Values, each with its weights in registers.
  const int slot = lane / LPR;
  const int cq = (a.Hq + RPW - 1) / RPW, ck = (a.H + RPW - 1) / RPW;
  for (int kind = 0; kind < (a.v ? 3 : 2); ++kind) {
    const int heads = kind ? a.H : a.Hq, all = kind ? ck : cq;
    if (kind == 1 && late) __syncthreads();  // the slots
    const int per = (all + gridDim.y - 1) / gridDim.y;
    const int c0 = blockIdx.y * per, chunks = min(all, c0 + per) - c0;  // this block's share of the heads
    if (chunks <= 0) continue;
    const RopeRows& x = kind == 0 ? a.q : kind == 1 ? a.k : a.v_rows;
    const void* wt = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
    float g[2 * E];
    if (wt) {
      Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const char*>(wt) + p0 * 16), g);
      Vec16<T>::unpack(*reinterpret_cast<const uint4*>(static_cast<const char*>(wt) + p1 * 16), g + E);
    }
    int node = w / chunks, chunk = w - node * chunks;
    const int step_n = kWarps / chunks, step_c = kWarps - step_n * chunks;
    while (node < nodes) {
      uint4 u[2], v[2];
      int k[2], h[2];
      bool real[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        k[i] = node;
        h[i] = (c0 + chunk) * RPW + slot;
        real[i] = node < nodes && h[i] < heads;
        u[i] = v[i] = make_uint4(0, 0, 0, 0);
        if (real[i]) {
          const char* from = static_cast<const char*>(x.base) + ((node0 + k[i]) * x.sn + h[i] * x.sh) * ES;
          u[i] = *reinterpret_cast<const uint4*>(from + p0 * 16);
          v[i] = *reinterpret_cast<const uint4*>(from + p1 * 16);
        }
        node += step_n;
        chunk += step_c;
        if (chunk >= chunks) chunk -= chunks, ++node;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (kind != 2) {  // the same for the warp
          float f[2 * E];
          Vec16<T>::unpack(u[i], f);
          Vec16<T>::unpack(v[i], f + E);
          auto two = [&](int e) { return make_float2(f[e], f[e + 1]); };
          if (wt) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 2 * E; e += 2) sq = fma2(two(e), two(e), sq);
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
            const float s = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 2 * E; e += 2)
              set2(f + e, mul2(mul2(two(e), make_float2(s, s)), make_float2(g[e], g[e + 1])));
          }
          if (rot) {
            const float4* cs = s_cs + (k[i] < nodes ? k[i] : 0) * (pairs / 2) + j;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float4 t = cs[e / 2 * turned];
              const float2 c = make_float2(t.x, t.y), n = make_float2(t.z, t.w);
              float2 y = two(HALF ? e : 2 * e), z = two(HALF ? E + e : 2 * e + 2);
              if (!HALF) {  // as they lie: a pair each
                const float x1 = y.y;
                y.y = z.x;
                z.x = x1;
              }
              const float2 p = sub2(mul2(y, c), mul2(z, n)), q = fma2(y, n, mul2(z, c));
              if (HALF) {
                set2(f + e, p);
                set2(f + E + e, q);
              } else {
                set2(f + 2 * e, make_float2(p.x, q.x));
                set2(f + 2 * e + 2, make_float2(p.y, q.y));
              }
            }
          }
          u[i] = pack_vec<T>(f);
          v[i] = pack_vec<T>(f + E);
        }
        if (!real[i]) continue;
        auto put = [&](char* to) {
          *reinterpret_cast<uint4*>(to + p0 * 16) = u[i];
          *reinterpret_cast<uint4*>(to + p1 * 16) = v[i];
        };
        const long long n = node0 + k[i];
        if (kind == 0) {
          put(static_cast<char*>(a.q_out.base) + (n * a.q_out.sn + h[i] * a.q_out.sh) * ES);
        } else if (kind == 1) {
          if (a.k_out.base) put(static_cast<char*>(a.k_out.base) + (n * a.k_out.sn + h[i] * a.k_out.sh) * ES);
          if (a.kc && s_slot[k[i]][0] >= 0) put(static_cast<char*>(a.kc) + s_slot[k[i]][0] + h[i] * a.kH * ES);
        } else if (s_slot[k[i]][1] >= 0) {
          put(static_cast<char*>(a.vc) + s_slot[k[i]][1] + h[i] * a.vH * ES);
        }
      }
    }
  }
}

template <typename T, int D>
cudaError_t go(const RopeArgs& a, cudaStream_t s) {
  // Nodes of a block: an equal share of them for each of three blocks an SM (their look-ups and sines are a chain
  // of latencies that a block pays once), at most kBatch; few nodes: their heads are spread over blocks.
  const int sms = sm_count();
  const int batch = std::min(kBatch, (a.nodes + 3 * sms - 1) / (3 * sms)), blocks = (a.nodes + batch - 1) / batch;
  constexpr int rows = 32 / (D / (2 * Vec16<T>::kElems));  // heads of a warp
  const int split = std::max(1, std::min((a.Hq + rows - 1) / rows, sms / blocks));
  const int smem = batch * (a.rd / 2) * (int)sizeof(float2);
  const dim3 grid((unsigned)blocks, (unsigned)split);
  return launch_pdl(a.half ? rope_kernel<T, D, true> : rope_kernel<T, D, false>, grid, kThreads, smem, s, a, batch);
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
