// The pieces of the attention over an 8-bit cache: codes widened to matrix operands,
// where tokens lie, and the state of a warp's query rows.
//
// A product's operands (m16n8k16): tokens are the M axis of S^T = K Q^T and dims
// that of O^T = V^T P^T, query rows the N axis. Lane 4g + t4 holds, of K, four dims
// of tokens g and g + 8 a step; of V, two dims of tokens 2 t4, 2 t4 + 1, 2 t4 + 8 and
// 2 t4 + 9; of results, rows 2 t4 and 2 t4 + 1 of tokens (dims) g and g + 8. The axis a
// product sums over, and the dims of O, may be in any order as long as both
// operands agree, so that a lane takes whole words of codes.
#pragma once
#include <cfloat>

#include "kk_attn.cuh"
#include "kk_f32x2.cuh"

namespace kk {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr float kNone = -FLT_MAX;  // a reference before the first score, below every finite one
constexpr float kLift = 6.f;     // a weight is below 2^(6 + 8) * 2 (a scale's mantissa): float16 holds 65504

// Two e4m3 codes (the low or the high half of a word) as float16, exactly.
__device__ __forceinline__ uint32_t widen(uint32_t w, int half) {
  uint32_t r;
  const uint16_t x = (uint16_t)(half ? w >> 16 : w);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The transpose of an 8 x 8 tile of 16-bit values (lane 4g + t holds row g, columns 2t and 2t + 1).
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_full16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// N consecutive words of shared memory.
template <int N>
__device__ __forceinline__ void lds(uint32_t (&x)[N], const unsigned char* p) {
  if constexpr (N == 4) {
    const uint4 y = *reinterpret_cast<const uint4*>(p);
    x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
  } else if constexpr (N == 2) {
    const uint2 y = *reinterpret_cast<const uint2*>(p);
    x[0] = y.x, x[1] = y.y;
  } else {
    x[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4 : 0) : "memory");
}

// A finite scale as m * 2^e, |m| < 2.
__device__ __forceinline__ void split_scale(float x, float* e, float* m) {
  const uint32_t b = __float_as_uint(x), f = (b >> 23) & 0xFFu;
  *e = f ? (float)((int)f - 127) : -126.f;
  *m = f ? __uint_as_float((b & 0x807FFFFFu) | 0x3F800000u) : x * 0x1p126f;
}

// What a warp loads next: 16 slots from slot o of `page`, the first n of which hold a token (PG: block_size is
// a multiple of 16, so they lie in one page), or the token of a lane's own number (n: 0 or 1).
struct Group {
  int page, o, n;
};
// Where that is: slot v of the request's context, slot o of its block b. It moves on by a tile at a time.
struct Cursor {
  int v, b, o;
  __device__ __forceinline__ Cursor(int slot, int bs) : v(slot), b(slot / bs), o(slot - slot / bs * bs) {}
  // n slots on: n = nb * bs + no
  __device__ __forceinline__ void move(int n, int nb, int no, int bs) {
    v += n;
    b += nb;
    o += no;
    if (o >= bs) o -= bs, ++b;
  }
};
template <bool PG>
__device__ __forceinline__ Group find_group(const AttnArgs& a, int r, const AttnReq& rq, const Cursor& c) {
  Group x = {0, 0, 0};
  if (c.v >= rq.ctx) return x;
  int left = rq.T - c.v;
  if (a.sel_pages) {
    const long long at = (long long)r * a.selK + c.b;
    const int logical = a.sel_logical[at];
    x.page = a.sel_pages[at];
    const long long first = (long long)logical * a.kc.bs;
    if (logical < 0 || first >= rq.T) {
      flag_error(a.err, kErrBadIndex);
      x.page = 0;
      return x;
    }
    left = (int)min((long long)rq.T - first - c.o, 16ll);
  } else {
    x.page = a.bt.pages[rq.off + c.b];
  }
  if (x.page < 0 || x.page >= a.kc.num_pages) {
    flag_error(a.err, kErrBadIndex);
    x.page = 0;
    return x;
  }
  x.o = c.o;
  x.n = max(0, min(left, PG ? 16 : 1));
  return x;
}

// First dim of the pair that accumulator tile n holds of lane group g.
template <int D>
__device__ __forceinline__ int dim_of(int n, int g) {
  return D == 256 ? (n >> 3) * 128 + g * 16 + (n & 7) * 2 : g * (D / 8) + n * 2;
}

// The query rows of an item as they are, [M][D] bf16, zeros past the last one.
template <int D, int M>
__device__ __forceinline__ void stage_queries(const AttnArgs& a, const AttnReq& rq, int h, int row0, int rows,
                                              unsigned char* raw) {
  for (int i = threadIdx.x; i < M * (D / 8); i += kThreads) {
    const int m = i / (D / 8), c = i - m * (D / 8), row = row0 + m;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (m < rows)
      x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (rq.node0 + row / a.G) * a.q_sn +
                                          (long long)(h * a.G + row % a.G) * a.q_sh + c * 8);
    *reinterpret_cast<uint4*>(raw + m * D * 2 + c * 16) = x;
  }
}

// Eight staged rows as float16 operands: a row's largest element is brought to [2^14, 2^15) by a power of two, so that
// what float16 cannot hold of a row is below 2^-39 of it. Step j's four dims of lane t4 are those of word j of the
// codes it reads. qf: what the scores of rows 2 t4 and 2 t4 + 1 are multiplied with.
template <int D>
__device__ __forceinline__ void query_operands(const unsigned char* raw, float scale_log2, uint2 (&q)[D / 16],
                                               float (&qf)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const uint16_t* row = reinterpret_cast<const uint16_t*>(raw) + g * D;
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    q[j] = *reinterpret_cast<const uint2*>(row + (D >= 64 ? (j >> 2) * 64 + t4 * 16 + (j & 3) * 4 : t4 * 8 + j * 4));
    top = max(top, max(max(q[j].x & 0x7FFFu, (q[j].x >> 16) & 0x7FFFu),
                       max(q[j].y & 0x7FFFu, (q[j].y >> 16) & 0x7FFFu)));
  }
  top = max(top, __shfl_xor_sync(kFull, top, 1));
  top = max(top, __shfl_xor_sync(kFull, top, 2));
  const int e = (int)(top >> 7);  // the exponent field; 0xFF: not finite, which stays so
  const int sh = e == 0xFF ? 0 : min(max(e - 127 - 14, -110), 113);
  const float down = __uint_as_float((uint32_t)(127 - sh) << 23);  // 2^-sh, sh in [-110, 113]
#pragma unroll
  for (int j = 0; j < D / 16; ++j)
    q[j] = make_uint2(pack_f16(bf16_lo(q[j].x) * down, bf16_hi(q[j].x) * down),
                      pack_f16(bf16_lo(q[j].y) * down, bf16_hi(q[j].y) * down));
  const float f = scale_log2 * __uint_as_float((uint32_t)(127 + sh) << 23);
  qf[0] = __shfl_sync(kFull, f, t4 * 8);
  qf[1] = __shfl_sync(kFull, f, t4 * 8 + 4);
}

// A warp's 8 NT query rows: accumulators, references and sums. ref_s: the reference of the sum of weights; gap: how far
// the other one, of weight times the Values' scale, lies above it. Exponents come from differences to ref_s alone, which
// are small where they matter however large the scores are.
template <int D, int NT>
struct Rows {
  static constexpr int KS = D / 16;
  float o[NT][KS][4], ref_s[NT][2], gap[NT][2], sum[NT][2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int n = 0; n < KS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][n][e] = 0.f;
      ref_s[nt][0] = ref_s[nt][1] = kNone;
      gap[nt][0] = gap[nt][1] = sum[nt][0] = sum[nt][1] = 0.f;
    }
  }

  // Scores of 16 tokens from their products: times the rows' factors and the Keys' scales; ONE: the tokens share a
  // page. Places without a token are hidden whatever they hold.
  template <bool ONE>
  __device__ __forceinline__ void score(float (&s)[NT][4], const float (&qf)[NT][2], float ks0, float ks1,
                                        uint32_t live) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 f0 = mul2(make_float2(qf[nt][0], qf[nt][1]), make_float2(ks0, ks0));
      const float2 f1 = ONE ? f0 : mul2(make_float2(qf[nt][0], qf[nt][1]), make_float2(ks1, ks1));
      set2(&s[nt][0], mul2(make_float2(s[nt][0], s[nt][1]), f0));
      set2(&s[nt][2], mul2(make_float2(s[nt][2], s[nt][3]), f1));
    }
    if (live == 0xFFFFu) return;
    const bool see0 = (live >> g) & 1, see1 = (live >> (g + 8)) & 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = (e < 2 ? see0 : see1) ? s[nt][e] : -INFINITY;
  }

  // Moves the references of rows whose scores (N groups of 16 tokens) passed them; lv: the exponent of the Values'
  // scale of a group's tokens g and g + 8 (ONE: the same).
  template <bool ONE, int N>
  __device__ __forceinline__ void settle(const float (&s)[N][NT][4], const float (&lv)[N][2]) {
    bool rise = false;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 r = make_float2(ref_s[nt][0], ref_s[nt][1]);
        const float2 top = ONE ? make_float2(fmaxf(s[i][nt][0], s[i][nt][2]), fmaxf(s[i][nt][1], s[i][nt][3]))
                               : make_float2(s[i][nt][0], s[i][nt][1]);
        const float2 p = sub2(top, r);
        rise |= p.x > 8.f + fminf(0.f, gap[nt][0] - lv[i][0]);
        rise |= p.y > 8.f + fminf(0.f, gap[nt][1] - lv[i][0]);
        if (!ONE) {
          const float2 q = sub2(make_float2(s[i][nt][2], s[i][nt][3]), r);
          rise |= q.x > 8.f + fminf(0.f, gap[nt][0] - lv[i][1]);
          rise |= q.y > 8.f + fminf(0.f, gap[nt][1] - lv[i][1]);
        }
      }
    if (!__any_sync(kFull, rise)) return;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float ms = ref_s[nt][e], mv = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) ms = fmaxf(ms, fmaxf(s[i][nt][e], s[i][nt][e + 2]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) ms = fmaxf(ms, __shfl_xor_sync(kFull, ms, x));
#pragma unroll
        for (int i = 0; i < N; ++i)
          mv = fmaxf(mv, fmaxf(s[i][nt][e] - ms + lv[i][0], s[i][nt][e + 2] - ms + lv[i][1]));
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) mv = fmaxf(mv, __shfl_xor_sync(kFull, mv, x));
        const float down = ref_s[nt][e] - ms, old = gap[nt][e] + down;
        mv = fmaxf(mv, old);
        sum[nt][e] *= ex2(down);
        f[e] = ex2(old - mv);
        ref_s[nt][e] = ms;
        gap[nt][e] = mv;
      }
#pragma unroll
      for (int n = 0; n < KS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][n][e] *= f[e & 1];
    }
  }

  // Weights of 16 tokens, added to the sums and turned into operands (vm: the Values' scales' mantissas).
  __device__ __forceinline__ void weigh(const float (&s)[NT][4], const float (&lv)[2], const float (&vm)[2],
                                        uint32_t (&b)[2][NT]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float2 l = make_float2(sum[nt][0], sum[nt][1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float2 y = make_float2(s[nt][2 * x], s[nt][2 * x + 1]);
        const float2 p = add2(y, make_float2(-ref_s[nt][0], -ref_s[nt][1]));
        l = add2(l, make_float2(ex2(p.x), ex2(p.y)));
        const float up = lv[x] + kLift;
        const float2 q = add2(p, make_float2(up - gap[nt][0], up - gap[nt][1]));
        const float2 z = mul2(make_float2(ex2(q.x), ex2(q.y)), make_float2(vm[x], vm[x]));
        b[x][nt] = turn(pack_f16(z.x, z.y));  // the weights' one rounding: float16 feeds the product
      }
      set2(sum[nt], l);
    }
  }

  // Drafted nodes j0 .. j0 + 15, bf16, straight from where they lie. raw: the rows' staged queries, the first of
  // them row `row0` of the request.
  __device__ __forceinline__ void drafts(const AttnArgs& a, const AttnReq& rq, int h, const unsigned char* raw,
                                         int row0, int j0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    float s[1][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][nt][e] = 0.f;
    const uint16_t* dk = static_cast<const uint16_t*>(a.dk) + rq.node0 * a.dk_sn + h * a.dk_sh;
    const uint16_t* dv = static_cast<const uint16_t*>(a.dv) + rq.node0 * a.dv_sn + h * a.dv_sh;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 x = make_uint4(0, 0, 0, 0), y = x;
      if (j0 + g < rq.n) x = *reinterpret_cast<const uint4*>(dk + (j0 + g) * a.dk_sn + i * 32 + t4 * 8);
      if (j0 + g + 8 < rq.n) y = *reinterpret_cast<const uint4*>(dk + (j0 + g + 8) * a.dk_sn + i * 32 + t4 * 8);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 b = *reinterpret_cast<const uint4*>(raw + ((nt * 8 + g) * D + i * 32 + t4 * 8) * 2);
        mma<true>(s[0][nt], x.x, y.x, x.y, y.y, b.x, b.y);
        mma<true>(s[0][nt], x.z, y.z, x.w, y.w, b.z, b.w);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = row0 + nt * 8 + 2 * t4 + (e & 1), j = j0 + (e < 2 ? g : g + 8);
        const bool see = j < rq.n && row < rq.n * a.G && sees(a, rq, row / a.G, j);
        s[0][nt][e] = see ? s[0][nt][e] * a.scale_log2 : -INFINITY;
      }
    const float lv[1][2] = {{0.f, 0.f}};
    settle<true>(s, lv);
    uint32_t b0[NT], b1[NT];
    float p[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = s[0][nt][e] - ref_s[nt][e & 1];
        sum[nt][e & 1] += ex2(x);
        p[nt][e] = ex2(x + (kLift - gap[nt][e & 1]));
      }
      b0[nt] = turn(pack_bf16(p[nt][0], p[nt][1]));  // bf16, as the Values they meet
      b1[nt] = turn(pack_bf16(p[nt][2], p[nt][3]));
    }
    // A Value that is not finite must not meet the zero weights of the nodes that do not see it: it is
    // taken out of the product and added for the nodes that do.
    bool odd = false;
    constexpr int VP = D >= 64 ? 4 : 2;  // words (of two dims) read at once
#pragma unroll
    for (int i = 0; i < KS / VP; ++i) {
      // the thread's dims, as the codes' products have them: D/8 in a row (D = 256: 16 and 16)
      const int d = dim_of<D>(i * VP, g);
      uint32_t x[4][VP];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = j0 + 2 * t4 + (k & 1) + (k >> 1) * 8;
#pragma unroll
        for (int c = 0; c < VP; ++c) x[k][c] = 0;
        if (j < rq.n) {
          const uint16_t* v = dv + j * a.dv_sn + d;
          if constexpr (VP == 4) {
            const uint4 y = *reinterpret_cast<const uint4*>(v);
            x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(v);
            x[k][0] = y.x, x[k][1] = y.y;
          }
#pragma unroll
          for (int c = 0; c < VP; ++c) {
            if ((x[k][c] & 0x7F800000u) == 0x7F800000u) x[k][c] &= 0x0000FFFFu, odd = true;
            if ((x[k][c] & 0x00007F80u) == 0x00007F80u) x[k][c] &= 0xFFFF0000u, odd = true;
          }
        }
      }
#pragma unroll
      for (int c = 0; c < VP; ++c) {
        const uint32_t a0 = __byte_perm(x[0][c], x[1][c], 0x5410), a1 = __byte_perm(x[0][c], x[1][c], 0x7632);
        const uint32_t a2 = __byte_perm(x[2][c], x[3][c], 0x5410), a3 = __byte_perm(x[2][c], x[3][c], 0x7632);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma<true>(o[nt][i * VP + c], a0, a1, a2, a3, b0[nt], b1[nt]);
      }
    }
    if (__any_sync(kFull, odd)) {
#pragma unroll 1
      for (int k = 0; k < 16 && j0 + k < rq.n; ++k)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w0 = __shfl_sync(kFull, p[nt][e], (k & 7) * 4 + t4);
            const float w1 = __shfl_sync(kFull, p[nt][e + 2], (k & 7) * 4 + t4);
            const int row = row0 + nt * 8 + 2 * t4 + e;
            if (row >= rq.n * a.G || !sees(a, rq, row / a.G, j0 + k)) continue;
#pragma unroll
            for (int n = 0; n < KS; ++n)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int d = dim_of<D>(n, g) + x;
                const uint32_t v = dv[(j0 + k) * a.dv_sn + d];
                if ((v & 0x7F80u) == 0x7F80u) o[nt][n][x * 2 + e] += (k < 8 ? w0 : w1) * __uint_as_float(v << 16);
              }
          }
    }
  }

  // Leaves the rows for the join: [parts][M][D] accumulators in terms of ref_s, maxima, sums; this warp's are rows m0
  // on of part p.
  __device__ __forceinline__ void leave(float* join, int parts, int p, int M, int m0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    float* jm = join + parts * M * D;
    float* jl = jm + parts * M;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = m0 + nt * 8 + 2 * t4 + e;
        float l = sum[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(kFull, l, x);
        if (g == 0) {
          jm[p * M + m] = ref_s[nt][e] == kNone ? -INFINITY : ref_s[nt][e];
          jl[p * M + m] = l;
        }
        // In two factors, of which the second is 1 but for Values below 2^-94: their scales and the lift may together be
        // below what one power of two holds.
        const float x = gap[nt][e] - kLift;
        const float f = ex2(fmaxf(x, -100.f)), f2 = ex2(fminf(x + 100.f, 0.f));
#pragma unroll
        for (int n = 0; n < KS; ++n)
          *reinterpret_cast<float2*>(join + (p * M + m) * D + dim_of<D>(n, g)) =
              make_float2(o[nt][n][e] * f * f2, o[nt][n][e + 2] * f * f2);
      }
  }
};

// Joins what the warps left of an item's rows and writes them out, or to the CTA's slot `part` of the workspace.
template <int D, int M, int P>
__device__ __forceinline__ void finish_rows(const AttnArgs& a, const AttnReq& rq, int h, int row0, int rows, bool whole,
                                            const float* join, float* part) {
  const float* jm = join + P * M * D;
  const float* jl = jm + P * M;
  for (int i = threadIdx.x; i < rows * (D / 4); i += kThreads) {
    const int m = i / (D / 4), d = (i - m * (D / 4)) * 4;
    float mm = jm[m];
#pragma unroll
    for (int x = 1; x < P; ++x) mm = fmaxf(mm, jm[x * M + m]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < P; ++x) {
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
}

}  // namespace
}  // namespace kk
