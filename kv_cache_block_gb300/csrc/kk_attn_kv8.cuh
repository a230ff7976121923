// kk_tree_attn_kv8: attention over a cache of e4m3 codes with a scale for each
// page and KV head, K = code * k_scale, V = code * v_scale; bound by the bytes of
// the codes.
//
// Four warps share an item's rows (M = 8, 16 or 32) and take 16 tokens each of
// every 64-token tile, streamed through a ring of shared-memory stages of their
// own as in kk_attn_mma.cu. Tokens are the M axis of the products (S^T = K Q^T,
// O^T = V^T P^T with m16n8k16 matrix instructions), query rows the N axis: a
// decode token's group of at most 8 rows fills it, where rows along M would
// leave half of 16 empty, and every 16 x 16 codes cost one instruction.
//
// e4m3 values are exact in float16, so codes are widened two at a time and
// multiplied as float16; a scale never meets the products, it multiplies the
// score (K) or the weight (V) of its page. The axes a product sums over and the
// dims of O may be in any order as long as both operands agree, so a thread
// reads whole words of codes: for K four dims of a token feed a whole step; for
// V the bytes of two tokens are interleaved (prmt) and widened into an operand
// register. No ldmatrix, no transposed copy; the weights, which come out of the
// first product with tokens along the wrong axis, are turned by movmatrix.
//
// Softmax. Two references a row (log2 domain): one for the sum of weights, 2^(s -
// ref_s) in float32, one for what multiplies the codes of V, 2^(s - ref_v + 6) *
// v_scale, which has to fit float16 whatever the pages' scales are. Both are
// left alone until a score passes one by 2^8 (one vote a step); until then sums
// below 2^8 cost nothing and no reduction over lanes is needed.
#pragma once
#include "kk_attn.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
// 16-token groups of a warp's share of a tile: two while registers allow, so that two chains of products are under
// way and what a step costs besides them is paid once for 32 tokens.
template <int D, int NT>
__host__ __device__ constexpr int kv8_groups() {
  return NT <= 2 && D <= 128 ? 2 : 1;
}
constexpr float kNone = -1e30f;                    // a reference before the first score
constexpr float kLift = 6.f;  // a weight is below 2^(6 + 8) * 2 (a scale's mantissa): float16 holds 65504

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
// Two float32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ void set2(float* p, float2 x) { p[0] = x.x, p[1] = x.y; }
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

// Byte offset of byte x (a multiple of 4) of token `row` in a stage's K or V: 16-byte pieces are
// exchanged so that the eight lanes of a quarter warp that read together (K: two tokens' four
// pieces; V: two pieces of four tokens two apart) fall into different banks.
template <int D>
__device__ __forceinline__ uint32_t at_k(int row, int x) {
  return D >= 128 ? row * D + (x ^ ((row & 1) << 6)) : row * D + x;
}
template <int D>
__device__ __forceinline__ uint32_t at_v(int row, int x) {
  return D >= 64 ? ((row * D + x) ^ (((row >> 1) & 3) << 5)) : row * D + x;
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

template <int D, int NT>
__host__ __device__ constexpr int kv8_stages() {
  return (D >= 128 ? 4 : D == 64 ? 6 : 8) / kv8_groups<D, NT>() - (D == 256 || NT == 4 ? 1 : 0);
}
template <int D, int NT>
struct Kv8Smem {
  static constexpr int M = NT * 8, S = kv8_stages<D, NT>(), kTok = 16 * kv8_groups<D, NT>(), kStage = kTok * D * 2;
  static constexpr int ring = kWarps * S * kStage, join = kWarps * M * (D + 2) * 4;
  static constexpr int scales = ring > join ? ring : join;       // [warps][stages][K, V][kTok] floats
  static constexpr int raw = scales + kWarps * S * 2 * kTok * 4;  // queries as they are, bf16 [M][D]
  static constexpr int frag = raw + M * D * 2;                   // and as float16 operands [NT][D/16][32 lanes]
  static constexpr int qf = frag + M * D * 2;                    // [M] what the scores are multiplied with
  static constexpr int bytes = qf + M * 4;
};

template <int D, int NT>
constexpr int kv8_blocks() {
  return NT == 1 ? (D < 128 ? 4 : D == 128 ? 3 : 2) : NT == 2 ? (D <= 128 ? 3 : 2) : 2;
}

template <int D, int NT, bool PG>
__global__ void __launch_bounds__(kThreads, (kv8_blocks<D, NT>())) attn_kv8_kernel(const AttnArgs a) {
  using Sm = Kv8Smem<D, NT>;
  constexpr int M = NT * 8, KS = D / 16, S = Sm::S, U = kv8_groups<D, NT>(), kTok = Sm::kTok, kTK = kTok * kWarps;
  constexpr bool kQReg = NT * D <= 256;  // query operands stay in registers
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_place[kWarps + 4];
  __shared__ uint32_t s_ok[kWarps][S];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  unsigned char* ring = smem + w * S * Sm::kStage;
  const uint32_t ring_at = smem_u32(ring);
  float* sc = reinterpret_cast<float*>(smem + Sm::scales) + w * S * 2 * kTok;
  const uint32_t sc_at = smem_u32(sc);
  uint2* frag = reinterpret_cast<uint2*>(smem + Sm::frag);
  float* qf_s = reinterpret_cast<float*>(smem + Sm::qf);
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

    // Copies a share of a tile (U groups of 16 tokens of K and V, their scales) into stage st. A lane copies the
    // pieces c of rows sub, sub + RI, ...; what does not change over the tiles is worked out here.
    constexpr int CH = D / 16, RI = 32 / CH, NI = 16 / RI > 0 ? 16 / RI : 1;
    const int c = lane % CH, sub = lane / CH;
    const char* k_lane = static_cast<const char*>(a.kc.base) + a.layer * a.kc.sL + h * a.kc.sH + c * 16 + (PG ? sub * a.kc.sT : 0);
    const char* v_lane = static_cast<const char*>(a.vc.base) + a.layer * a.vc.sL + h * a.vc.sH + c * 16 + (PG ? sub * a.vc.sT : 0);
    const long long s_at = (long long)a.layer * a.kc.num_pages * a.kc.H + h;
    constexpr int NG = PG ? U : 1;  // groups a lane knows: all of the share, or (its own token) one
    auto load = [&](const Group (&x)[NG], int st, bool on) {
      const uint32_t kst = ring_at + st * Sm::kStage, vst = kst + kTok * D, sst = sc_at + st * (2 * kTok * 4);
      uint32_t live = 0;
      if constexpr (PG) {
        if (on) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int n = x[i].n;
            live |= ((1u << n) - 1u) << (16 * i);
            const char* k = k_lane + x[i].page * a.kc.sP + x[i].o * a.kc.sT;
            const char* v = v_lane + x[i].page * a.vc.sP + x[i].o * a.vc.sT;
            if (n == 16) {
#pragma unroll
              for (int j = 0; j < NI; ++j) {
                cp_full16(kst + at_k<D>(i * 16 + j * RI + sub, c * 16), k);
                cp_full16(vst + at_v<D>(i * 16 + j * RI + sub, c * 16), v);
                k += RI * a.kc.sT;
                v += RI * a.vc.sT;
              }
            } else {
#pragma unroll
              for (int j = 0; j < NI; ++j) {
                const bool real = j * RI + sub < n;
                cp_async16(kst + at_k<D>(i * 16 + j * RI + sub, c * 16), real ? k : k_lane, real);
                cp_async16(vst + at_v<D>(i * 16 + j * RI + sub, c * 16), real ? v : v_lane, real);
                k += RI * a.kc.sT;
                v += RI * a.vc.sT;
              }
            }
            if (lane < 2)
              cp_async4(sst + (lane * kTok + i) * 4, (lane ? a.v_scale : a.k_scale) + s_at + x[i].page * a.kc.H, n > 0);
          }
        }
      } else {
        live = __ballot_sync(kFull, on && x[0].n > 0);
        if (kTok == 16) live &= 0xFFFFu;
        const long long ko = x[0].page * a.kc.sP + x[0].o * a.kc.sT, vo = x[0].page * a.vc.sP + x[0].o * a.vc.sT;
        if (on) {
#pragma unroll
          for (int j = 0; j < NI * U; ++j) {
            const int row = j * RI + sub;
            const char* k = k_lane + __shfl_sync(kFull, ko, row);
            const char* v = v_lane + __shfl_sync(kFull, vo, row);
            cp_async16(kst + at_k<D>(row, c * 16), k, (live >> row) & 1);
            cp_async16(vst + at_v<D>(row, c * 16), v, (live >> row) & 1);
          }
          const long long at = s_at + (long long)x[0].page * a.kc.H;
          if (lane < kTok) {
            cp_async4(sst + lane * 4, a.k_scale + at, x[0].n > 0);
            cp_async4(sst + (kTok + lane) * 4, a.v_scale + at, x[0].n > 0);
          }
        }
      }
      cp_commit();
      if (lane == 0) s_ok[w][st] = live;
    };

    // the first tiles' copies go out before the queries are read
    const int tc = min(t1, rq.tiles_c);  // tiles of cached tokens end here
    const int bs = a.kc.bs, tile_b = kTK / bs, tile_o = kTK - tile_b * bs;
    Cursor at(t0 * kTK + w * kTok + (PG ? 0 : lane & (kTok - 1)), bs);
    auto find = [&](Group (&x)[NG]) {
      Cursor y = at;
      x[0] = find_group<PG>(a, r, rq, y);
#pragma unroll
      for (int i = 1; i < NG; ++i) {
        y.move(16, 0, 16, bs);
        x[i] = find_group<PG>(a, r, rq, y);
      }
    };
    Group nx[NG] = {};
    if (t0 < tc) find(nx);
#pragma unroll 1
    for (int st = 0; st < S - 1; ++st) {
      load(nx, st, t0 + st < tc);
      at.move(kTK, tile_b, tile_o, bs);
      if (t0 + st + 1 < tc) find(nx);
    }
    for (int i = tid; i < M * (D / 8); i += kThreads) {
      const int m = i / (D / 8), c = i - m * (D / 8), row = row0 + m;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (m < rows)
        x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (rq.node0 + row / a.G) * a.q_sn +
                                            (long long)(h * a.G + row % a.G) * a.q_sh + c * 8);
      *reinterpret_cast<uint4*>(smem + Sm::raw + m * D * 2 + c * 16) = x;
    }
    __syncthreads();
    // Queries as float16 operands: the row's largest element is brought to [2^14, 2^15) by a power of two, so
    // that what float16 cannot hold of a row is below 2^-39 of it. Step j's four dims of thread t4 are those of
    // word j of the codes it reads.
    for (int nt = w; nt < NT; nt += kWarps) {
      const uint16_t* qr = reinterpret_cast<const uint16_t*>(smem + Sm::raw) + (nt * 8 + g) * D;
      auto dim = [&](int j) { return D >= 64 ? (j >> 2) * 64 + t4 * 16 + (j & 3) * 4 : t4 * 8 + j * 4; };
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(qr + dim(j));
        top = max(max(top, max(x.x & 0x7FFFu, (x.x >> 16) & 0x7FFFu)), max(x.y & 0x7FFFu, (x.y >> 16) & 0x7FFFu));
      }
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      const int e = (int)(top >> 7);  // the exponent field; 0xFF: not finite, which stays so
      const int sh = e == 0xFF ? 0 : min(max(e - 127 - 14, -110), 113);
      const float down = __uint_as_float((uint32_t)(127 - sh) << 23);  // 2^-sh, sh in [-110, 113]
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const uint2 x = *reinterpret_cast<const uint2*>(qr + dim(j));
        frag[(nt * KS + j) * 32 + lane] = make_uint2(pack_f16(bf16_lo(x.x) * down, bf16_hi(x.x) * down),
                                                     pack_f16(bf16_lo(x.y) * down, bf16_hi(x.y) * down));
      }
      if (t4 == 0) qf_s[nt * 8 + g] = a.scale_log2 * __uint_as_float((uint32_t)(127 + sh) << 23);
    }
    __syncthreads();
    uint2 qr[kQReg ? NT : 1][kQReg ? KS : 1];
    if constexpr (kQReg) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < KS; ++j) qr[nt][j] = frag[(nt * KS + j) * 32 + lane];
    }
    float qf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      qf[nt][0] = qf_s[nt * 8 + 2 * t4];
      qf[nt][1] = qf_s[nt * 8 + 2 * t4 + 1];
    }

    float o[NT][KS][4], ref_s[NT][2], ref_v[NT][2], l_run[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int n = 0; n < KS; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][n][e] = 0.f;
      ref_s[nt][0] = ref_s[nt][1] = ref_v[nt][0] = ref_v[nt][1] = kNone;
      l_run[nt][0] = l_run[nt][1] = 0.f;
    }
    // Moves the references of rows whose scores passed them; lv: the exponent of the Values' scale of a group's
    // tokens g and g + 8 (PG: the same).
    auto settle = [&](const auto& s, const auto& lv) {
      constexpr int N = sizeof(s) / sizeof(s[0]);
      bool rise = false;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = PG ? fmaxf(s[i][nt][e], s[i][nt][e + 2]) : s[i][nt][e];
            rise |= top > 8.f + fminf(ref_s[nt][e], ref_v[nt][e] - lv[i][0]);
            if (!PG) rise |= s[i][nt][e + 2] > 8.f + fminf(ref_s[nt][e], ref_v[nt][e] - lv[i][1]);
          }
      if (!__any_sync(kFull, rise)) return;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float ms = -INFINITY, mv = -INFINITY;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            ms = fmaxf(ms, fmaxf(s[i][nt][e], s[i][nt][e + 2]));
            mv = fmaxf(mv, fmaxf(s[i][nt][e] + lv[i][0], s[i][nt][e + 2] + lv[i][1]));
          }
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) {
            ms = fmaxf(ms, __shfl_xor_sync(kFull, ms, x));
            mv = fmaxf(mv, __shfl_xor_sync(kFull, mv, x));
          }
          ms = fmaxf(ms, ref_s[nt][e]);
          mv = fmaxf(mv, ref_v[nt][e]);
          l_run[nt][e] *= ex2(ref_s[nt][e] - ms);
          f[e] = ex2(ref_v[nt][e] - mv);
          ref_s[nt][e] = ms;
          ref_v[nt][e] = mv;
        }
#pragma unroll
        for (int n = 0; n < KS; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][n][e] *= f[e & 1];
      }
    };

    int st = 0;
#pragma unroll 1
    for (int t = t0; t < t1; ++t) {
      cp_wait<S - 2>();
      __syncwarp();
      {  // refill the stage read in the last turn
        load(nx, st == 0 ? S - 1 : st - 1, t + S - 1 < tc);
        at.move(kTK, tile_b, tile_o, bs);
        if (t + S < tc) find(nx);
      }
      if (t < rq.tiles_c) {
        const unsigned char *kst = ring + st * Sm::kStage, *vst = kst + kTok * D;
        const uint32_t live = s_ok[w][st];
        float s[U][NT][4];
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][nt][e] = 0.f;
        constexpr int KW = D >= 64 ? 4 : 2;  // words of codes read at once
#pragma unroll
        for (int i = 0; i < KS / KW; ++i) {
          uint32_t x[U][KW], y[U][KW];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            lds<KW>(x[k], kst + at_k<D>(k * 16 + g, i * 64 + t4 * KW * 4));
            lds<KW>(y[k], kst + at_k<D>(k * 16 + g + 8, i * 64 + t4 * KW * 4));
          }
#pragma unroll
          for (int c = 0; c < KW; ++c)
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const uint32_t a0 = widen(x[k][c], 0), a1 = widen(y[k][c], 0), a2 = widen(x[k][c], 1), a3 = widen(y[k][c], 1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint2 b;
                if constexpr (kQReg) b = qr[nt][i * KW + c];
                else b = frag[(nt * KS + i * KW + c) * 32 + lane];
                mma<false>(s[k][nt], a0, a1, a2, a3, b.x, b.y);
              }
            }
        }
        const float* ss = sc + st * 2 * kTok;
        float lv[U][2], vm[U][2];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float ks0 = ss[PG ? k : k * 16 + g], ks1 = PG ? ks0 : ss[k * 16 + 8 + g];
          split_scale(ss[kTok + (PG ? k : k * 16 + g)], &lv[k][0], &vm[k][0]);
          lv[k][1] = lv[k][0], vm[k][1] = vm[k][0];
          if (!PG) split_scale(ss[kTok + k * 16 + 8 + g], &lv[k][1], &vm[k][1]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 f0 = mul2(make_float2(qf[nt][0], qf[nt][1]), make_float2(ks0, ks0));
            const float2 f1 = PG ? f0 : mul2(make_float2(qf[nt][0], qf[nt][1]), make_float2(ks1, ks1));
            set2(&s[k][nt][0], mul2(make_float2(s[k][nt][0], s[k][nt][1]), f0));
            set2(&s[k][nt][2], mul2(make_float2(s[k][nt][2], s[k][nt][3]), f1));
          }
        }
        if (live != (kTok == 32 ? 0xFFFFFFFFu : 0xFFFFu)) {  // selected, whatever a place without a token holds
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const bool see0 = (live >> (k * 16 + g)) & 1, see1 = (live >> (k * 16 + 8 + g)) & 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[k][nt][e] = (e < 2 ? see0 : see1) ? s[k][nt][e] : -INFINITY;
          }
        }
        settle(s, lv);
        uint32_t b0[U][NT], b1[U][NT];
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 down = make_float2(-ref_s[nt][0], -ref_s[nt][1]);
            float2 sum = make_float2(l_run[nt][0], l_run[nt][1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 y = make_float2(s[k][nt][2 * x], s[k][nt][2 * x + 1]);
              const float2 p = add2(y, down);
              sum = add2(sum, make_float2(ex2(p.x), ex2(p.y)));
              const float up = lv[k][x] + kLift;
              const float2 q = add2(y, make_float2(up - ref_v[nt][0], up - ref_v[nt][1]));
              const float2 z = mul2(make_float2(ex2(q.x), ex2(q.y)), make_float2(vm[k][x], vm[k][x]));
              // the weights' one rounding: float16 feeds the product
              (x ? b1 : b0)[k][nt] = turn(pack_f16(z.x, z.y));
            }
            l_run[nt][0] = sum.x;
            l_run[nt][1] = sum.y;
          }
        constexpr int VW = D >= 128 ? 4 : D / 32;  // words of a thread's D/8 dims read at once
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
          for (int i = 0; i < KS / (2 * VW); ++i) {
            uint32_t x[4][VW];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              lds<VW>(x[j], vst + at_v<D>(k * 16 + 2 * t4 + (j & 1) + (j >> 1) * 8, i * 128 + g * VW * 4));
#pragma unroll
            for (int c = 0; c < VW; ++c)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                const uint32_t p = __byte_perm(x[0][c], x[1][c], hf ? 0x7362 : 0x5140);
                const uint32_t q = __byte_perm(x[2][c], x[3][c], hf ? 0x7362 : 0x5140);
                const uint32_t a0 = widen(p, 0), a1 = widen(p, 1), a2 = widen(q, 0), a3 = widen(q, 1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma<false>(o[nt][(i * VW + c) * 2 + hf], a0, a1, a2, a3, b0[k][nt], b1[k][nt]);
              }
          }
      } else if (a.dk) {
        // drafted nodes, bf16, 16 at a time straight from where they lie; at most 16 of these steps an item
#pragma unroll 1
        for (int j0 = (t - rq.tiles_c) * kTK + w * kTok, je = min(rq.n, j0 + kTok); j0 < je; j0 += 16) {
          float s[1][NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[0][nt][e] = 0.f;
          const uint16_t* dk = static_cast<const uint16_t*>(a.dk) + rq.node0 * a.dk_sn + h * a.dk_sh;
          const uint16_t* dv = static_cast<const uint16_t*>(a.dv) + rq.node0 * a.dv_sn + h * a.dv_sh;
          const unsigned char* raw = smem + Sm::raw;
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
          settle(s, lv);
          uint32_t b0[NT], b1[NT];
          float p[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              l_run[nt][e & 1] += ex2(s[0][nt][e] - ref_s[nt][e & 1]);
              p[nt][e] = ex2(s[0][nt][e] - ref_v[nt][e & 1] + kLift);
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
            const int d = D == 256 ? (i >> 1) * 128 + g * 16 + (i & 1) * 8 : g * (D / 8) + i * 8;
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
                      const int d = (D == 256 ? (n >> 3) * 128 + g * 16 + (n & 7) * 2 : g * (D / 8) + n * 2) + x;
                      const uint32_t v = dv[(j0 + k) * a.dv_sn + d];
                      if ((v & 0x7F80u) == 0x7F80u) o[nt][n][x * 2 + e] += (k < 8 ? w0 : w1) * __uint_as_float(v << 16);
                    }
                }
          }
        }
      }
      __syncwarp();
      st = st == S - 1 ? 0 : st + 1;
    }
    cp_wait<0>();
    __syncthreads();
    // the warps' shares, joined through the ring's memory, in terms of ref_s
    float* jm = join + kWarps * M * D;
    float* jl = jm + kWarps * M;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = nt * 8 + 2 * t4 + e;
        float l = l_run[nt][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(kFull, l, x);
        if (g == 0) {
          jm[w * M + m] = ref_s[nt][e] == kNone ? -INFINITY : ref_s[nt][e];
          jl[w * M + m] = l;
        }
        const float f = ex2(ref_v[nt][e] - kLift - ref_s[nt][e]);
#pragma unroll
        for (int n = 0; n < KS; ++n) {
          const int d = D == 256 ? (n >> 3) * 128 + g * 16 + (n & 7) * 2 : g * (D / 8) + n * 2;
          *reinterpret_cast<float2*>(join + (w * M + m) * D + d) = make_float2(o[nt][n][e] * f, o[nt][n][e + 2] * f);
        }
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

template <int D, int NT, bool PG>
cudaError_t go(const AttnArgs& a, cudaStream_t s) {
  constexpr int smem = Kv8Smem<D, NT>::bytes;
  const cudaError_t e =
      cudaFuncSetAttribute(attn_kv8_kernel<D, NT, PG>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attn_kv8_kernel<D, NT, PG><<<a.grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D, int NT>
AttnPlan plan_n() {
  int per = 227 * 1024 / (Kv8Smem<D, NT>::bytes + 1024 + 256);
  if (per > kv8_blocks<D, NT>()) per = kv8_blocks<D, NT>();
  return AttnPlan{AttnPlan::kKv8, NT * 8, Kv8Smem<D, NT>::kTok * kWarps, sm_count() * (per < 1 ? 1 : per)};
}
template <int D>
AttnPlan plan_d(int rows) {
  if (rows <= 8) return plan_n<D, 1>();
  if (rows <= 16 || D == 256) return plan_n<D, 2>();
  return plan_n<D, D == 256 ? 2 : 4>();
}
template <int D>
cudaError_t go_d(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  const bool pg = a.kc.bs % 16 == 0;
  if (pl.M == 8) return pg ? go<D, 1, true>(a, s) : go<D, 1, false>(a, s);
  if (pl.M == 16) return pg ? go<D, 2, true>(a, s) : go<D, 2, false>(a, s);
  return pg ? go<D, D == 256 ? 2 : 4, true>(a, s) : go<D, D == 256 ? 2 : 4, false>(a, s);
}

}  // namespace
}  // namespace kk
