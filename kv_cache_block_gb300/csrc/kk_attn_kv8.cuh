// kk_tree_attn_kv8: attention over a cache of e4m3 codes with a scale for each
// page and KV head, K = code * k_scale, V = code * v_scale; bound by the bytes of
// the codes.
//
// Four warps share an item's rows (M = 8 or 16) and take 32 tokens each of every
// 128-token tile (256 dims: 16 of 64), streamed through a ring of shared-memory
// stages of their own as in kk_attn_mma.cu. Tokens are the M axis of the
// products (S^T = K Q^T, O^T = V^T P^T with m16n8k16 matrix instructions), query
// rows the N axis: a decode token's group of at most 8 rows fills it, where rows
// along M would leave half of 16 empty, and every 16 x 16 codes cost one
// instruction.
//
// e4m3 values are exact in float16, so codes are widened two at a time and
// multiplied as float16; a scale never meets the products, it multiplies the
// score (K) or the weight (V) of its page. For V the bytes of two tokens are
// interleaved (prmt) and widened into an operand register. No ldmatrix, no
// transposed copy; the weights, which come out of the first product with tokens
// along the wrong axis, are turned by movmatrix.
//
// Softmax. Two references a row (log2 domain): one for the sum of weights, 2^(s -
// ref) in float32, one for what multiplies the codes of V, 2^(s - ref - gap + 6) *
// v_scale, which has to fit float16 whatever the pages' scales are. Both are
// left alone until a score passes one by 2^8 (one vote a step); until then sums
// below 2^8 cost nothing and no reduction over lanes is needed.
//
// Measured, D = 128, groups of 7, one node, with the join: 8 requests of up to
// 32768 tokens (189 MB of codes) 44 us, 4.3 TB/s; a million tokens in pages of 16
// (1.07 GB) 177 us, 6.05 TB/s (the main kernel 166: DRAM 83 % busy, an instruction
// in half of all slots); 63 rows over 8 requests of up to 8191 tokens 49 us. With one group a step and four CTAs
// an SM the first two took 46 and 182, with 340 instead of 300 instructions for 16
// tokens and rows; before blocks were followed without divisions 51 and 212. What
// is left of the first: about 12 us of starting, first loads and join.
#pragma once
#include "kk_kv8.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

// 16-token groups of a warp's share of a tile: two while registers allow, so that two chains of products are under
// way and what a step costs besides them is paid once for 32 tokens.
template <int D, int NT>
__host__ __device__ constexpr int kv8_groups() {
  return D <= 128 ? 2 : 1;
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

template <int D, int NT>
__host__ __device__ constexpr int kv8_stages() {
  return (D >= 128 ? 4 : D == 64 ? 6 : 8) / kv8_groups<D, NT>() - (D == 256 ? 1 : 0);
}
template <int D, int NT>
struct Kv8Smem {
  static constexpr int M = NT * 8, S = kv8_stages<D, NT>(), kTok = 16 * kv8_groups<D, NT>(), kStage = kTok * D * 2;
  static constexpr int ring = kWarps * S * kStage, join = kWarps * M * (D + 2) * 4;
  static constexpr int scales = ring > join ? ring : join;       // [warps][stages][K, V][kTok] floats
  static constexpr int raw = scales + kWarps * S * 2 * kTok * 4;  // queries as they are, bf16 [M][D]
  static constexpr bool kQReg = NT * D <= 256;                   // query operands stay in registers
  static constexpr int frag = raw + M * D * 2;                   // else lie here: [NT][D/16][32 lanes]
  static constexpr int bytes = frag + (kQReg ? 0 : M * D * 2);
};

template <int D, int NT>
constexpr int kv8_blocks() {
  return D == 256 ? 2 : NT == 1 && D < 128 ? 4 : 3;
}

template <int D, int NT, bool PG>
__global__ void __launch_bounds__(kThreads, (kv8_blocks<D, NT>())) attn_kv8_kernel(const AttnArgs a) {
  using Sm = Kv8Smem<D, NT>;
  constexpr int M = NT * 8, KS = D / 16, S = Sm::S, U = kv8_groups<D, NT>(), kTok = Sm::kTok, kTK = kTok * kWarps;
  constexpr bool kQReg = Sm::kQReg;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_place[kWarps + 4];
  __shared__ uint32_t s_ok[kWarps][S];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  unsigned char* ring = smem + w * S * Sm::kStage;
  const uint32_t ring_at = smem_u32(ring);
  float* sc = reinterpret_cast<float*>(smem + Sm::scales) + w * S * 2 * kTok;
  const uint32_t sc_at = smem_u32(sc);
  uint2* frag = reinterpret_cast<uint2*>(smem + Sm::frag);
  unsigned char* raw = smem + Sm::raw;
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
    const char* k_lane =
        static_cast<const char*>(a.kc.base) + a.layer * a.kc.sL + h * a.kc.sH + c * 16 + (PG ? sub * a.kc.sT : 0);
    const char* v_lane =
        static_cast<const char*>(a.vc.base) + a.layer * a.vc.sL + h * a.vc.sH + c * 16 + (PG ? sub * a.vc.sT : 0);
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
              cp_async4(sst + (lane * kTok + i) * 4,
                        (lane ? a.v_scale : a.k_scale) + s_at + (long long)x[i].page * a.kc.H, n > 0);
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
    stage_queries<D, M>(a, rq, h, row0, rows, raw);
    __syncthreads();
    float qf[NT][2];
    uint2 qr[kQReg ? NT : 1][KS];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint2(&q)[KS] = qr[kQReg ? nt : 0];
      query_operands<D>(raw + nt * 8 * D * 2, a.scale_log2, q, qf[nt]);
      if constexpr (!kQReg) {
        if (w == nt)
#pragma unroll
          for (int j = 0; j < KS; ++j) frag[(nt * KS + j) * 32 + lane] = q[j];
      }
    }
    if constexpr (!kQReg) __syncthreads();

    Rows<D, NT> rs;
    rs.clear();
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
              const uint32_t a0 = widen(x[k][c], 0), a1 = widen(y[k][c], 0);
              const uint32_t a2 = widen(x[k][c], 1), a3 = widen(y[k][c], 1);
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
          rs.template score<PG>(s[k], qf, ks0, ks1, live >> (16 * k) & 0xFFFFu);
        }
        rs.template settle<PG>(s, lv);
        uint32_t wt[U][2][NT];
#pragma unroll
        for (int k = 0; k < U; ++k) rs.weigh(s[k], lv[k], vm[k], wt[k]);
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
                  mma<false>(rs.o[nt][(i * VW + c) * 2 + hf], a0, a1, a2, a3, wt[k][0][nt], wt[k][1][nt]);
              }
          }
      } else if (a.dk) {
        const int j0 = (t - rq.tiles_c) * kTK + w * kTok;
#pragma unroll 1
        for (int j = j0; j < min(rq.n, j0 + kTok); j += 16) rs.drafts(a, rq, h, raw, row0, j);
      }
      __syncwarp();
      st = st == S - 1 ? 0 : st + 1;
    }
    cp_wait<0>();
    __syncthreads();
    rs.leave(join, kWarps, w, M, 0);  // over the ring's memory
    __syncthreads();
    finish_rows<D, M, kWarps>(a, rq, h, row0, rows, t0 == 0 && t1 == rq.tiles, join,
                              partial_slot(a, blockIdx.x, u == pl.u0 ? 0 : 1, M, D));
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
  // not before the launch in front of it has ended: CTAs that took the room some SMs had early left others idle (a
  // million tokens 176 -> 239 us)
  attn_kv8_kernel<D, NT, PG><<<a.grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D, int NT>
AttnPlan plan_n() {
  int per = 227 * 1024 / (Kv8Smem<D, NT>::bytes + 1024 + 256);
  if (per > kv8_blocks<D, NT>()) per = kv8_blocks<D, NT>();
  return AttnPlan{AttnPlan::kKv8, NT * 8, Kv8Smem<D, NT>::kTok * kWarps, sm_count() * (per < 1 ? 1 : per)};
}

// The kernel by rows, 8 or 16 an item.
template <int D>
AttnPlan plan_d(int rows) {
  return rows <= 8 ? plan_n<D, 1>() : plan_n<D, 2>();
}
template <int D>
cudaError_t go_d(const AttnArgs& a, const AttnPlan& pl, cudaStream_t s) {
  const bool pg = a.kc.bs % 16 == 0;  // 16 tokens in a row lie in one page
  if (pl.M == 8) return pg ? go<D, 1, true>(a, s) : go<D, 1, false>(a, s);
  return pg ? go<D, 2, true>(a, s) : go<D, 2, false>(a, s);
}

}  // namespace
}  // namespace kk
