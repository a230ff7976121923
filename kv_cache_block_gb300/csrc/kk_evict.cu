// Eviction by accumulated attention weight, per (request, layer, KV head):
//  * evict_select_kernel: the first `sinks` tokens, the last `recent` ones and
//    the heaviest of the rest, `keep` in all, in ascending order (equal weights
//    to the lower index, NaN below everything);
//  * evict_compact_kernel: their Keys, Values and weights moved to slots
//    0 .. keep-1 of the request's pages, or of new ones.
#include "kk_device.cuh"

namespace kk {
namespace {

// ---- selection -------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;

// Order of a weight as an unsigned integer (larger: heavier): -0 as +0, NaN 0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  return m != m ? 0u : f32_to_ordered(m + 0.f);
}

// One CTA per (request, layer, head). The key of the (keep - sinks - recent)-th
// heaviest token of the middle is found digit by digit (11, 11 and 10 bits)
// from histograms in shared memory; then one ordered pass writes the tokens
// above it and the first of those equal to it.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(KCache kc, Table bt, const float* mass, int sinks,
                                                                   int recent, int keep, int* kept, int* new_lens,
                                                                   int* err) {
  __shared__ uint32_t s_hist[kBins];
  __shared__ uint32_t s_scan[kSelThreads / 32];
  __shared__ uint32_t s_digit, s_left;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int h = blockIdx.x % kc.H, l = (blockIdx.x / kc.H) % kc.L, r = blockIdx.x / (kc.H * kc.L);
  const int off = bt.offsets[r], nb = bt.offsets[r + 1] - off;
  int T = bt.seq_lens[r];
  if (T < 0 || nb < 0 || nb > bt.max_blocks || nb != (int)(((long long)T + kc.bs - 1) / kc.bs)) {
    if (tid == 0) flag_error(err, kErrBadIndex);
    T = 0;
  }
  int* out = kept + (long long)blockIdx.x * keep;
  const int n = min(T, keep);
  if (tid == 0 && l == 0 && h == 0 && new_lens) new_lens[r] = n;
  for (int i = n + tid; i < keep; i += kSelThreads) out[i] = -1;
  if (T <= keep) {
    for (int i = tid; i < n; i += kSelThreads) out[i] = i;
    return;
  }
  const int m0 = sinks, m1 = T - recent;  // the middle [m0, m1)
  const uint32_t want = (uint32_t)(keep - sinks - recent);
  for (int i = tid; i < sinks; i += kSelThreads) out[i] = i;
  for (int i = tid; i < recent; i += kSelThreads) out[keep - recent + i] = T - recent + i;
  if (want == 0) return;
  const float* mbase = mass + ((long long)l * kc.num_pages * kc.H + h) * kc.bs;
  auto key_at = [&](int t) -> uint32_t {
    const int b = t / kc.bs, page = bt.pages[off + b];
    if (page < 0 || page >= kc.num_pages) {
      flag_error(err, kErrBadIndex);
      return 0u;
    }
    return mass_key(mbase[(long long)page * kc.H * kc.bs + (t - b * kc.bs)]);
  };
  uint32_t prefix = 0, left = want;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass == 2 ? 10 : 11, bins = 1 << bits;
    const int up = shift;
    shift -= bits;
    for (int i = tid; i < bins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int t = m0 + tid; t < m1; t += kSelThreads) {
      const uint32_t k = key_at(t);
      if (pass == 0 || (k >> up) == prefix) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // from the top bin down: the bin in which the `left`-th key lies
    constexpr int PER = kBins / kSelThreads;
    const int per = bins / kSelThreads;
    uint32_t c[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < per) sum += c[i] = s_hist[bins - 1 - (tid * per + i)];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) s_scan[w] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (int x = 0; x < w; ++x) before += s_scan[x];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (i >= per) break;
      if (before < left && left <= before + c[i]) {
        s_digit = (uint32_t)(bins - 1 - (tid * per + i));
        s_left = left - before;
      }
      before += c[i];
    }
    __syncthreads();
    prefix = (prefix << bits) | s_digit;
    left = s_left;
    __syncthreads();
  }
  // `prefix` is the threshold key; the first `left` tokens equal to it stay
  uint32_t done = (uint32_t)sinks, eq_done = 0;
  for (int t0 = m0; t0 < m1; t0 += kSelThreads) {
    const int t = t0 + tid;
    const uint32_t k = t < m1 ? key_at(t) : 0u;
    const bool gt = t < m1 && k > prefix, eq = t < m1 && k == prefix;
    const uint32_t bg = __ballot_sync(kFull, gt), be = __ballot_sync(kFull, eq), lt = (1u << lane) - 1u;
    if (lane == 0) s_scan[w] = (uint32_t)__popc(bg) | ((uint32_t)__popc(be) << 16);
    __syncthreads();
    uint32_t g = 0, e = 0, gs = 0, es = 0;
    for (int x = 0; x < kSelThreads / 32; ++x) {
      const uint32_t y = s_scan[x];
      if (x < w) {
        g += y & 0xFFFFu;
        e += y >> 16;
      }
      gs += y & 0xFFFFu;
      es += y >> 16;
    }
    const uint32_t my_g = g + __popc(bg & lt), my_e = eq_done + e + __popc(be & lt);
    const uint32_t e_before = min(my_e, left) - min(eq_done, left);  // equal ones kept earlier in this pass
    if (gt || (eq && my_e < left)) out[done + my_g + e_before] = t;
    done += gs + min(eq_done + es, left) - min(eq_done, left);
    eq_done += es;
    __syncthreads();
  }
}

// ---- move --------------------------------------------------------------------
constexpr int kMoveThreads = 256;

struct MoveArgs {
  KCache kc, vc;
  Table bt;
  const int* kept;
  int keep, dst_blocks;
  const float* mass_in;
  float* mass_out;
  const int* dst_pages;  // [R][dst_blocks], or null: the request's own pages
  int row16;             // 16-byte pieces of a row
  int* err;
};

// One CTA per (request, layer, head). Slots are taken in chunks; a chunk is
// read whole before any of it is written, and since kept[i] >= i its writes
// never reach a source of a later chunk: the move is safe in place.
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const MoveArgs a) {
  constexpr int U = 4;
  const int tid = threadIdx.x;
  const int H = a.kc.H, bs = a.kc.bs;
  const int h = blockIdx.x % H, l = (blockIdx.x / H) % a.kc.L, r = blockIdx.x / (H * a.kc.L);
  const int off = a.bt.offsets[r], nb = a.bt.offsets[r + 1] - off, T = a.bt.seq_lens[r];
  if (T < 0 || nb < 0 || nb > a.bt.max_blocks || nb != (int)(((long long)T + bs - 1) / bs)) {
    if (tid == 0) flag_error(a.err, kErrBadIndex);
    return;
  }
  const int n = min(T, a.keep), es = a.kc.dtype == 1 ? 2 : 4;
  const int* kept = a.kept + (long long)blockIdx.x * a.keep;
  const int* dst = a.dst_pages ? a.dst_pages + (long long)r * a.dst_blocks : a.bt.pages + off;
  const int* src = a.bt.pages + off;
  auto place = [&](int i, int* sp, int* st, int* dp, int* dt) -> bool {
    const int t = kept[i];
    if (t < 0 || t >= T) {
      flag_error(a.err, kErrBadIndex);
      return false;
    }
    *sp = src[t / bs];
    *st = t % bs;
    *dp = dst[i / bs];
    *dt = i % bs;
    if (*sp < 0 || *sp >= a.kc.num_pages || *dp < 0 || *dp >= a.kc.num_pages) {
      flag_error(a.err, kErrBadIndex);
      return false;
    }
    return true;
  };
  const int per = kMoveThreads / a.row16 * U;  // rows of a chunk
  const int piece = tid % a.row16, sub = tid / a.row16;
  for (int c = 0; c < n; c += per) {
    uint4 kx[U], vx[U];
    long long kd[U], vd[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int i = c + x * (kMoveThreads / a.row16) + sub;
      int sp, st, dp, dt;
      kd[x] = -1;
      if (i < min(n, c + per) && place(i, &sp, &st, &dp, &dt)) {
        kx[x] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.kc.base) +
                                                (l * a.kc.sL + sp * a.kc.sP + h * a.kc.sH + st * a.kc.sT) * es +
                                                piece * 16);
        kd[x] = (l * a.kc.sL + dp * a.kc.sP + h * a.kc.sH + dt * a.kc.sT) * es + piece * 16;
        if (a.vc.base) {
          vx[x] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.vc.base) +
                                                  (l * a.vc.sL + sp * a.vc.sP + h * a.vc.sH + st * a.vc.sT) * es +
                                                  piece * 16);
          vd[x] = (l * a.vc.sL + dp * a.vc.sP + h * a.vc.sH + dt * a.vc.sT) * es + piece * 16;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < U; ++x)
      if (kd[x] >= 0) {
        *reinterpret_cast<uint4*>(const_cast<char*>(static_cast<const char*>(a.kc.base)) + kd[x]) = kx[x];
        if (a.vc.base)
          *reinterpret_cast<uint4*>(const_cast<char*>(static_cast<const char*>(a.vc.base)) + vd[x]) = vx[x];
      }
  }
  if (!a.mass_in) return;
  const long long mrow = ((long long)l * a.kc.num_pages * H + h) * bs;
  for (int c = 0; c < n; c += kMoveThreads) {
    const int i = c + tid;
    int sp, st, dp, dt;
    const bool ok = i < n && place(i, &sp, &st, &dp, &dt);
    const float m = ok ? a.mass_in[mrow + (long long)sp * H * bs + st] : 0.f;
    __syncthreads();
    if (ok) a.mass_out[mrow + (long long)dp * H * bs + dt] = m;
  }
}

}  // namespace

cudaError_t launch_evict_select(const KCache& kc, const Table& bt, const float* mass, int sinks, int recent, int keep,
                                int* kept, int* new_lens, int* err, cudaStream_t s) {
  evict_select_kernel<<<bt.R * kc.L * kc.H, kSelThreads, 0, s>>>(kc, bt, mass, sinks, recent, keep, kept, new_lens,
                                                                 err);
  return cudaGetLastError();
}

cudaError_t launch_evict_compact(const KCache& kc, const KCache& vc, const Table& bt, const int* kept, int keep,
                                 const float* mass_in, float* mass_out, const int* dst_pages, int* err,
                                 cudaStream_t s) {
  const MoveArgs a{kc, vc, bt, kept, keep, (keep + kc.bs - 1) / kc.bs, mass_in, mass_out, dst_pages,
                   kc.D * (kc.dtype == 1 ? 2 : 4) / 16, err};
  evict_compact_kernel<<<bt.R * kc.L * kc.H, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kk
