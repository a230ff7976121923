// kk_kv8_write: new tokens' Keys and Values as e4m3 codes with a power-of-two
// scale for each (page, layer, KV head), bound by the bytes of the new tokens.
//
// An item is what one request adds to one page of one (layer, head), Keys or
// Values: the largest finite magnitude of its new tokens gives the scale, then
// they are divided by it (a multiplication by its inverse, exact) and rounded
// once, to nearest even. Where the page held older tokens and its scale changes,
// their codes move with it. A scale of the caller's own that is no power of two
// costs its item a second round of stores, with exact divisions. One warp takes
// an item of few tokens (a decode step: the item is one row), a block of eight
// warps one of many. The new tokens stay in registers between the two passes, up
// to 8 vectors of 16 bytes a thread (a page of 128 tokens of 128 bf16 dims in a
// block); larger items read them again, from L2.
//
// Measured: one token of 8 requests in 28 layers of 4 heads of 128 dims 6.2 us
// (a launch and a chain of four loads); prompts of 22.5 K tokens, one layer (69 MB
// read and written), 16 us on new inputs each time, 4.3 TB/s (13.4 where a call
// repeats on the same, its codes in L2). Two and a half rounds of blocks, each a
// chain of look-ups, loads and a block-wide maximum, are what is left; magnitudes
// as packed integers and 64 registers, four blocks an SM instead of two, took the
// repeated call there from 22.5.
#include "kk_device.cuh"
#include "kk_pdl.cuh"
#include "kk_write8.cuh"

namespace kk {
namespace {

constexpr int kThreads = 256;
constexpr int kKeep = 8;  // vectors a thread keeps

// Two values as e4m3, each rounded to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float only_finite(float x) {  // infinity becomes NaN
  return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : x;
}

// The largest magnitude of vectors, as the bits of the type (they order like the values, infinity and NaN
// above all): two bf16 halves at a time.
template <typename T>
struct Top;
template <>
struct Top<bf16_t> {
  static constexpr uint32_t kInf = 0x7F80u;
  uint32_t x = 0;
  __device__ __forceinline__ void add(const uint4& v) {
    x = __vmaxu2(__vmaxu2(x, __vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu)),
                 __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  }
  __device__ __forceinline__ uint32_t bits() const { return max(x & 0xFFFFu, x >> 16); }
  __device__ static float value(uint32_t b) { return __uint_as_float(b << 16); }
};
template <>
struct Top<float> {
  static constexpr uint32_t kInf = 0x7F800000u;
  uint32_t x = 0;
  __device__ __forceinline__ void add(const uint4& v) {
    x = max(max(max(x, v.x & 0x7FFFFFFFu), max(v.y & 0x7FFFFFFFu, v.z & 0x7FFFFFFFu)), v.w & 0x7FFFFFFFu);
  }
  __device__ __forceinline__ uint32_t bits() const { return x; }
  __device__ static float value(uint32_t b) { return __uint_as_float(b); }
};

// The smallest power of two that is at least amax / 448, and at least 2^-126.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  // 448 = 1.75 * 2^8: one exponent more where the mantissa is above 1.75
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  return __uint_as_float((uint32_t)(e < 1 ? 1 : e) << 23);
}

// q, rounded from a value that is r's sign further on (r 0: exact): moved off e4m3's halfway points by its last bit,
// so that rounding it once more gives what the value itself rounds to. (Halfway points have 5 bits; a product or
// quotient of two float32 numbers that rounds to one lies next to it.)
__device__ __forceinline__ float keep_side(float q, float r) {
  const uint32_t b = __float_as_uint(q);
  if (r == 0.f || (b & 0xFFFFu) || q == 0.f || !(fabsf(q) <= 448.f)) return q;
  return __uint_as_float((r > 0.f) == (q > 0.f) ? b + 1 : b - 1);
}

template <typename T, int D, int W>
__global__ void __launch_bounds__(kThreads, 4) write8_kernel(const Write8Args a) {
  constexpr int E = Vec16<T>::kElems, CH = D / E;  // elements of a vector, vectors of a row
  constexpr int NTH = W * 32, IPB = kThreads / NTH;  // threads of an item, items of a block
  __shared__ uint32_t s_max[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x % NTH, sub = threadIdx.x / NTH;
  const int r = blockIdx.z, H = a.kc.H;
  const int item = blockIdx.y * IPB + sub, items = a.layers * H * a.sides;
  // the request's new tokens, and the page this item is about
  const int n0 = a.token_off ? a.token_off[r] : r * a.max_new;
  const int n = (a.token_off ? a.token_off[r + 1] : n0 + a.max_new) - n0;
  const int off = a.bt.offsets[r], nb = a.bt.offsets[r + 1] - off, T1 = a.bt.seq_lens[r], bs = a.kc.bs;
  const bool ok = n0 >= 0 && n >= 0 && n <= a.max_new && n0 + (long long)n <= a.num_nodes && T1 >= n &&
                  T1 <= kMaxTokens && nb >= 0 && nb <= a.bt.max_blocks &&
                  nb == (int)(((unsigned)T1 + (unsigned)bs - 1u) / (unsigned)bs);
  const bool first = threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0;
  if (!ok) {
    if (first) flag_error(a.err, kErrBadIndex);
    return;
  }
  const int t0 = T1 - n;
  const long long bl = t0 / bs + (long long)blockIdx.x;
  if (n == 0 || bl >= nb) return;
  const int b = (int)bl;
  const int page = a.bt.pages[off + b];
  if (page < 0 || page >= a.kc.num_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err, kErrBadIndex);
    return;
  }
  const bool real = item < items;  // a block of several items may have some left over
  const int kv = real ? item % a.sides : 0, h = real ? item / a.sides % H : 0, l = real ? item / (a.sides * H) : 0;
  const Write8Side& x = a.side[kv];
  const int lo = max(t0, b * bs), hi = min((long long)T1, (b + 1ll) * bs), had = lo - b * bs;
  const int vecs = real ? (hi - lo) * CH : 0;
  const long long src = (l * x.sl + (n0 + lo - t0) * x.sn + h * x.sh) * (16 / E);
  const char* from = static_cast<const char*>(x.src) + src;
  const long long row_bytes = x.sn * (16 / E);
  auto at_vec = [&](int i) { return *reinterpret_cast<const uint4*>(from + (i / CH) * row_bytes + (i % CH) * 16); };
  // The largest of the item's threads.
  auto largest = [&](uint32_t x) {
    x = __reduce_max_sync(kFull, x);
    if constexpr (W > 1) {
      if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = x;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) x = max(x, s_max[w]);
      __syncthreads();
    }
    return x;
  };
  uint4 keep[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) {
    const int i = tid + k * NTH;
    keep[k] = make_uint4(0, 0, 0, 0);
    if (i < vecs) keep[k] = at_vec(i);
  }
  Top<T> all;
#pragma unroll
  for (int k = 0; k < kKeep; ++k) all.add(keep[k]);
  for (int i = tid + kKeep * NTH; i < vecs; i += NTH) all.add(at_vec(i));
  uint32_t bits = largest(all.bits());
  const bool odd = bits >= Top<T>::kInf;  // something is not finite: the same for the item
  if (odd) {
    float top = 0.f;
    for (int i = tid; i < vecs; i += NTH) {
      float f[E];
      Vec16<T>::unpack(at_vec(i), f);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (fabsf(f[e]) < INFINITY) top = fmaxf(top, fabsf(f[e]));
    }
    bits = __float_as_uint(top) >> (E == 8 ? 16 : 0);
  }
  if (odd) bits = largest(bits);
  const float top = Top<T>::value(bits);
  if (!real) return;
  float* at = x.scale + ((long long)(a.layer + l) * a.kc.num_pages + page) * H + h;
  const float old = had ? *at : 0.f, now = fmaxf(fabsf(old), pow2_scale(top));
  const float inv = 1.f / now;
  char* codes = static_cast<char*>(x.codes) + (a.layer + l) * x.dL + page * x.dP + h * x.dH;
  if constexpr (W > 1) __syncthreads();  // every thread has read the scale
  else __syncwarp();
  if (tid == 0) *at = now;
  auto store = [&](int i, const uint4& v, auto divide) {
    float f[E];
    Vec16<T>::unpack(v, f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = divide(f[e]);
    if (odd)
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = only_finite(f[e]);
    char* to = codes + (had + i / CH) * x.dT + (i % CH) * E;
    const uint32_t p = to_e4m3x2(f[0], f[1]) | to_e4m3x2(f[2], f[3]) << 16;
    if constexpr (E == 8)
      *reinterpret_cast<uint2*>(to) = make_uint2(p, to_e4m3x2(f[4], f[5]) | to_e4m3x2(f[6], f[7]) << 16);
    else
      *reinterpret_cast<uint32_t*>(to) = p;
  };
  auto scaled = [&](float x) { return x * inv; };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (tid + k * NTH < vecs) store(tid + k * NTH, keep[k], scaled);
  for (int i = tid + kKeep * NTH; i < vecs; i += NTH)
    store(i, at_vec(i), scaled);
  if ((__float_as_uint(now) & 0x7FFFFFu) != 0) {  // no power of two: over again, as exact quotients round
    const float up = now < 0x1p-60f ? 0x1p64f : 1.f, by = now * up;  // remainders stay in float32's normal range
    for (int i = tid; i < vecs; i += NTH)
      store(i, at_vec(i), [&](float x) {
        const float y = x * up / by;
        return keep_side(y, fmaf(-y, by, x * up));
      });
  }
  // The page's older codes, in terms of the new scale. In a decode step a warp does this by itself, a word a lane at a
  // time: pages of 128 tokens, half full, 8.9 us a call where no scale grows, 21 where one does, 36 where all do (pages
  // of 16: 8.9, 9.0, 11.4).
  if (had && old != now) {
    const float f = old == -now ? -1.f : old * inv;  // else `now` is the new tokens' power of two
    for (int i = tid; i < had * (D / 4); i += NTH) {
      uint32_t* p = reinterpret_cast<uint32_t*>(codes + (i / (D / 4)) * x.dT + (i % (D / 4)) * 4);
      const uint32_t c = *p;
      float y[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t two;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"((uint16_t)(e ? c >> 16 : c)));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(y[2 * e]), "=f"(y[2 * e + 1])
            : "r"(two));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = y[e] * f;
        y[e] = keep_side(z, fmaf(y[e], f, -z));
      }
      *p = to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16;
    }
  }
}

template <typename T, int D>
cudaError_t go(const Write8Args& a, cudaStream_t s) {
  const long long pieces = (a.max_new + a.kc.bs - 2ll) / a.kc.bs + 1;  // pages that max_new tokens reach, at most
  const int items = a.layers * a.kc.H * a.sides;
  // a warp an item while its threads keep every vector
  const bool small = std::min(a.max_new, a.kc.bs) * (D / Vec16<T>::kElems) <= kKeep * 32;
  const int ipb = small ? kThreads / 32 : 1;
  const dim3 grid((unsigned)pieces, (unsigned)((items + ipb - 1) / ipb), (unsigned)a.bt.R);
  return launch_pdl(small ? write8_kernel<T, D, 1> : write8_kernel<T, D, kThreads / 32>, grid, kThreads, 0, s, a);
}
template <typename T>
cudaError_t go_t(const Write8Args& a, cudaStream_t s) {
  switch (a.kc.D) {
    case 32: return go<T, 32>(a, s);
    case 64: return go<T, 64>(a, s);
    case 128: return go<T, 128>(a, s);
    case 256: return go<T, 256>(a, s);
  }
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_kv8_write(const Write8Args& a, cudaStream_t s) {
  return a.f32 ? go_t<float>(a, s) : go_t<bf16_t>(a, s);
}

}  // namespace kk
