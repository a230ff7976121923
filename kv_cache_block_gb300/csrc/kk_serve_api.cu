// C ABI of the calls around a serving step (include/kk.h): norm and rotation, the
// 8-bit cache, pages. Argument checks on the host, then launches.
#include <cmath>

#include "../../include/kk.h"

#include "kk_attn.cuh"
#include "kk_internal.h"
#include "kk_pages.cuh"
#include "kk_rope.cuh"
#include "kk_write8.cuh"

namespace kk {
// kk_api.cu
kk_status check_kcache_desc(const kk_kcache_desc* kc, KCache* out);
kk_status check_block_table(const kk_block_table* bt, Table* out);
// kk_attn_api.cu
kk_status tree_attn_call(AttnArgs* a, const kk_block_table* bt, int32_t layer, const kk_selection* sel,
                         const kk_tree* tree, const void* q, int64_t q_sn, int64_t q_sh, int32_t Hq, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream);
}  // namespace kk

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
kk_status done(cudaError_t e) {
  return e == cudaSuccess ? KK_OK : e == cudaErrorNotSupported ? KK_ERR_UNSUPPORTED : KK_ERR_CUDA;
}
bool same_sizes(const kk::KCache& a, const kk::KCache& b) {
  return a.dtype == b.dtype && a.L == b.L && a.H == b.H && a.D == b.D && a.bs == b.bs && a.num_pages == b.num_pages;
}
bool dim_ok(int D) { return D == 32 || D == 64 || D == 128 || D == 256; }

// An e4m3 cache.
kk_status check_cache8(const kk_kcache_desc* kc, kk::KCache* out) {
  if (!kc || !kc->base || kc->dtype != KK_E4M3) return KK_ERR_INVALID;
  if (kc->num_layers <= 0 || kc->num_kv_heads <= 0 || kc->head_dim <= 0 || kc->block_size <= 0 || kc->num_pages <= 0)
    return KK_ERR_INVALID;
  if ((long long)kc->num_layers * kc->num_kv_heads > kk::kMaxLH || !dim_ok(kc->head_dim)) return KK_ERR_UNSUPPORTED;
  if (!aligned(kc->base, 16) || kc->block_size > 65536) return KK_ERR_UNSUPPORTED;
  for (int64_t st : {kc->stride_layer, kc->stride_page, kc->stride_head, kc->stride_token})
    if (st < 0 || st % 16) return KK_ERR_UNSUPPORTED;
  *out = kk::KCache{kc->base,      kc->dtype,        kc->num_layers,   kc->num_kv_heads, kc->head_dim,    kc->block_size,
                    kc->num_pages, kc->stride_layer, kc->stride_page, kc->stride_head,  kc->stride_token};
  return KK_OK;
}

// Rows of n nodes (a tensor without any has no address).
kk_status check_rows(const kk_rows* r, int es, int n) {
  if (!r || (!r->base && n > 0)) return KK_ERR_INVALID;
  if (!aligned(r->base, 16)) return KK_ERR_UNSUPPORTED;
  for (int64_t st : {r->stride_node, r->stride_head, r->stride_layer})
    if (st < 0 || st * es % 16) return KK_ERR_UNSUPPORTED;
  return KK_OK;
}

// The page arrays of a call.
kk_status check_arrays(const kk_page_array* arrays, int32_t n, kk::PageArrays* out) {
  if (n < 0 || n > kk::kMaxPageArrays || (n > 0 && !arrays)) return KK_ERR_INVALID;
  out->n = n;
  for (int i = 0; i < n; ++i) {
    const kk_page_array& a = arrays[i];
    if (!a.base || a.bytes <= 0 || a.slices <= 0 || a.stride_slice < 0 || a.stride_page < a.bytes)
      return KK_ERR_INVALID;
    if (!aligned(a.base, 4) || a.bytes % 4 || a.stride_slice % 4 || a.stride_page % 4) return KK_ERR_UNSUPPORTED;
    out->a[i] = kk::PageArray{static_cast<char*>(a.base), a.stride_slice, a.stride_page, a.bytes, a.slices};
  }
  return kk::plan_page_arrays(out) ? KK_OK : KK_ERR_UNSUPPORTED;
}

// An array of ints of a call, and whether two of them share memory.
struct Ints {
  const int32_t* p;
  long long n;
};
bool share(const Ints& a, const Ints& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n > 0 && b.n > 0 && x < y + 4 * (unsigned long long)b.n && y < x + 4 * (unsigned long long)a.n;
}
// Whether any of what is written shares memory with what is read while it is, or with another of them.
template <size_t W, size_t N>
bool collide(const Ints (&written)[W], const Ints (&read)[N]) {
  for (size_t i = 0; i < W; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (share(written[i], written[j])) return true;
    for (const Ints& r : read)
      if (share(written[i], r)) return true;
  }
  return false;
}

constexpr int kMaxInts = 1 << 30;  // pages, or elements of a list

kk_status check_refs(const int32_t* in, int32_t* out, int32_t num_pages) {
  if (!in || !out || num_pages < 1) return KK_ERR_INVALID;
  if (!aligned(in, 4) || !aligned(out, 4) || num_pages > kMaxInts) return KK_ERR_UNSUPPORTED;
  return in != out && share({in, num_pages}, {out, num_pages}) ? KK_ERR_INVALID : KK_OK;  // the same, or apart
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

extern "C" {

kk_status kk_qk_norm_rope(int32_t dtype, int32_t num_nodes, int32_t num_q_heads, int32_t num_kv_heads, int32_t D,
                          const kk_rows* q, const kk_rows* k, const kk_rows* v, const void* q_weight,
                          const void* k_weight, float eps, const int32_t* positions, const kk_rope* rope,
                          const kk_rows* q_out, const kk_rows* k_out, const kk_kcache_desc* kc,
                          const kk_kcache_desc* vc, const kk_block_table* bt, const int32_t* token_offsets,
                          int32_t layer, cudaStream_t stream) {
  if ((dtype != KK_BF16 && dtype != KK_F32) || num_nodes < 0 || num_q_heads < 0 || num_kv_heads < 0)
    return KK_ERR_INVALID;
  if (num_q_heads + (long long)num_kv_heads == 0 || !(eps >= 0.f) || !std::isfinite(eps)) return KK_ERR_INVALID;
  if (!dim_ok(D) || num_nodes > kk::kMaxTokens || num_q_heads > 65536 || num_kv_heads > 65536)
    return KK_ERR_UNSUPPORTED;
  const int es = dtype == KK_F32 ? 4 : 2;
  kk::RopeArgs a = {};
  a.f32 = dtype == KK_F32;
  a.nodes = num_nodes;
  a.Hq = num_q_heads;
  a.H = num_kv_heads;
  a.D = D;
  kk_status st;
  auto rows = [&](const kk_rows* r, kk::RopeRows* out) {
    const kk_status s = check_rows(r, es, num_nodes);
    if (s == KK_OK) *out = kk::RopeRows{r->base, r->stride_node, r->stride_head};
    return s;
  };
  if (num_q_heads && ((st = rows(q, &a.q)) != KK_OK || (st = rows(q_out, &a.q_out)) != KK_OK)) return st;
  if (num_kv_heads && (st = rows(k, &a.k)) != KK_OK) return st;
  if (k_out && (!num_kv_heads || (st = rows(k_out, &a.k_out)) != KK_OK)) return num_kv_heads ? st : KK_ERR_INVALID;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4) || !aligned(token_offsets, 4))
    return KK_ERR_UNSUPPORTED;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  if (rope) {
    if (rope->rotary_dim < 0 || rope->rotary_dim > D || (rope->rotary_dim && !rope->inv_freq) ||
        !std::isfinite(rope->scale))
      return KK_ERR_INVALID;
    if (rope->rotary_dim % 16 || !aligned(rope->inv_freq, 4)) return KK_ERR_UNSUPPORTED;
    a.inv_freq = rope->inv_freq;
    a.rd = rope->rotary_dim;
    a.half = !rope->interleaved;
    a.rope_scale = rope->scale;
  }
  if ((kc || vc) && !bt) return KK_ERR_INVALID;
  if ((vc && (!v || !kc)) || (v && !vc)) return KK_ERR_INVALID;  // Values go to the cache, next to their Keys
  if (bt) {
    if ((st = kk::check_block_table(bt, &a.bt)) != KK_OK) return st;
    if (!token_offsets && a.bt.R != num_nodes) return KK_ERR_INVALID;
    if (num_nodes > 0 && a.bt.R == 0) return KK_ERR_INVALID;
    if (!kc) return KK_ERR_INVALID;  // it says how long a block is
    kk::KCache c, d = {};
    if ((st = kk::check_kcache_desc(kc, &c)) != KK_OK) return st;
    if (c.dtype != dtype || c.D != D || c.H != num_kv_heads || layer < 0 || layer >= c.L) return KK_ERR_INVALID;
    if (vc) {
      if ((st = kk::check_kcache_desc(vc, &d)) != KK_OK || (st = rows(v, &a.v_rows)) != KK_OK) return st;
      if (!same_sizes(c, d)) return KK_ERR_INVALID;
      a.v = true;
    }
    a.kc = const_cast<void*>(c.base);
    a.kL = c.sL, a.kP = c.sP, a.kH = c.sH, a.kT = c.sT;
    a.vc = const_cast<void*>(d.base);
    a.vL = d.sL, a.vP = d.sP, a.vH = d.sH, a.vT = d.sT;
    a.bs = c.bs;
    a.num_pages = c.num_pages;
    a.layer = layer;
    a.token_off = token_offsets;
  }
  if (num_nodes == 0) return KK_OK;
  if (!(a.err = kk::device_error_word())) return KK_ERR_CUDA;
  return done(kk::launch_qk_norm_rope(a, stream));
}

kk_status kk_kv8_write(const kk_kcache_desc* kc, float* k_scale, const kk_kcache_desc* vc, float* v_scale,
                       const kk_block_table* bt, int32_t layer, int32_t num_layers, int32_t dtype, const kk_rows* k,
                       const kk_rows* v, const int32_t* token_offsets, int32_t max_new, int32_t num_nodes,
                       cudaStream_t stream) {
  kk::Write8Args a = {};
  kk_status st = kk::check_block_table(bt, &a.bt);
  if (st != KK_OK) return st;
  if (dtype != KK_BF16 && dtype != KK_F32) return KK_ERR_INVALID;
  const int es = dtype == KK_F32 ? 4 : 2;
  if ((!kc && !vc) || (kc == nullptr) != (k == nullptr) || (vc == nullptr) != (v == nullptr)) return KK_ERR_INVALID;
  auto side = [&](const kk_kcache_desc* desc, float* scale, const kk_rows* src) {
    kk::KCache c;
    kk_status s = check_cache8(desc, &c);
    if (s != KK_OK || (s = check_rows(src, es, num_nodes)) != KK_OK) return s;
    if (!scale || (a.sides && !same_sizes(c, a.kc))) return KK_ERR_INVALID;
    if (!aligned(scale, 4)) return KK_ERR_UNSUPPORTED;
    a.kc = c;
    a.side[a.sides++] = kk::Write8Side{src->base, src->stride_layer, src->stride_node, src->stride_head,
                                       const_cast<void*>(c.base), c.sL, c.sP, c.sH, c.sT, scale};
    return KK_OK;
  };
  if (kc && (st = side(kc, k_scale, k)) != KK_OK) return st;
  if (vc && (st = side(vc, v_scale, v)) != KK_OK) return st;
  if (layer < 0 || num_layers < 1 || layer > a.kc.L - num_layers || max_new < 1 || num_nodes < 0) return KK_ERR_INVALID;
  if (!token_offsets && (long long)max_new * a.bt.R != num_nodes) return KK_ERR_INVALID;
  if (!aligned(token_offsets, 4) || max_new > kk::kMaxTokens) return KK_ERR_UNSUPPORTED;
  if (a.bt.R == 0 || num_nodes == 0) return KK_OK;
  a.f32 = dtype == KK_F32;
  a.layer = layer;
  a.layers = num_layers;
  a.token_off = token_offsets;
  a.max_new = max_new;
  a.num_nodes = num_nodes;
  if (!(a.err = kk::device_error_word())) return KK_ERR_CUDA;
  return done(kk::launch_kv8_write(a, stream));
}

size_t kk_tree_attn_kv8_workspace_bytes(const kk_kcache_desc* kc, const kk_block_table* bt, int32_t max_nodes,
                                        int32_t num_q_heads) {
  kk::KCache c = {};
  if (check_cache8(kc, &c) != KK_OK || !bt || max_nodes < 1 || max_nodes > kk::kMaxNodes || num_q_heads < 1 ||
      num_q_heads % c.H || bt->num_requests < 0 || bt->num_requests > 65535)
    return 0;
  return kk::attn_workspace_bytes(c, bt->num_requests, max_nodes, num_q_heads / c.H);
}

kk_status kk_tree_attn_kv8(const kk_kcache_desc* kc, const float* k_scale, const kk_kcache_desc* vc,
                           const float* v_scale, const kk_block_table* bt, int32_t layer, const kk_selection* sel,
                           const kk_tree* tree, const void* q, int64_t q_stride_node, int64_t q_stride_head,
                           int32_t num_q_heads, float scale, void* out, float* lse, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  kk::AttnArgs a = {};
  kk_status st = check_cache8(kc, &a.kc);
  if (st != KK_OK || (st = check_cache8(vc, &a.vc)) != KK_OK) return st;
  if (!same_sizes(a.kc, a.vc) || !k_scale || !v_scale) return KK_ERR_INVALID;
  if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return KK_ERR_UNSUPPORTED;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return kk::tree_attn_call(&a, bt, layer, sel, tree, q, q_stride_node, q_stride_head, num_q_heads, scale, out, lse,
                            workspace, workspace_bytes, stream);
}

kk_status kk_pages_alloc(const int32_t* refs_in, int32_t* refs_out, int32_t num_pages, const int32_t* want, int32_t n,
                         int32_t* out, cudaStream_t stream) {
  const kk_status st = check_refs(refs_in, refs_out, num_pages);
  if (st != KK_OK) return st;
  if (n < 0 || (n > 0 && !out)) return KK_ERR_INVALID;
  if (!aligned(want, 4) || !aligned(out, 4) || n > kMaxInts) return KK_ERR_UNSUPPORTED;
  if (collide({{out, n}, {refs_out, num_pages}}, {{want, n}}) ||
      (refs_in != refs_out && share({out, n}, {refs_in, num_pages})))
    return KK_ERR_INVALID;
  if (n == 0 && refs_in == refs_out) return KK_OK;
  int* err = kk::device_error_word();
  if (!err) return KK_ERR_CUDA;
  return done(kk::launch_pages_alloc(refs_in, refs_out, num_pages, want, n, out, err, stream));
}

kk_status kk_pages_free(const kk_block_table* bt, const int32_t* refs_in, int32_t* refs_out, int32_t num_pages,
                        cudaStream_t stream) {
  kk::Table t;
  kk_status st = kk::check_block_table(bt, &t);
  if (st != KK_OK || (st = check_refs(refs_in, refs_out, num_pages)) != KK_OK) return st;
  if (collide({{refs_out, num_pages}}, {{t.offsets, t.R + 1ll}, {t.pages, t.max_blocks > 0 ? 1 : 0}}))
    return KK_ERR_INVALID;
  if (t.R == 0 && refs_in == refs_out) return KK_OK;
  int* err = kk::device_error_word();
  if (!err) return KK_ERR_CUDA;
  return done(kk::launch_pages_free(t, refs_in, refs_out, num_pages, err, stream));
}

size_t kk_pages_fork_workspace_bytes(int32_t num_requests, int32_t F) {
  if (num_requests < 0 || F < 0) return 0;
  return up256(8ull * num_requests) + up256(4ull * F + 4) + up256(8ull * F) + 256;
}

kk_status kk_pages_fork(const kk_block_table* bt, int32_t block_size, const int32_t* parent, int32_t F,
                        int32_t keep_parents, const int32_t* refs_in, int32_t* refs_out, int32_t num_pages,
                        int32_t* child_pages, int64_t child_capacity, int32_t* child_offsets, int32_t* child_lens,
                        const kk_page_array* arrays, int32_t n_arrays, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  kk::ForkArgs a = {};
  kk::PageArrays pa = {};
  kk_status st = kk::check_block_table(bt, &a.bt);
  if (st != KK_OK || (st = check_refs(refs_in, refs_out, num_pages)) != KK_OK ||
      (st = check_arrays(arrays, n_arrays, &pa)) != KK_OK)
    return st;
  if (block_size < 1 || F < 0 || !child_offsets || (F > 0 && (!parent || !child_lens))) return KK_ERR_INVALID;
  const long long most = (long long)F * a.bt.max_blocks;
  if (child_capacity < most || (most > 0 && !child_pages)) return KK_ERR_INVALID;
  if (most > 0x7FFFFFFFll) return KK_ERR_UNSUPPORTED;
  if (!aligned(parent, 4) || !aligned(child_pages, 4) || !aligned(child_offsets, 4) || !aligned(child_lens, 4))
    return KK_ERR_UNSUPPORTED;
  // children are laid out, and counts moved, while their parents are read (how long bt's pages are is not known here)
  if (collide({{child_pages, most}, {child_offsets, F + 1ll}, {child_lens, F}, {refs_out, num_pages}},
              {{parent, F},
               {a.bt.offsets, a.bt.R + 1ll},
               {a.bt.seq_lens, a.bt.R},
               {a.bt.pages, a.bt.max_blocks > 0 ? 1 : 0}}) ||
      (refs_in != refs_out &&
       collide({{child_pages, most}, {child_offsets, F + 1ll}, {child_lens, F}}, {{refs_in, num_pages}})))
    return KK_ERR_INVALID;
  if (!workspace || workspace_bytes < kk_pages_fork_workspace_bytes(a.bt.R, F)) return KK_ERR_INVALID;
  if (!aligned(workspace, 256)) return KK_ERR_UNSUPPORTED;
  a.bs = block_size;
  a.F = F;
  a.keep = keep_parents != 0;
  a.num_pages = num_pages;
  a.parent = parent;
  a.refs_in = refs_in;
  a.refs_out = refs_out;
  a.child_pages = child_pages;
  a.child_offsets = child_offsets;
  a.child_lens = child_lens;
  char* p = static_cast<char*>(workspace);
  a.kids = reinterpret_cast<int*>(p);
  a.first = a.kids + a.bt.R;
  p += up256(8ull * a.bt.R);
  a.at = reinterpret_cast<int*>(p);
  p += up256(4ull * F + 4);
  a.pairs = reinterpret_cast<int2*>(p);
  p += up256(8ull * F);
  a.n_pairs = reinterpret_cast<int*>(p);
  if (!(a.err = kk::device_error_word())) return KK_ERR_CUDA;
  return done(kk::launch_pages_fork(a, pa, stream));
}

size_t kk_pages_compact_workspace_bytes(int32_t num_pages) {
  return num_pages < 1 ? 0 : up256(8ull * (num_pages / 2 + 1)) + 256;
}

kk_status kk_pages_compact(const int32_t* refs_in, int32_t* refs_out, int32_t num_pages, const int32_t* pages_in,
                           int32_t* pages_out, int64_t n, int32_t* remap, int32_t* used, const kk_page_array* arrays,
                           int32_t n_arrays, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  kk::CompactArgs a = {};
  kk::PageArrays pa = {};
  kk_status st = check_refs(refs_in, refs_out, num_pages);
  if (st != KK_OK || (st = check_arrays(arrays, n_arrays, &pa)) != KK_OK) return st;
  if (n < 0 || (n > 0 && (!pages_in || !pages_out)) || !remap || !used) return KK_ERR_INVALID;
  if (!aligned(pages_in, 4) || !aligned(pages_out, 4) || !aligned(remap, 4) || !aligned(used, 4))
    return KK_ERR_UNSUPPORTED;
  if ((pages_in != pages_out && share({pages_in, n}, {pages_out, n})) ||  // the same, or apart
      collide({{pages_out, n}, {remap, num_pages}, {used, 1}, {refs_out, num_pages}}, {{nullptr, 0}}) ||
      (refs_in != refs_out && collide({{pages_out, n}, {remap, num_pages}, {used, 1}}, {{refs_in, num_pages}})) ||
      (pages_in != pages_out && collide({{remap, num_pages}, {used, 1}, {refs_out, num_pages}}, {{pages_in, n}})))
    return KK_ERR_INVALID;
  if (!workspace || workspace_bytes < kk_pages_compact_workspace_bytes(num_pages)) return KK_ERR_INVALID;
  if (!aligned(workspace, 256)) return KK_ERR_UNSUPPORTED;
  a.num_pages = num_pages;
  a.refs_in = refs_in;
  a.refs_out = refs_out;
  a.pages_in = pages_in;
  a.pages_out = pages_out;
  a.n = n;
  a.remap = remap;
  a.used = used;
  a.pairs = static_cast<int2*>(workspace);
  a.n_pairs = reinterpret_cast<int*>(static_cast<char*>(workspace) + up256(8ull * (num_pages / 2 + 1)));
  if (!(a.err = kk::device_error_word())) return KK_ERR_CUDA;
  return done(kk::launch_pages_compact(a, pa, stream));
}

}  // extern "C"
