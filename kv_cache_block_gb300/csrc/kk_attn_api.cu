// C ABI of the attention, attention-mass and eviction calls (include/kk.h):
// argument checks on the host, then launches.
#include <cmath>
#include <cstdlib>

#include "../../include/kk.h"

#include "kk_attn.cuh"
#include "kk_internal.h"

namespace kk {
// kk_api.cu
kk_status check_kcache_desc(const kk_kcache_desc* kc, KCache* out);
kk_status check_block_table(const kk_block_table* bt, Table* out);
}  // namespace kk

namespace {

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool same_sizes(const kk::KCache& a, const kk::KCache& b) {
  return a.dtype == b.dtype && a.L == b.L && a.H == b.H && a.D == b.D && a.bs == b.bs && a.num_pages == b.num_pages;
}

// A strided [node][head][D] tensor: 16-byte rows.
bool rows_ok(const void* p, int64_t sn, int64_t sh, int es) {
  return aligned(p, 16) && sn >= 0 && sh >= 0 && sn * es % 16 == 0 && sh * es % 16 == 0;
}

// Table, nodes and queries, as the attention calls and kk_attn_mass share them; a->kc is set.
kk_status common_args(const kk_block_table* bt, int32_t layer, const kk_tree* tree, const void* q, int64_t q_sn,
                      int64_t q_sh, int32_t Hq, float scale, kk::AttnArgs* a) {
  const kk_status st = kk::check_block_table(bt, &a->bt);
  if (st != KK_OK) return st;
  if (layer < 0 || layer >= a->kc.L || !tree || !std::isfinite(scale)) return KK_ERR_INVALID;
  if (tree->max_nodes < 1 || tree->max_nodes > kk::kMaxNodes || tree->total_nodes < 0) return KK_ERR_INVALID;
  if (!tree->node_offsets && (long long)tree->max_nodes * a->bt.R != tree->total_nodes) return KK_ERR_INVALID;
  if (Hq < 1 || Hq % a->kc.H) return KK_ERR_INVALID;
  const int es = a->kc.dtype == KK_F32 ? 4 : 2;
  if (tree->total_nodes > 0) {
    if (!q) return KK_ERR_INVALID;
    if (!rows_ok(q, q_sn, q_sh, es)) return KK_ERR_UNSUPPORTED;
  }
  if ((long long)tree->max_nodes * Hq > (1 << 20) || !aligned(tree->node_offsets, 4)) return KK_ERR_UNSUPPORTED;
  a->layer = layer;
  a->node_off = tree->node_offsets;
  a->max_nodes = tree->max_nodes;
  a->total_nodes = tree->total_nodes;
  a->mask_words = (tree->max_nodes + 31) / 32;
  a->q = q;
  a->q_sn = q_sn;
  a->q_sh = q_sh;
  a->Hq = Hq;
  a->G = Hq / a->kc.H;
  a->scale_log2 = scale * 1.44269504088896341f;
  a->wait_ns = kk::wait_limit_ns();
  return KK_OK;
}

kk_status done(cudaError_t e) {
  return e == cudaSuccess ? KK_OK : e == cudaErrorNotSupported ? KK_ERR_UNSUPPORTED : KK_ERR_CUDA;
}

}  // namespace

namespace kk {
// kk_tree_attn and kk_tree_attn_kv8 (kk_serve_api.cu) once the caches are checked: a->kc, a->vc and the scales are set.
kk_status tree_attn_call(AttnArgs* a, const kk_block_table* bt, int32_t layer, const kk_selection* sel,
                         const kk_tree* tree, const void* q, int64_t q_sn, int64_t q_sh, int32_t Hq, float scale,
                         void* out, float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const kk_status st = common_args(bt, layer, tree, q, q_sn, q_sh, Hq, scale, a);
  if (st != KK_OK) return st;
  const int es = a->kc.dtype == KK_F32 ? 4 : 2;
  if ((tree->k == nullptr) != (tree->v == nullptr)) return KK_ERR_INVALID;
  if (tree->k) {
    if (!rows_ok(tree->k, tree->k_stride_node, tree->k_stride_head, es) ||
        !rows_ok(tree->v, tree->v_stride_node, tree->v_stride_head, es) || !aligned(tree->mask, 4))
      return KK_ERR_UNSUPPORTED;
    a->dk = tree->k;
    a->dv = tree->v;
    a->dk_sn = tree->k_stride_node;
    a->dk_sh = tree->k_stride_head;
    a->dv_sn = tree->v_stride_node;
    a->dv_sh = tree->v_stride_head;
    a->mask = tree->mask;
  }
  if (sel) {
    if (!sel->pages || !sel->logical || !sel->count || sel->K < 1) return KK_ERR_INVALID;
    if (!aligned(sel->pages, 4) || !aligned(sel->logical, 4) || !aligned(sel->count, 4)) return KK_ERR_UNSUPPORTED;
    a->sel_pages = sel->pages;
    a->sel_logical = sel->logical;
    a->sel_count = sel->count;
    a->selK = sel->K;
  }
  if (a->bt.R == 0 || a->total_nodes == 0) return KK_OK;
  if (!out) return KK_ERR_INVALID;
  if (!aligned(out, 16) || !aligned(lse, 4)) return KK_ERR_UNSUPPORTED;
  if ((long long)a->bt.R * a->kc.H * a->max_nodes * a->G > 0x7FFFFFFFll) return KK_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < attn_workspace_bytes(a->kc, a->bt.R, a->max_nodes, a->G)) return KK_ERR_INVALID;
  if (!aligned(workspace, 256)) return KK_ERR_UNSUPPORTED;
  a->out = out;
  a->lse = lse;
  a->ws = static_cast<float*>(workspace);
  if (!(a->err = device_error_word())) return KK_ERR_CUDA;
  return done(launch_tree_attn(*a, stream));
}
}  // namespace kk

extern "C" {

size_t kk_tree_attn_workspace_bytes(const kk_kcache_desc* kc, const kk_block_table* bt, int32_t max_nodes,
                                    int32_t num_q_heads) {
  if (!kc || !bt || kc->num_kv_heads < 1 || max_nodes < 1 || max_nodes > kk::kMaxNodes || num_q_heads < 1 ||
      num_q_heads % kc->num_kv_heads)
    return 0;
  kk::KCache c = {};
  if (kk::check_kcache_desc(kc, &c) != KK_OK) return 0;
  if (bt->num_requests < 0 || bt->num_requests > 65535) return 0;
  return kk::attn_workspace_bytes(c, bt->num_requests, max_nodes, num_q_heads / c.H);
}

kk_status kk_tree_attn(const kk_kcache_desc* kc, const kk_kcache_desc* vc, const kk_block_table* bt, int32_t layer,
                       const kk_selection* sel, const kk_tree* tree, const void* q, int64_t q_stride_node,
                       int64_t q_stride_head, int32_t num_q_heads, float scale, void* out, float* lse,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  kk::AttnArgs a = {};
  kk_status st = kk::check_kcache_desc(kc, &a.kc);
  if (st != KK_OK || (st = kk::check_kcache_desc(vc, &a.vc)) != KK_OK) return st;
  if (!same_sizes(a.kc, a.vc)) return KK_ERR_INVALID;
  return kk::tree_attn_call(&a, bt, layer, sel, tree, q, q_stride_node, q_stride_head, num_q_heads, scale, out, lse,
                            workspace, workspace_bytes, stream);
}

kk_status kk_attn_mass(const kk_kcache_desc* kc, const kk_block_table* bt, int32_t layer, const kk_tree* tree,
                       const void* q, int64_t q_stride_node, int64_t q_stride_head, int32_t num_q_heads, float scale,
                       const float* lse, const float* row_w, const int32_t* row_lens, const int32_t* old_lens,
                       float decay, const float* mass_in, float* mass_out, cudaStream_t stream) {
  kk::AttnArgs a = {};
  kk_status st = kk::check_kcache_desc(kc, &a.kc);
  if (st != KK_OK) return st;
  if ((st = common_args(bt, layer, tree, q, q_stride_node, q_stride_head, num_q_heads, scale, &a)) != KK_OK) return st;
  if (!std::isfinite(decay)) return KK_ERR_INVALID;
  if (a.bt.R == 0) return KK_OK;
  if (!mass_out || (a.total_nodes > 0 && !lse)) return KK_ERR_INVALID;
  if (!aligned(mass_in, 4) || !aligned(mass_out, 4) || !aligned(lse, 4) || !aligned(row_w, 4) ||
      !aligned(row_lens, 4) || !aligned(old_lens, 4))
    return KK_ERR_UNSUPPORTED;
  a.lse = const_cast<float*>(lse);
  a.row_w = row_w;
  a.row_lens = row_lens;
  a.old_lens = old_lens;
  a.decay = decay;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  if (!(a.err = kk::device_error_word())) return KK_ERR_CUDA;
  return done(kk::launch_attn_mass(a, stream));
}

static kk_status evict_args(const kk_kcache_desc* kc, const kk_block_table* bt, int32_t keep, kk::KCache* c,
                            kk::Table* t) {
  kk_status st = kk::check_kcache_desc(kc, c);
  if (st != KK_OK) return st;
  if ((st = kk::check_block_table(bt, t)) != KK_OK) return st;
  if (keep < 1) return KK_ERR_INVALID;
  if ((long long)t->R * c->L * c->H > 0x7FFFFFFFll || keep > kk::kMaxTokens) return KK_ERR_UNSUPPORTED;
  return KK_OK;
}

kk_status kk_evict_select(const kk_kcache_desc* kc, const kk_block_table* bt, const float* mass, int32_t sinks,
                          int32_t recent, int32_t keep, int32_t* kept, int32_t* new_lens, cudaStream_t stream) {
  kk::KCache c;
  kk::Table t;
  const kk_status st = evict_args(kc, bt, keep, &c, &t);
  if (st != KK_OK) return st;
  if (sinks < 0 || recent < 0 || (long long)sinks + recent > keep) return KK_ERR_INVALID;
  if (t.R == 0) return KK_OK;
  if (!mass || !kept) return KK_ERR_INVALID;
  if (!aligned(mass, 4) || !aligned(kept, 4) || !aligned(new_lens, 4)) return KK_ERR_UNSUPPORTED;
  // other CTAs of a request still read its length when the first one writes the new one
  const intptr_t apart = reinterpret_cast<intptr_t>(new_lens) - reinterpret_cast<intptr_t>(t.seq_lens);
  if (new_lens && std::llabs(apart) < 4ll * t.R) return KK_ERR_INVALID;
  int* err = kk::device_error_word();
  if (!err) return KK_ERR_CUDA;
  return done(kk::launch_evict_select(c, t, mass, sinks, recent, keep, kept, new_lens, err, stream));
}

kk_status kk_evict_compact(const kk_kcache_desc* kc, const kk_kcache_desc* vc, const kk_block_table* bt,
                           const int32_t* kept, int32_t keep, const float* mass_in, float* mass_out,
                           const int32_t* dst_pages, cudaStream_t stream) {
  kk::KCache c, v = {};
  kk::Table t;
  kk_status st = evict_args(kc, bt, keep, &c, &t);
  if (st != KK_OK) return st;
  if (vc) {
    if ((st = kk::check_kcache_desc(vc, &v)) != KK_OK) return st;
    if (!same_sizes(c, v)) return KK_ERR_INVALID;
  }
  if ((mass_in == nullptr) != (mass_out == nullptr)) return KK_ERR_INVALID;
  if (t.R == 0) return KK_OK;
  if (!kept) return KK_ERR_INVALID;
  if (!aligned(kept, 4) || !aligned(mass_in, 4) || !aligned(mass_out, 4) || !aligned(dst_pages, 4))
    return KK_ERR_UNSUPPORTED;
  int* err = kk::device_error_word();
  if (!err) return KK_ERR_CUDA;
  return done(kk::launch_evict_compact(c, v, t, kept, keep, mass_in, mass_out, dst_pages, err, stream));
}

}  // extern "C"
