// kda_tree_api.cu -- the C ABI of the tree-verification and paged-cache calls (include/kda.h, include/mla.h):
// host-side validation, then kernel launches, as kda_api.cu does for the rest.
#include "../../include/kda.h"
#include "../../include/mla.h"

#include <cstdint>
#include <cstring>

#include "kda_internal.h"
#include "kda_trace.h"

namespace kda {
kda_status validate_params(const kda_params *p);  // kda_api.cu
void note_launches(int n);
int *device_error();
}  // namespace kda

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given(const void *p) { return p != nullptr && aligned16(p); }
bool optional(const void *p) { return p == nullptr || aligned16(p); }

kda_status done(cudaError_t e, int launches) {
  kda::note_launches(launches);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

constexpr int64_t kMaxTreeRows = (int64_t)1 << 22;  // 65535 sequences of 64 nodes

bool page_size_known(int n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }

// What the paged calls share; `tables`: the call reads or writes page tables and lengths.
kda_status check_cache(const void *pool, int n_layers, int n_pages, int page_size, bool tables,
                       const int32_t *table, int max_pages, const int32_t *lengths) {
  if (!given(pool) || n_layers < 1 || n_layers > 4096 || n_pages < 1 || page_size < 1)
    return KDA_ERR_INVALID_ARG;
  if (tables && (!given(table) || !given(lengths) || max_pages < 1 || max_pages > 1 << 20))
    return KDA_ERR_INVALID_ARG;
  if (!page_size_known(page_size)) return KDA_ERR_UNSUPPORTED;
  if (n_pages > 1 << 26) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda::PagedCache cache_args(const void *pool, int n_layers, int n_pages, int page_size,
                           const int32_t *table, int max_pages, const int32_t *lengths) {
  kda::PagedCache c;
  c.pool = const_cast<void *>(pool);
  c.n_layers = n_layers, c.n_pages = n_pages, c.page_size = page_size;
  c.table = table, c.max_pages = max_pages, c.lengths = lengths;
  c.err = kda::device_error();
  return c;
}

kda_status check_tree_call(const kda_params *p, const void *x_raw, const void *conv_w,
                           const void *conv_state, const float *g, const float *beta,
                           const void *state, int n_slots, const int32_t *slot_idx,
                           const int32_t *cu_nodes, const int32_t *parent, int n_seqs,
                           int64_t total_nodes) {
  kda_status st = kda::validate_params(p);
  if (st != KDA_OK) return st;
  if (n_seqs < 0 || n_seqs > 65535 || n_slots < 0 || total_nodes < 0 || total_nodes > kMaxTreeRows)
    return KDA_ERR_INVALID_ARG;
  if (n_seqs == 0 || total_nodes == 0) return total_nodes == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
  if (!given(x_raw) || !given(conv_w) || !given(conv_state) || !given(g) || !given(beta) ||
      !given(state) || !given(cu_nodes) || !given(parent) || !optional(slot_idx))
    return KDA_ERR_INVALID_ARG;
  if (!slot_idx && n_slots < n_seqs) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda::TreeArgs tree_args(const kda_params *p, const void *x_raw, const void *conv_w,
                        void *conv_state, const float *g, const float *beta, void *state,
                        int n_slots, const int32_t *slot_idx, const int32_t *cu_nodes,
                        const int32_t *parent, int n_seqs, int64_t total_nodes) {
  kda::TreeArgs a;
  std::memset(&a, 0, sizeof a);
  a.H = p->H, a.n_seqs = n_seqs, a.n_slots = n_slots, a.max_nodes = 64, a.total = total_nodes;
  a.scale = p->scale, a.l2_eps = p->l2_eps, a.norm_eps = p->norm_eps, a.g_min = p->g_min;
  a.qk_l2norm = p->qk_l2norm ? 1 : 0;
  a.x_raw = x_raw, a.conv_w = conv_w, a.conv_state = conv_state, a.g = g, a.beta = beta;
  a.state = state, a.slot_idx = slot_idx, a.cu_nodes = cu_nodes, a.parent = parent;
  a.err = kda::device_error();
  return a;
}

}  // namespace

extern "C" {

kda_status kda_tree_verify(const kda_params *p, const void *x_raw, const void *conv_w,
                           const void *conv_state, const float *g, const float *beta,
                           const void *state, int n_slots, const int32_t *slot_idx,
                           const int32_t *cu_nodes, const int32_t *parent, int n_seqs,
                           int64_t total_nodes, int max_nodes, const void *gate_logit,
                           const float *norm_w, void *out, cudaStream_t stream) {
  KDA_TRACE(TR_TREE_VERIFY);
  kda_status st = check_tree_call(p, x_raw, conv_w, conv_state, g, beta, state, n_slots, slot_idx,
                                  cu_nodes, parent, n_seqs, total_nodes);
  if (st != KDA_OK || total_nodes == 0) return st;
  if (max_nodes < 1 || max_nodes > 64 || !given(out) || !optional(gate_logit) || !optional(norm_w))
    return KDA_ERR_INVALID_ARG;
  kda::TreeArgs a = tree_args(p, x_raw, conv_w, const_cast<void *>(conv_state), g, beta,
                              const_cast<void *>(state), n_slots, slot_idx, cu_nodes, parent, n_seqs,
                              total_nodes);
  a.max_nodes = max_nodes;
  // e^g below the normal fp32 range (2^-126) counts as 0: the kernel takes differences of sums of g along
  // a path, which would be NaN of two infinities, and counts their multiples of 32 (64 nodes x 127.1 / 32) in a byte
  if (a.g_min < -88.1f) a.g_min = -88.1f;
  a.gate = gate_logit, a.norm_w = norm_w, a.out = out;
  return done(kda::launch_tree(a, false, p->d_k, p->io_dtype == KDA_BF16, p->state_dtype == KDA_BF16, stream), 1);
}

kda_status kda_tree_accept(const kda_params *p, const void *x_raw, const void *conv_w,
                           void *conv_state, const float *g, const float *beta, void *state,
                           int n_slots, const int32_t *slot_idx, const int32_t *cu_nodes,
                           const int32_t *parent, int n_seqs, int64_t total_nodes,
                           const int32_t *accept_node, cudaStream_t stream) {
  KDA_TRACE(TR_TREE_ACCEPT);
  kda_status st = check_tree_call(p, x_raw, conv_w, conv_state, g, beta, state, n_slots, slot_idx,
                                  cu_nodes, parent, n_seqs, total_nodes);
  if (st != KDA_OK || total_nodes == 0) return st;
  if (!given(accept_node)) return KDA_ERR_INVALID_ARG;
  kda::TreeArgs a = tree_args(p, x_raw, conv_w, conv_state, g, beta, state, n_slots, slot_idx,
                              cu_nodes, parent, n_seqs, total_nodes);
  a.accept = accept_node;
  return done(kda::launch_tree(a, true, p->d_k, p->io_dtype == KDA_BF16, p->state_dtype == KDA_BF16, stream), 1);
}

kda_status mla_tree_mask(const int32_t *parent, const int32_t *cu_nodes, int n_seqs,
                         int64_t total_nodes, int64_t *mask, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_TREE_MASK);
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows) return KDA_ERR_INVALID_ARG;
  if (total_nodes == 0) return KDA_OK;
  if (n_seqs == 0 || !given(parent) || !given(cu_nodes) || !given(mask)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_tree_mask(parent, cu_nodes, n_seqs, total_nodes, mask, kda::device_error(), stream), 1);
}

size_t mla_tree_workspace_size(int n_seqs, int64_t total_nodes, int H) {
  if (n_seqs < 1 || n_seqs > 65535 || total_nodes < 1 || total_nodes > kMaxTreeRows || H < 1 || H > 128) return 0;
  return kda::mla_tree_ws_bytes(n_seqs, total_nodes, H);
}

// The checks of the two tree attention calls; fills *a.
static kda_status tree_attention(const void *q_cat, int H, const void *pool, int n_pages, int page_size,
                                 const int32_t *page_table, int max_pages, const int32_t *lengths,
                                 const int32_t *cu_nodes, int n_seqs, int64_t total_nodes,
                                 const int64_t *mask, float scale, void *z, kda_dtype z_dtype,
                                 void *workspace, size_t ws_bytes, kda::TreeAttnArgs *a) {
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows || H < 1 || H > 128)
    return KDA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < 1e30f) || (z_dtype != KDA_F32 && z_dtype != KDA_BF16)) return KDA_ERR_INVALID_ARG;
  if (total_nodes == 0) return KDA_OK;
  kda_status st = check_cache(pool, 1, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st != KDA_OK) return st;
  if (n_seqs == 0 || !given(q_cat) || !given(cu_nodes) || !given(z) || !optional(mask) || !optional(workspace))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < kda::mla_tree_ws_bytes(n_seqs, total_nodes, H)) return KDA_ERR_WORKSPACE;
  if (!kda::mla_latent_supported()) return KDA_ERR_UNSUPPORTED;
  std::memset(a, 0, sizeof *a);
  a->c = cache_args(pool, 1, n_pages, page_size, page_table, max_pages, lengths);
  a->n_seqs = n_seqs, a->H = H, a->total = total_nodes;
  a->scale_log2 = scale * 1.4426950408889634f;
  a->q = q_cat, a->cu_nodes = cu_nodes, a->mask = mask, a->z = z, a->z_bf16 = z_dtype == KDA_BF16;
  a->ws = workspace, a->err = a->c.err;
  return KDA_OK;
}

kda_status mla_tree_latent(const void *q_cat, int H, const void *pool, int n_pages, int page_size,
                           const int32_t *page_table, int max_pages, const int32_t *lengths,
                           const int32_t *cu_nodes, int n_seqs, int64_t total_nodes,
                           const int64_t *mask, float scale, void *z, kda_dtype z_dtype,
                           void *workspace, size_t ws_bytes, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_TREE_LATENT);
  kda::TreeAttnArgs a;
  kda_status st = tree_attention(q_cat, H, pool, n_pages, page_size, page_table, max_pages, lengths, cu_nodes,
                                 n_seqs, total_nodes, mask, scale, z, z_dtype, workspace, ws_bytes, &a);
  if (st != KDA_OK || total_nodes == 0) return st;
  int launches = 0;
  const cudaError_t e = kda::launch_mla_tree(a, &launches, stream);
  return done(e, launches);
}

kda_status mla_tree_latent_lse(const void *q_cat, int H, const void *pool, int n_pages, int page_size,
                               const int32_t *page_table, int max_pages, const int32_t *lengths,
                               const int32_t *cu_nodes, int n_seqs, int64_t total_nodes,
                               const int64_t *mask, float scale, void *z, kda_dtype z_dtype, float *lse,
                               void *workspace, size_t ws_bytes, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_TREE_LATENT_LSE);
  if (total_nodes > 0 && !given(lse)) return KDA_ERR_INVALID_ARG;
  kda::TreeAttnArgs a;
  kda_status st = tree_attention(q_cat, H, pool, n_pages, page_size, page_table, max_pages, lengths, cu_nodes,
                                 n_seqs, total_nodes, mask, scale, z, z_dtype, workspace, ws_bytes, &a);
  if (st != KDA_OK || total_nodes == 0) return st;
  a.lse = lse;
  int launches = 0;
  const cudaError_t e = kda::launch_mla_tree(a, &launches, stream);
  return done(e, launches);
}

// What the decode calls put around the attention: the projections see one query row per node.
static kda_status node_projections(const void *q_nope, const void *q_rope, const void *w_uk, const void *w_uv,
                                   const void *gate_logit, void *out, void *q_cat, float *z, int64_t total_nodes,
                                   kda::MlaArgs *m) {
  if (!given(q_nope) || !given(q_rope) || !given(w_uk) || !given(w_uv) || !given(gate_logit) || !given(out))
    return KDA_ERR_INVALID_ARG;
  std::memset(m, 0, sizeof *m);
  m->B = (int)total_nodes;
  m->q_nope = q_nope, m->q_rope = q_rope, m->w_uk = w_uk, m->w_uv = w_uv, m->gate = gate_logit;
  m->q_cat = q_cat, m->z = z, m->out = out, m->err = kda::device_error();
  return KDA_OK;
}

kda_status mla_tree_decode(const void *q_nope, const void *q_rope, const void *w_uk, const void *w_uv,
                           const void *pool, int n_pages, int page_size, const int32_t *page_table,
                           int max_pages, const int32_t *lengths, const int32_t *cu_nodes, int n_seqs,
                           int64_t total_nodes, const int64_t *mask, const void *gate_logit, float scale,
                           void *q_cat, float *z, void *out, void *workspace, size_t ws_bytes,
                           cudaStream_t stream) {
  KDA_TRACE(TR_MLA_TREE_DECODE);
  kda::TreeAttnArgs a;
  kda::MlaArgs m;
  kda_status st = tree_attention(q_cat, 64, pool, n_pages, page_size, page_table, max_pages, lengths, cu_nodes,
                                 n_seqs, total_nodes, mask, scale, z, KDA_F32, workspace, ws_bytes, &a);
  if (st != KDA_OK || total_nodes == 0) return st;
  st = node_projections(q_nope, q_rope, w_uk, w_uv, gate_logit, out, q_cat, z, total_nodes, &m);
  if (st != KDA_OK) return st;
  int launches = 0;
  cudaError_t e = kda::launch_mla_absorb(m, stream);
  if (e == cudaSuccess) e = kda::launch_mla_tree(a, &launches, stream);
  if (e == cudaSuccess) e = kda::launch_mla_up_gate(m, stream);
  return done(e, launches + 2);
}

kda_status mla_tree_decode_lse(const void *q_nope, const void *q_rope, const void *w_uk, const void *w_uv,
                               const void *pool, int n_pages, int page_size, const int32_t *page_table,
                               int max_pages, const int32_t *lengths, const int32_t *cu_nodes, int n_seqs,
                               int64_t total_nodes, const int64_t *mask, const void *gate_logit, float scale,
                               void *q_cat, float *z, void *out, float *lse, void *workspace, size_t ws_bytes,
                               cudaStream_t stream) {
  KDA_TRACE(TR_MLA_TREE_DECODE_LSE);
  kda::TreeAttnArgs a;
  kda::MlaArgs m;
  kda_status st = node_projections(q_nope, q_rope, w_uk, w_uv, gate_logit, out, q_cat, z, total_nodes, &m);
  if (total_nodes > 0 && (st != KDA_OK || !given(lse))) return KDA_ERR_INVALID_ARG;
  st = tree_attention(q_cat, 64, pool, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs, total_nodes,
                      mask, scale, z, KDA_F32, workspace, ws_bytes, &a);
  if (st != KDA_OK || total_nodes == 0) return st;
  a.lse = lse;
  int launches = 0;
  cudaError_t e = kda::launch_mla_absorb(m, stream);
  if (e == cudaSuccess) e = kda::launch_mla_tree(a, &launches, stream);
  if (e == cudaSuccess) e = kda::launch_mla_up_gate(m, stream);
  return done(e, launches + 2);
}

kda_status mla_cache_append(void *pool, int n_layers, int n_pages, int page_size, const int32_t *page_table,
                            int max_pages, const int32_t *lengths, const int32_t *cu_rows, int n_seqs,
                            int64_t total_rows, const void *rows, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_CACHE_APPEND);
  if (n_seqs < 0 || n_seqs > 65535 || total_rows < 0 || total_rows > INT32_MAX) return KDA_ERR_INVALID_ARG;
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st != KDA_OK || total_rows == 0) return st;
  if (n_seqs == 0 || !given(cu_rows) || !given(rows)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_cache_append(cache_args(pool, n_layers, n_pages, page_size, page_table, max_pages, lengths),
                                       cu_rows, n_seqs, total_rows, rows, stream), 1);
}

kda_status mla_cache_accept(void *pool, int n_layers, int n_pages, int page_size, const int32_t *page_table,
                            int max_pages, const int32_t *lengths, const int32_t *cu_nodes, int n_seqs,
                            int64_t total_nodes, const int32_t *parent, const int32_t *accept_node,
                            int32_t *new_lengths, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_CACHE_ACCEPT);
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows) return KDA_ERR_INVALID_ARG;
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st != KDA_OK || n_seqs == 0) return st;
  if (!given(cu_nodes) || (total_nodes > 0 && !given(parent)) || !given(accept_node) || !given(new_lengths))
    return KDA_ERR_INVALID_ARG;
  return done(kda::launch_cache_accept(cache_args(pool, n_layers, n_pages, page_size, page_table, max_pages, lengths),
                                       cu_nodes, n_seqs, total_nodes, parent, accept_node, new_lengths, stream), 1);
}

kda_status mla_pages_copy(void *pool, int n_layers, int n_pages, int page_size, const int32_t *src,
                          const int32_t *dst, int n_copies, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_PAGES_COPY);
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, false, nullptr, 0, nullptr);
  if (st != KDA_OK) return st;
  if (n_copies < 0 || n_copies > 8192) return KDA_ERR_INVALID_ARG;  // every entry is compared with every other
  if (n_copies == 0) return KDA_OK;
  if (!given(src) || !given(dst)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_pages_copy(cache_args(pool, n_layers, n_pages, page_size, nullptr, 0, nullptr), src, dst,
                                     n_copies, stream), 1);
}

size_t mla_pages_workspace_size(int n) { return n < 1 || n > 65535 ? 0 : kda::pages_ws_bytes(n); }

// What the bookkeeping calls share.
static kda_status check_pages(int n_pages, const int32_t *refcount, const int32_t *page_table, int max_pages,
                              const int32_t *held, const int32_t *lengths, int n_slots, int n) {
  if (n < 0 || n > 65535 || n_slots < 1 || n_pages < 1 || n_pages > 1 << 26 || max_pages < 1 || max_pages > 1 << 20)
    return KDA_ERR_INVALID_ARG;
  if (!given(refcount) || !given(page_table) || !given(held) || !given(lengths)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status mla_pages_free(int n_pages, int32_t *refcount, int32_t *page_table, int max_pages, int32_t *held,
                          int32_t *lengths, int n_slots, const int32_t *slots, int n, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_PAGES_FREE);
  kda_status st = check_pages(n_pages, refcount, page_table, max_pages, held, lengths, n_slots, n);
  if (st != KDA_OK || n == 0) return st;
  if (!given(slots)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_pages_free(cache_args(nullptr, 1, n_pages, 1, page_table, max_pages, lengths), refcount,
                                     held, n_slots, slots, n, stream), 1);
}

kda_status mla_pages_fork(void *pool, int n_layers, int n_pages, int page_size, int32_t *refcount,
                          int32_t *page_table, int max_pages, int32_t *held, int32_t *lengths, int n_slots,
                          const int32_t *src, const int32_t *dst, int n, void *workspace, size_t ws_bytes,
                          cudaStream_t stream) {
  KDA_TRACE(TR_MLA_PAGES_FORK);
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st == KDA_OK) st = check_pages(n_pages, refcount, page_table, max_pages, held, lengths, n_slots, n);
  if (st != KDA_OK || n == 0) return st;
  if (!given(src) || !given(dst) || !optional(workspace)) return KDA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < kda::pages_ws_bytes(n)) return KDA_ERR_WORKSPACE;
  return done(kda::launch_pages_fork(cache_args(pool, n_layers, n_pages, page_size, page_table, max_pages, lengths),
                                     refcount, held, n_slots, src, dst, n, workspace, stream), 2);
}

kda_status mla_pages_reserve(int n_pages, int page_size, int32_t *refcount, int32_t *page_table, int max_pages,
                             int32_t *held, const int32_t *lengths, int n_slots, const int32_t *slots,
                             const int32_t *extra, int n, void *workspace, size_t ws_bytes, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_PAGES_RESERVE);
  if (page_size < 1) return KDA_ERR_INVALID_ARG;
  if (!page_size_known(page_size)) return KDA_ERR_UNSUPPORTED;
  kda_status st = check_pages(n_pages, refcount, page_table, max_pages, held, lengths, n_slots, n);
  if (st != KDA_OK || n == 0) return st;
  if (!given(slots) || !given(extra) || !optional(workspace)) return KDA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < kda::pages_ws_bytes(n)) return KDA_ERR_WORKSPACE;
  return done(kda::launch_pages_reserve(cache_args(nullptr, 1, n_pages, page_size, page_table, max_pages, lengths),
                                        refcount, held, n_slots, slots, extra, n, workspace, stream), 1);
}

kda_status mla_pages_trim(int n_pages, int page_size, int32_t *refcount, int32_t *page_table, int max_pages,
                          int32_t *held, const int32_t *lengths, int n_slots, const int32_t *slots, int n,
                          cudaStream_t stream) {
  KDA_TRACE(TR_MLA_PAGES_TRIM);
  if (page_size < 1) return KDA_ERR_INVALID_ARG;
  if (!page_size_known(page_size)) return KDA_ERR_UNSUPPORTED;
  kda_status st = check_pages(n_pages, refcount, page_table, max_pages, held, lengths, n_slots, n);
  if (st != KDA_OK || n == 0) return st;
  if (!given(slots)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_pages_trim(cache_args(nullptr, 1, n_pages, page_size, page_table, max_pages, lengths), refcount,
                                     held, n_slots, slots, n, stream), 1);
}

// ---- long contexts -----------------------------------------------------------------------------

// The checks that the two sums over query rows share; fills *a but for its results.
static kda_status key_sums(const void *q_cat, int H, const void *keys, int n_pages, int page_size,
                           const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *cu_nodes,
                           int n_seqs, int64_t total_nodes, float scale, kda::KeySumArgs *a) {
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows || H < 1 || H > 128)
    return KDA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < 1e30f)) return KDA_ERR_INVALID_ARG;
  if (total_nodes == 0) return KDA_OK;
  kda_status st = check_cache(keys, 1, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st != KDA_OK) return st;
  if (n_seqs == 0 || !given(q_cat) || !given(cu_nodes)) return KDA_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof *a);
  a->c = cache_args(keys, 1, n_pages, page_size, page_table, max_pages, lengths);
  a->n_seqs = n_seqs, a->H = H, a->total = total_nodes;
  a->scale_log2 = scale * 1.4426950408889634f;
  a->q = q_cat, a->cu_nodes = cu_nodes, a->err = a->c.err;
  return KDA_OK;
}

kda_status mla_cache_weights(const void *q_cat, int H, const void *pool, int n_pages, int page_size,
                             const int32_t *page_table, int max_pages, const int32_t *lengths,
                             const int32_t *cu_nodes, int n_seqs, int64_t total_nodes, const int64_t *mask,
                             const float *node_weight, const float *lse, float scale, float *weights,
                             int64_t weights_stride, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_CACHE_WEIGHTS);
  kda::KeySumArgs a;
  kda_status st = key_sums(q_cat, H, pool, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                           total_nodes, scale, &a);
  if (st != KDA_OK || total_nodes == 0) return st;
  if (!optional(mask) || !optional(node_weight) || !given(lse) || !given(weights) || weights_stride < 1)
    return KDA_ERR_INVALID_ARG;
  if (!kda::mla_latent_supported()) return KDA_ERR_UNSUPPORTED;
  a.mask = mask, a.node_weight = node_weight, a.lse = lse;
  a.out = weights, a.out_stride = weights_stride;
  return done(kda::launch_cache_weights(a, stream), 1);
}

kda_status mla_weights_accept(float *weights, int64_t weights_stride, const int32_t *lengths, const int32_t *cu_nodes,
                              int n_seqs, int64_t total_nodes, const int32_t *parent, const int32_t *accept_node,
                              cudaStream_t stream) {
  KDA_TRACE(TR_MLA_WEIGHTS_ACCEPT);
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows) return KDA_ERR_INVALID_ARG;
  if (n_seqs == 0 || total_nodes == 0) return KDA_OK;
  if (!given(weights) || weights_stride < 1 || !given(lengths) || !given(cu_nodes) || !given(parent) || !given(accept_node))
    return KDA_ERR_INVALID_ARG;
  return done(kda::launch_weights_accept(weights, weights_stride, lengths, cu_nodes, n_seqs, total_nodes, parent, accept_node,
                                         kda::device_error(), stream), 1);
}

// What the selections share.
static kda_status check_choice(int most, int first, int recent) {
  return most < 1 || first < 0 || recent < 0 || first > most || recent > most - first ? KDA_ERR_INVALID_ARG : KDA_OK;
}

kda_status mla_cache_evict(void *pool, int n_layers, int n_pages, int page_size, const int32_t *page_table,
                           int max_pages, const int32_t *lengths, const int32_t *refcount, int n_seqs,
                           const float *weights, int64_t weights_stride, int budget, int first, int recent,
                           int32_t *kept, int32_t *new_lengths, float *new_weights, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_CACHE_EVICT);
  if (n_seqs < 0 || n_seqs > 65535) return KDA_ERR_INVALID_ARG;
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st == KDA_OK) st = check_choice(budget, first, recent);
  if (st != KDA_OK || n_seqs == 0) return st;
  if (!optional(refcount) || !given(weights) || weights_stride < 1 || !given(kept) || !given(new_lengths) ||
      !optional(new_weights))
    return KDA_ERR_INVALID_ARG;
  kda::SelectArgs a;
  std::memset(&a, 0, sizeof a);
  a.c = cache_args(pool, n_layers, n_pages, page_size, page_table, max_pages, lengths);
  a.n_seqs = n_seqs, a.values = weights, a.stride = weights_stride;
  a.most = budget, a.first = first, a.recent = recent;
  a.out = kept, a.out_stride = budget, a.out_lengths = new_lengths;
  a.refs = refcount, a.new_values = new_weights;
  int launches = 0;
  const cudaError_t e = kda::launch_cache_evict(a, &launches, stream);
  return done(e, launches);
}

kda_status mla_block_keys(const void *pool, int n_layers, int n_pages, int page_size, const int32_t *page_table,
                          int max_pages, const int32_t *from_lengths, const int32_t *lengths, int n_seqs, void *keys,
                          cudaStream_t stream) {
  KDA_TRACE(TR_MLA_BLOCK_KEYS);
  if (n_seqs < 0 || n_seqs > 65535) return KDA_ERR_INVALID_ARG;
  kda_status st = check_cache(pool, n_layers, n_pages, page_size, true, page_table, max_pages, lengths);
  if (st != KDA_OK || n_seqs == 0) return st;
  if (!given(from_lengths) || !given(keys)) return KDA_ERR_INVALID_ARG;
  return done(kda::launch_block_keys(cache_args(pool, n_layers, n_pages, page_size, page_table, max_pages, lengths),
                                     from_lengths, n_seqs, keys, stream), 1);
}

// every row's scores of the blocks, rows a multiple of 16 bytes long, and its (maximum, sum) over every 32
static int64_t score_stride(int max_pages) { return ((int64_t)max_pages + 3) & ~(int64_t)3; }
static int64_t part_stride(int max_pages) { return ((int64_t)max_pages + 31) / 32; }

size_t mla_block_scores_workspace_size(int64_t total_nodes, int H, int max_pages) {
  if (total_nodes < 1 || total_nodes > kMaxTreeRows || H < 1 || H > 128 || max_pages < 1 || max_pages > 1 << 20) return 0;
  return (size_t)total_nodes * H * (score_stride(max_pages) * sizeof(float) + part_stride(max_pages) * sizeof(float2));
}

// mla_block_scores but for the launches: the products (*a) and what makes scores of them (*s, which may
// hold a selection).
static kda_status block_scores(const void *q_cat, int H, const void *keys, int n_pages, int page_size,
                               const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *cu_nodes,
                               int n_seqs, int64_t total_nodes, float scale, float *scores, int64_t scores_stride,
                               void *workspace, size_t ws_bytes, kda::KeySumArgs *a, kda::SelectArgs *s) {
  kda_status st = key_sums(q_cat, H, keys, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                           total_nodes, scale, a);
  if (st != KDA_OK || total_nodes == 0) return st;
  if (!given(scores) || scores_stride < max_pages || !optional(workspace)) return KDA_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < mla_block_scores_workspace_size(total_nodes, H, max_pages)) return KDA_ERR_WORKSPACE;
  a->out = static_cast<float *>(workspace), a->out_stride = score_stride(max_pages);
  a->part = reinterpret_cast<float2 *>(a->out + total_nodes * H * a->out_stride), a->part_stride = part_stride(max_pages);
  s->c = a->c, s->n_seqs = n_seqs, s->cu_nodes = cu_nodes, s->total = total_nodes;
  s->values = s->scores = scores, s->stride = scores_stride;
  s->rows = a->out, s->rows_stride = a->out_stride, s->parts = a->part, s->parts_stride = a->part_stride, s->H = H;
  return KDA_OK;
}

kda_status mla_block_scores(const void *q_cat, int H, const void *keys, int n_pages, int page_size,
                            const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *cu_nodes,
                            int n_seqs, int64_t total_nodes, float scale, float *scores, int64_t scores_stride,
                            void *workspace, size_t ws_bytes, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_BLOCK_SCORES);
  kda::KeySumArgs a;
  kda::SelectArgs s;
  std::memset(&s, 0, sizeof s);
  kda_status st = block_scores(q_cat, H, keys, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                               total_nodes, scale, scores, scores_stride, workspace, ws_bytes, &a, &s);
  if (st != KDA_OK || total_nodes == 0) return st;
  if (!kda::mla_latent_supported()) return KDA_ERR_UNSUPPORTED;
  int launches = 0;
  cudaError_t e = kda::launch_block_products(a, stream);
  if (e == cudaSuccess) e = kda::launch_block_select(s, &launches, stream);
  return done(e, launches + 1);
}

// mla_block_select but for the launch; fills *a.
static kda_status block_select(const float *scores, int64_t scores_stride, int page_size, const int32_t *page_table,
                               int max_pages, const int32_t *lengths, const int32_t *cu_nodes, int n_seqs,
                               int64_t total_nodes, int blocks, int first, int recent, int32_t *sel_table, int sel_pages,
                               int32_t *sel_lengths, kda::SelectArgs *a) {
  if (n_seqs < 0 || n_seqs > 65535 || total_nodes < 0 || total_nodes > kMaxTreeRows || page_size < 1)
    return KDA_ERR_INVALID_ARG;
  if (!page_size_known(page_size)) return KDA_ERR_UNSUPPORTED;
  if (check_choice(blocks, first, recent) != KDA_OK) return KDA_ERR_INVALID_ARG;
  if (n_seqs == 0) return KDA_OK;
  if (!given(scores) || !given(page_table) || max_pages < 1 || max_pages > 1 << 20 || scores_stride < max_pages ||
      !given(lengths) || !given(cu_nodes) || !given(sel_table) || sel_pages < 1 || sel_pages > 1 << 20 || !given(sel_lengths))
    return KDA_ERR_INVALID_ARG;
  std::memset(a, 0, sizeof *a);
  a->c = cache_args(nullptr, 1, 1, page_size, page_table, max_pages, lengths);
  a->n_seqs = n_seqs, a->values = scores, a->stride = scores_stride;
  a->most = blocks, a->first = first, a->recent = recent;
  a->out = sel_table, a->out_stride = sel_pages, a->out_lengths = sel_lengths;
  a->cu_nodes = cu_nodes, a->total = total_nodes;
  return KDA_OK;
}

kda_status mla_block_select(const float *scores, int64_t scores_stride, int page_size, const int32_t *page_table,
                            int max_pages, const int32_t *lengths, const int32_t *cu_nodes, int n_seqs,
                            int64_t total_nodes, int blocks, int first, int recent, int32_t *sel_table, int sel_pages,
                            int32_t *sel_lengths, cudaStream_t stream) {
  KDA_TRACE(TR_MLA_BLOCK_SELECT);
  kda::SelectArgs a;
  kda_status st = block_select(scores, scores_stride, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                               total_nodes, blocks, first, recent, sel_table, sel_pages, sel_lengths, &a);
  if (st != KDA_OK || n_seqs == 0) return st;
  int launches = 0;
  const cudaError_t e = kda::launch_block_select(a, &launches, stream);
  return done(e, launches);
}

size_t mla_sparse_workspace_size(int n_seqs, int64_t total_nodes, int H, int max_pages) {
  const size_t scores = mla_block_scores_workspace_size(total_nodes, H, max_pages);
  const size_t tree = mla_tree_workspace_size(n_seqs, total_nodes, H);
  return scores == 0 || tree == 0 ? 0 : scores > tree ? scores : tree;
}

// The three parts of a sparse step; they follow one another, so they share the workspace.
struct SparseStep {
  kda::KeySumArgs scores;
  kda::SelectArgs choice;
  kda::TreeAttnArgs attention;
};
static kda_status sparse_step(const void *q_cat, int H, const void *pool, const void *keys, int n_pages, int page_size,
                              const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *cu_nodes,
                              int n_seqs, int64_t total_nodes, const int64_t *mask, float scale, int blocks, int first,
                              int recent, float *scores, int64_t scores_stride, int32_t *sel_table, int sel_pages,
                              int32_t *sel_lengths, void *z, kda_dtype z_dtype, void *workspace, size_t ws_bytes,
                              SparseStep *s) {
  std::memset(&s->choice, 0, sizeof s->choice);
  if (check_choice(blocks, first, recent) != KDA_OK) return KDA_ERR_INVALID_ARG;  // without nodes too
  kda_status st = KDA_OK;
  if (total_nodes != 0)
    st = block_select(scores, scores_stride, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs, total_nodes, blocks, first,
                      recent, sel_table, sel_pages, sel_lengths, &s->choice);
  if (st != KDA_OK) return st;
  st = block_scores(q_cat, H, keys, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs, total_nodes, scale,
                    scores, scores_stride, workspace, ws_bytes, &s->scores, &s->choice);
  if (st != KDA_OK || total_nodes == 0) return st;
  return tree_attention(q_cat, H, pool, n_pages, page_size, sel_table, sel_pages, sel_lengths, cu_nodes, n_seqs,
                        total_nodes, mask, scale, z, z_dtype, workspace, ws_bytes, &s->attention);
}
static cudaError_t launch_sparse(const SparseStep &s, int *launches, cudaStream_t stream) {
  cudaError_t e = kda::launch_block_products(s.scores, stream);
  int more = 0;
  if (e == cudaSuccess) e = kda::launch_block_select(s.choice, &more, stream);
  if (e == cudaSuccess) e = kda::launch_mla_tree(s.attention, launches, stream);
  *launches += more + 1;
  return e;
}

kda_status mla_sparse_latent(const void *q_cat, int H, const void *pool, const void *keys, int n_pages, int page_size,
                             const int32_t *page_table, int max_pages, const int32_t *lengths, const int32_t *cu_nodes,
                             int n_seqs, int64_t total_nodes, const int64_t *mask, float scale, int blocks, int first,
                             int recent, float *scores, int64_t scores_stride, int32_t *sel_table, int sel_pages,
                             int32_t *sel_lengths, void *z, kda_dtype z_dtype, void *workspace, size_t ws_bytes,
                             cudaStream_t stream) {
  KDA_TRACE(TR_MLA_SPARSE_LATENT);
  SparseStep s;
  kda_status st = sparse_step(q_cat, H, pool, keys, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                              total_nodes, mask, scale, blocks, first, recent, scores, scores_stride, sel_table, sel_pages,
                              sel_lengths, z, z_dtype, workspace, ws_bytes, &s);
  if (st != KDA_OK || total_nodes == 0) return st;
  int launches = 0;
  const cudaError_t e = launch_sparse(s, &launches, stream);
  return done(e, launches);
}

kda_status mla_sparse_decode(const void *q_nope, const void *q_rope, const void *w_uk, const void *w_uv, const void *pool,
                             const void *keys, int n_pages, int page_size, const int32_t *page_table, int max_pages,
                             const int32_t *lengths, const int32_t *cu_nodes, int n_seqs, int64_t total_nodes,
                             const int64_t *mask, const void *gate_logit, float scale, int blocks, int first, int recent,
                             float *scores, int64_t scores_stride, int32_t *sel_table, int sel_pages,
                             int32_t *sel_lengths, void *q_cat, float *z, void *out, void *workspace, size_t ws_bytes,
                             cudaStream_t stream) {
  KDA_TRACE(TR_MLA_SPARSE_DECODE);
  SparseStep s;
  kda::MlaArgs m;
  kda_status st = node_projections(q_nope, q_rope, w_uk, w_uv, gate_logit, out, q_cat, z, total_nodes, &m);
  if (total_nodes > 0 && st != KDA_OK) return st;
  st = sparse_step(q_cat, 64, pool, keys, n_pages, page_size, page_table, max_pages, lengths, cu_nodes, n_seqs,
                   total_nodes, mask, scale, blocks, first, recent, scores, scores_stride, sel_table, sel_pages,
                   sel_lengths, z, KDA_F32, workspace, ws_bytes, &s);
  if (st != KDA_OK || total_nodes == 0) return st;
  int launches = 0;
  cudaError_t e = kda::launch_mla_absorb(m, stream);
  if (e == cudaSuccess) e = launch_sparse(s, &launches, stream);
  if (e == cudaSuccess) e = kda::launch_mla_up_gate(m, stream);
  return done(e, launches + 2);
}

}  // extern "C"
