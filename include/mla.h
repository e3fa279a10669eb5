/*
 * mla.h -- C ABI of the absorbed gated-MLA decode (the hybrid's other token mixer) in the
 * same GB300 (sm_103a) library as kda.h; conventions as kda.h (device pointers, caller-owned
 * buffers, asynchronous on the stream, host validation with status codes, 16-byte alignment,
 * device-side index checks reported by kda_check_device_error).
 *
 * What it computes ("Ling-3.1-flash: Grouped Routing and Two Different MLA Caches",
 * sections "MLA's expanded reference path" and "Why weight absorption keeps the same
 * attention function"): each cached position t of a sequence keeps the normalised latent
 * c_t (512) and the rotated positional key r_t (64) shared by the 64 heads.  For the query
 * token, head i has non-positional part q_i^N (128) and rotated positional part q_i^R (64);
 * the key and value up-projections W_K,i, W_V,i are 128 x 512.  Absorbed execution:
 *     q~_i = W_K,i^T q_i^N                             (512)
 *     s_t  = scale * ([q~_i ; q_i^R] . [c_t ; r_t])      over t < length
 *     z_i  = sum_t softmax_t(s)_t c_t                  (512: the latent is the value)
 *     o_i  = W_V,i z_i * sigmoid(gate_i)               (128; one gate logit per head)
 * the same attention function as expanding every cached position into 64 heads of 192-wide
 * keys and 128-wide values (scale 1/sqrt(192) in the pages' configuration).
 * The shapes are the pages': 64 heads, latent 512, positional key 64, 128-wide q^N and o.
 */
#ifndef MLA_H_
#define MLA_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device workspace that lets mla_decode_latent / mla_decode split each sequence's cached
 * positions across several CTAs (so a small batch still fills the GPU): partial sums of each
 * split, merged by a second launch.  0 when no split pays (then no workspace is needed).
 * With less than this, the calls use as many splits as fit (down to none). */
size_t mla_decode_workspace_size(int n_seqs, int64_t cache_len);

/* Tuning and testing only: forces the split count of every later mla_decode_latent /
 * mla_decode_latent_noalloc / mla_decode call and of mla_decode_workspace_size in this
 * process (1..64; 0 restores the automatic rule: as many splits as fill the SMs in one wave,
 * each at least 512 positions).  Process-wide, not per device or stream; set it only while
 * no MLA call is being issued.  KDA_ERR_INVALID_ARG outside 0..64. */
kda_status mla_set_split_override(int n_split);

/*
 * mla_decode_latent -- the attention over the latent cache (the part that streams it).
 *
 *   q_cat      [n_seqs, 64, 576] bf16: [q~_i ; q_i^R] per head.
 *   cache      [n_seqs, cache_len, 576] bf16: row t of sequence n = [c_t ; r_t]; rows at or
 *              past lengths[n] are ignored (their contents may be anything).
 *   lengths    [n_seqs] int32 (device), 0..cache_len; a length outside that range is
 *              treated as 0 and reported (KDA_ERR_BAD_INDEX).  Length 0 gives z = 0.
 *   scale      score scale (> 0).
 *   z          [n_seqs, 64, 512] fp32 output.
 *   workspace / ws_bytes: caller-owned, up to mla_decode_workspace_size() bytes, or NULL / 0
 *              (one CTA per sequence).  Splits write each head's unnormalised sum with its
 *              running maximum and normaliser; the merge rescales them to a common maximum.
 * Scores and the weighted sum run on the tensor cores with bf16 operands and fp32
 * accumulation (the weights are rounded to bf16 as operands; the normaliser sums the same
 * rounded weights).
 */
kda_status mla_decode_latent(const void* q_cat, const void* cache, int64_t cache_len,
                             const int32_t* lengths, int n_seqs, float scale, float* z,
                             void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mla_decode_latent_noalloc -- mla_decode_latent with no caller workspace and no allocation.
 * No counterpart on the pages (they describe the attention, not how its scratch memory is
 * provided): the split partial sums go to a fixed 24 MiB device buffer inside the library
 * (each device its own copy), so the call needs no memory from the caller.  The split count
 * is the one mla_decode_workspace_size() sizes; if that needs more than the fixed buffer, the
 * call returns KDA_ERR_WORKSPACE and launches nothing.  Calls on one device share the buffer:
 * issue them in one stream (or otherwise ordered), never concurrently.  Arguments, layouts
 * and results as mla_decode_latent; bit-identical to it with a workspace of that size.
 */
kda_status mla_decode_latent_noalloc(const void* q_cat, const void* cache, int64_t cache_len,
                                     const int32_t* lengths, int n_seqs, float scale, float* z,
                                     cudaStream_t stream);

/*
 * mla_decode -- one absorbed gated-MLA decode step: absorption, mla_decode_latent, value
 * up-projection and gate.
 *
 *   q_nope     [n_seqs, 64, 128] bf16;  q_rope [n_seqs, 64, 64] bf16 (already rotated).
 *   w_uk, w_uv [64, 128, 512] bf16: W_K,i and W_V,i of each head.
 *   gate_logit [n_seqs, 64] bf16: one logit per head.
 *   q_cat      [n_seqs, 64, 576] bf16 and z [n_seqs, 64, 512] fp32: caller-owned
 *              intermediates (the absorbed query, the latent attention output).
 *   out        [n_seqs, 64, 128] bf16: o_i of every head.
 *   cache, cache_len, lengths, scale, workspace, ws_bytes as mla_decode_latent.
 */
kda_status mla_decode(const void* q_nope, const void* q_rope, const void* w_uk,
                      const void* w_uv, const void* cache, int64_t cache_len,
                      const int32_t* lengths, int n_seqs, const void* gate_logit, float scale,
                      void* q_cat, float* z, void* out, void* workspace, size_t ws_bytes,
                      cudaStream_t stream);

/* ---- the paged latent cache ---------------------------------------------------------------
 *
 * pool        [n_layers, n_pages, page_size, 576] bf16: every latent layer's pages (the calls of
 *             one layer take that layer's [n_pages, page_size, 576] part).  page_size 16, 32, 64,
 *             128 or 256 (KDA_ERR_UNSUPPORTED otherwise); n_pages at most 2^26.
 * page_table  [n_slots, max_pages] int32 (device): the pages of a sequence in order; position t
 *             is row t % page_size of page page_table[n][t / page_size], in every layer.
 *             max_pages at most 2^20.
 * lengths     [n_slots] int32 (device): cached positions of each sequence; rows past it may hold
 *             anything, and the table past the pages in use is not read.
 * refcount    [n_pages] int32: table rows that name the page; 0 marks a free page.
 * held        [n_slots] int32: pages that a sequence's table row holds.
 * Sequences that share a prefix share its full pages; a write never goes to a shared page as long
 * as the pages come from mla_pages_reserve and mla_pages_fork.  Free pages are taken in ascending
 * order, so the same calls always give the same tables.  A sequence that is cut back into a page it
 * shares must not be appended to (fork it first: the child's last page is a copy).  Calls that write
 * the same tables run one after another (one stream, or events between them), each with a workspace
 * that no other call in flight uses.  No counterpart interface is printed on the pages.
 */

/*
 * mla_cache_append -- writes new rows (drafted tokens, or a prompt's) behind each sequence:
 * row cu_rows[n] + t of `rows` goes to position lengths[n] + t of sequence n, in every layer.
 *   rows        [n_layers, total_rows, 576] bf16;  cu_rows [n_seqs + 1] int32 (device).
 * Lengths are not changed.  Bit-exact copies.  Sequences whose offsets fall outside [0, total_rows] or
 * run backwards are skipped and reported (KDA_ERR_BAD_SEQLENS; a row that other sequences around them
 * share goes to one of these); a position without a page is skipped and reported (KDA_ERR_BAD_INDEX).
 * Rows of no sequence are not read into the pool.
 */
kda_status mla_cache_append(void* pool, int n_layers, int n_pages, int page_size,
                            const int32_t* page_table, int max_pages, const int32_t* lengths,
                            const int32_t* cu_rows, int n_seqs, int64_t total_rows,
                            const void* rows, cudaStream_t stream);

/*
 * mla_cache_accept -- compacts the accepted path of each verified tree: with the drafted rows at
 * positions lengths[n] + node, the row of the path's step d (0 = root) moves to lengths[n] + d in
 * every layer, and new_lengths[n] = lengths[n] + steps on the path.
 *   cu_nodes, parent, accept_node as kda_tree_accept (-1 accepts nothing);  new_lengths [n_seqs]
 *   int32 output, may be `lengths`.
 * Bit-exact moves.  A sequence with bad offsets, more than 64 nodes, an accept_node outside -1 ..
 * nodes - 1, or a path on which a node's position or the one that it moves to has no page keeps its rows
 * and length and is reported.
 */
kda_status mla_cache_accept(void* pool, int n_layers, int n_pages, int page_size,
                            const int32_t* page_table, int max_pages, const int32_t* lengths,
                            const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                            const int32_t* parent, const int32_t* accept_node,
                            int32_t* new_lengths, cudaStream_t stream);

/*
 * mla_pages_copy -- copies page src[i] to page dst[i] in every layer, i < n_copies (at most
 * 8192; device int32 arrays).  An entry out of range, one whose target an earlier entry has, or
 * one whose target is the source of another is skipped and reported (KDA_ERR_BAD_INDEX); a page named
 * as its own target stays as it is.
 */
kda_status mla_pages_copy(void* pool, int n_layers, int n_pages, int page_size,
                          const int32_t* src, const int32_t* dst, int n_copies,
                          cudaStream_t stream);

/* Device workspace of mla_pages_fork and mla_pages_reserve for n entries (1..65535; else 0). */
size_t mla_pages_workspace_size(int n);

/*
 * mla_pages_free -- releases every page of the sequences slots[0..n-1] (device int32): their
 * refcounts drop by one, their table entries become -1, held and lengths 0.  A sequence listed
 * twice is released once.  Indices out of range, table entries that name no page and counts that
 * are already 0 are skipped and reported (KDA_ERR_BAD_INDEX).
 */
kda_status mla_pages_free(int n_pages, int32_t* refcount, int32_t* page_table, int max_pages,
                          int32_t* held, int32_t* lengths, int n_slots, const int32_t* slots,
                          int n, cudaStream_t stream);

/*
 * mla_pages_fork -- sequence dst[i] becomes a copy of sequence src[i] (i < n): it names the same
 * full pages, and the rows of a partly filled last page are copied, in every layer, to the lowest
 * free page (entries take pages in order).
 * A child must hold no pages (mla_pages_free releases them) and may not be a parent of the same
 * call; one parent may have many children.  An entry that breaks this, is out of range, or whose
 * child an earlier entry has is skipped and reported (KDA_ERR_BAD_INDEX); where pages run out the
 * child stays empty and KDA_ERR_NO_PAGES is reported.
 *   workspace / ws_bytes: at least mla_pages_workspace_size(n) bytes, 16-byte aligned
 *   (KDA_ERR_WORKSPACE otherwise).
 */
kda_status mla_pages_fork(void* pool, int n_layers, int n_pages, int page_size,
                          int32_t* refcount, int32_t* page_table, int max_pages, int32_t* held,
                          int32_t* lengths, int n_slots, const int32_t* src, const int32_t* dst,
                          int n, void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mla_pages_reserve -- gives the sequences slots[i] the pages they lack for lengths + extra[i]
 * positions (i < n; device int32 arrays), lowest free pages first, entries in order.  The first
 * entry for which not all pages are left, and every later one that needs any, gets none and
 * KDA_ERR_NO_PAGES is reported; held[] tells which got theirs.  An entry out of range, longer than
 * the table row, or naming a sequence of an earlier entry is skipped and reported
 * (KDA_ERR_BAD_INDEX).  Workspace as mla_pages_fork.
 */
kda_status mla_pages_reserve(int n_pages, int page_size, int32_t* refcount, int32_t* page_table,
                             int max_pages, int32_t* held, const int32_t* lengths, int n_slots,
                             const int32_t* slots, const int32_t* extra, int n, void* workspace,
                             size_t ws_bytes, cudaStream_t stream);

/* ---- attention of drafted trees ------------------------------------------------------------ */

/*
 * mla_tree_mask -- the visibility words of trees given by parents: bit j of mask[row] is set iff
 * node j of the row's sequence is the row's node or one of its ancestors.  cu_nodes and parent as
 * kda_tree_verify (at most 64 nodes a sequence; bad offsets and parents are reported as there).
 * One call serves every latent layer of a step.
 */
kda_status mla_tree_mask(const int32_t* parent, const int32_t* cu_nodes, int n_seqs,
                         int64_t total_nodes, int64_t* mask, cudaStream_t stream);

/* Device workspace of mla_tree_latent and mla_tree_decode, and of those with lse (H heads; 64 for
 * mla_tree_decode); 0 for invalid arguments. */
size_t mla_tree_workspace_size(int n_seqs, int64_t total_nodes, int H);

/*
 * mla_tree_latent -- mla_decode_latent for a tree of drafted tokens of each sequence over the
 * paged cache; with one node a sequence it is the one-token decode step over pages.
 *
 *   q_cat       [total_nodes, H, 576] bf16, H in 1..128 (a head shard's queries; the latent cache
 *               is shared by all heads).
 *   pool        [n_pages, page_size, 576] bf16, page_table, max_pages, lengths: the layer's paged
 *               cache; the drafted nodes' rows are already at positions lengths[n] + node
 *               (mla_cache_append).
 *   cu_nodes    [n_seqs + 1] int32 (device): nodes of sequence n are rows cu_nodes[n] ..
 *               cu_nodes[n+1]-1, at most 64.  Offsets outside [0, total_nodes], running backwards
 *               or holding more are skipped (their z rows stay as they were) and reported
 *               (KDA_ERR_BAD_SEQLENS).
 *   mask        [total_nodes] int64 (device): node i attends to the drafted node j of its sequence
 *               where bit j is set (any pattern; bits past the last node are ignored), and to
 *               every cached position.  NULL: a chain (node i attends to nodes 0..i).
 *   scale       score scale (> 0).
 *   z           [total_nodes, H, 512] output, fp32 or bf16 (z_dtype).  A node that sees no
 *               position gets z = 0.
 *   workspace / ws_bytes: at least mla_tree_workspace_size() bytes, 16-byte aligned
 *               (KDA_ERR_WORKSPACE otherwise); calls that may run at the same time need their own.
 * A length below 0, or more positions than the table row holds, counts as an empty sequence without
 * visible positions; positions whose page is out of range are invisible; both are reported
 * (KDA_ERR_BAD_INDEX).  Scores and the weighted sum run with bf16 operands and fp32 accumulation
 * (weights rounded to bf16, the normaliser sums the rounded weights).  Rows past the drafted
 * nodes may hold anything; a drafted row that holds NaN or infinities reaches only the nodes
 * that see it.
 */
kda_status mla_tree_latent(const void* q_cat, int H, const void* pool, int n_pages, int page_size,
                           const int32_t* page_table, int max_pages, const int32_t* lengths,
                           const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                           const int64_t* mask, float scale, void* z, kda_dtype z_dtype,
                           void* workspace, size_t ws_bytes, cudaStream_t stream);

/*
 * mla_tree_decode -- mla_decode for drafted trees over the paged cache: absorption,
 * mla_tree_latent with fp32 z, value up-projection and gate, one query row per node.
 *   q_nope [total_nodes, 64, 128], q_rope [total_nodes, 64, 64], gate_logit [total_nodes, 64],
 *   q_cat [total_nodes, 64, 576], z [total_nodes, 64, 512] fp32 and out [total_nodes, 64, 128]
 *   as mla_decode's with total_nodes for n_seqs; the rest as mla_tree_latent with H = 64.  Rows of
 *   no sequence keep their z, and their out is computed from it.
 */
kda_status mla_tree_decode(const void* q_nope, const void* q_rope, const void* w_uk,
                           const void* w_uv, const void* pool, int n_pages, int page_size,
                           const int32_t* page_table, int max_pages, const int32_t* lengths,
                           const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                           const int64_t* mask, const void* gate_logit, float scale, void* q_cat,
                           float* z, void* out, void* workspace, size_t ws_bytes,
                           cudaStream_t stream);

/* ---- long contexts: eviction by accumulated attention ----------------------------------------
 *
 * A sequence's positions are ranked by the attention that they received: mla_tree_latent_lse (or
 * mla_tree_decode_lse) leaves each row's log-sum, mla_cache_weights adds what each position got to a
 * running sum (in every latent layer that counts), mla_cache_evict keeps the heaviest positions of a
 * sequence and moves their rows together in every layer, mla_pages_trim releases the pages behind
 * them.  The rows' positional keys are as they were cached, so later queries are rotated by the
 * token's own position, which is no longer the sequence's length.
 */

/*
 * mla_tree_latent_lse, mla_tree_decode_lse -- mla_tree_latent and mla_tree_decode that also write
 *   lse         [total_nodes, H] fp32: ln sum_t exp(s_t) over what the row sees, -infinity for a row
 *               that sees nothing.  Summed in fp32 from the weights before they are rounded.
 * All else as there; z and out are bit-identical to theirs.
 */
kda_status mla_tree_latent_lse(const void* q_cat, int H, const void* pool, int n_pages, int page_size,
                               const int32_t* page_table, int max_pages, const int32_t* lengths,
                               const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                               const int64_t* mask, float scale, void* z, kda_dtype z_dtype,
                               float* lse, void* workspace, size_t ws_bytes, cudaStream_t stream);
kda_status mla_tree_decode_lse(const void* q_nope, const void* q_rope, const void* w_uk,
                               const void* w_uv, const void* pool, int n_pages, int page_size,
                               const int32_t* page_table, int max_pages, const int32_t* lengths,
                               const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                               const int64_t* mask, const void* gate_logit, float scale, void* q_cat,
                               float* z, void* out, float* lse, void* workspace, size_t ws_bytes,
                               cudaStream_t stream);

/*
 * mla_cache_weights -- weights[n][t] += sum_i u_i sum_h exp(s_iht - lse_ih) over the nodes i of
 * sequence n that see position t (as mla_tree_latent: every cached position, and the drafted row of
 * node j at position lengths[n] + j where bit j of mask[i] is set; NULL: a chain).
 *   q_cat, H, pool .. lengths, cu_nodes, n_seqs, total_nodes, mask, scale as mla_tree_latent.
 *   node_weight [total_nodes] fp32 u_i, or NULL (ones).  A node of weight 0 (a rejected draft)
 *               adds nothing, whatever its row holds.
 *   lse         [total_nodes, H] fp32 from mla_tree_latent_lse on the same arguments; a row whose lse is
 *               -infinity adds nothing.
 *   weights     [n_seqs, weights_stride] fp32, added to: positions 0 .. lengths[n] + nodes - 1; others
 *               keep their values.
 * Products with bf16 operands and fp32 accumulation; the sum over rows is in fp32 in a fixed order.
 * Sequences with bad offsets or lengths (also more positions than weights_stride) are skipped and
 * reported as there; a position whose page is out of range gets nothing and is reported.
 */
kda_status mla_cache_weights(const void* q_cat, int H, const void* pool, int n_pages, int page_size,
                             const int32_t* page_table, int max_pages, const int32_t* lengths,
                             const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                             const int64_t* mask, const float* node_weight, const float* lse,
                             float scale, float* weights, int64_t weights_stride,
                             cudaStream_t stream);

/*
 * mla_weights_accept -- what mla_cache_accept does to the rows, for the weights of drafted trees: the
 * weight of the accepted path's step d (0 = root), at position lengths[n] + its node, moves to
 * lengths[n] + d; those of the other drafted positions become 0.  Called with the lengths before the
 * acceptance.  (A chain of which a prefix is accepted needs no such call.)
 *   weights, weights_stride, lengths as mla_cache_weights;  cu_nodes, parent, accept_node as
 *   mla_cache_accept.
 * A sequence with bad offsets or more than 64 nodes (KDA_ERR_BAD_SEQLENS), an accept_node outside
 * -1 .. nodes - 1, or a length below 0 or with which the nodes pass weights_stride (KDA_ERR_BAD_INDEX) keeps
 * its weights and is reported; a bad parent is reported and counts as none.  Pages are not looked at: of a
 * path that mla_cache_accept refuses for a page that is not there the weights move all the same.
 */
kda_status mla_weights_accept(float* weights, int64_t weights_stride, const int32_t* lengths,
                              const int32_t* cu_nodes, int n_seqs, int64_t total_nodes,
                              const int32_t* parent, const int32_t* accept_node,
                              cudaStream_t stream);

/*
 * mla_cache_evict -- cuts each sequence of more than `budget` positions to `budget`: it keeps its
 * first `first` and its last `recent` positions and, of those between, the ones of the largest
 * weights (among equals the lower position first; NaN counts as less than anything).  The kept rows
 * move to positions 0 .. budget - 1 in their order, in every layer; shorter sequences stay as they are.
 *   weights     [n_seqs, weights_stride] fp32.
 *   budget      at least 1;  first, recent: at least 0, first + recent <= budget.
 *   refcount    [n_pages] int32 or NULL: where given, a sequence whose kept rows would move into a page
 *               that other sequences share is refused; without it the caller answers for that.
 *   kept        [n_seqs, budget] int32 output: the kept positions in ascending order, then -1.
 *   new_lengths [n_seqs] int32 output, may be `lengths`.
 *   new_weights NULL, or [n_seqs, weights_stride] fp32: the kept positions' weights, then zeros up to
 *               the old length, what is behind left as it was; may be `weights`, must not overlap it
 *               otherwise.
 * Bit-exact moves; pages stay held (mla_pages_trim).  There are no drafted rows at the time of the
 * call.  A sequence with a bad length (below 0, more than the table row or weights_stride hold), a
 * row that would move from or to a position without a page, or into a shared page keeps its rows, length
 * and weights, has a `kept` row of -1 and is reported (KDA_ERR_BAD_INDEX); other pages may be missing or
 * shared.  A new_weights of its own gets such a sequence's weights up to its length, the whole row where that is
 * bad.  Keys of pages that the rows moved into are written anew by mla_block_keys.
 */
kda_status mla_cache_evict(void* pool, int n_layers, int n_pages, int page_size,
                           const int32_t* page_table, int max_pages, const int32_t* lengths,
                           const int32_t* refcount, int n_seqs, const float* weights,
                           int64_t weights_stride, int budget, int first, int recent,
                           int32_t* kept, int32_t* new_lengths, float* new_weights,
                           cudaStream_t stream);

/*
 * mla_pages_trim -- releases the pages of the sequences slots[0..n-1] that lie wholly behind their
 * lengths: refcounts drop by one, table entries become -1, held the pages that are left.  A
 * sequence listed twice is cut once.  Indices out of range, bad lengths, sequences that hold fewer pages
 * than their length needs, table entries that name no page and counts that are already 0 are skipped
 * and reported (KDA_ERR_BAD_INDEX).
 */
kda_status mla_pages_trim(int n_pages, int page_size, int32_t* refcount, int32_t* page_table,
                          int max_pages, int32_t* held, const int32_t* lengths, int n_slots,
                          const int32_t* slots, int n, cudaStream_t stream);

/* ---- long contexts: attention over chosen blocks ------------------------------------------------
 *
 * A block is a page.  Every full page has a key, the mean of its rows; a step scores a sequence's
 * full pages by their keys, keeps the best, and attends to those and to what is behind the last full
 * page.  The choice is the sequence's: all its heads and drafted nodes read the same pages.  Keys go by
 * page, so sequences that share pages share their keys, and a fork needs none of its own.
 */

/*
 * mla_block_keys -- keys[layer][page] = mean of the page's rows (fp32 sum, rounded once), for the
 * pages that filled up: sequence n's pages from_lengths[n] / page_size .. lengths[n] / page_size - 1, in
 * every layer.  After mla_cache_append or mla_cache_accept with the lengths before and after.
 *   keys        [n_layers, n_pages, 576] bf16;  from_lengths [n_seqs] int32 (from 0: all).
 * Sequences with a bad length and pages out of range are skipped and reported (KDA_ERR_BAD_INDEX);
 * from_lengths[n] >= lengths[n] is no work.
 */
kda_status mla_block_keys(const void* pool, int n_layers, int n_pages, int page_size,
                          const int32_t* page_table, int max_pages, const int32_t* from_lengths,
                          const int32_t* lengths, int n_seqs, void* keys, cudaStream_t stream);

/* Device workspace of mla_block_scores; 0 for invalid arguments. */
size_t mla_block_scores_workspace_size(int64_t total_nodes, int H, int max_pages);

/*
 * mla_block_scores -- scores[n][b] = sum over the rows r (nodes x heads) of sequence n's step of
 * softmax_b(scale q_r . key_b), b over its full pages (b < lengths[n] / page_size).
 *   q_cat, H, page_table .. lengths, cu_nodes, n_seqs, total_nodes, scale as mla_tree_latent.
 *   keys        [n_pages, 576] bf16, the layer's.
 *   scores      [n_seqs, scores_stride] fp32 (scores_stride >= max_pages); entries behind the full
 *               pages keep their values.
 *   workspace / ws_bytes: at least mla_block_scores_workspace_size() bytes, 16-byte aligned.
 * Sequences without nodes or with bad offsets or lengths are skipped (and reported as there); a block
 * whose page is out of range scores 0 and is reported.
 */
kda_status mla_block_scores(const void* q_cat, int H, const void* keys, int n_pages, int page_size,
                            const int32_t* page_table, int max_pages, const int32_t* lengths,
                            const int32_t* cu_nodes, int n_seqs, int64_t total_nodes, float scale,
                            float* scores, int64_t scores_stride, void* workspace, size_t ws_bytes,
                            cudaStream_t stream);

/*
 * mla_block_select -- the page table of what a step reads: of each sequence's full pages the first
 * `first`, the last `recent` and those of the largest scores, `blocks` in all (among equals the earlier
 * page; NaN counts as less than anything; all of them where there are no more), in their order; then the
 * page in use and those of the drafted rows.
 *   sel_table   [n_seqs, sel_pages] int32 output, -1 behind the last page;  sel_lengths [n_seqs] int32
 *               output: the cached positions among them.  Both are what mla_tree_latent and
 *               mla_tree_decode take as page_table and lengths.
 *   blocks      at least 1;  first, recent: at least 0, first + recent <= blocks.
 * A sequence without nodes gets an empty row; so does one with bad offsets or lengths or that needs more
 * than sel_pages entries, which is reported.
 */
kda_status mla_block_select(const float* scores, int64_t scores_stride, int page_size,
                            const int32_t* page_table, int max_pages, const int32_t* lengths,
                            const int32_t* cu_nodes, int n_seqs, int64_t total_nodes, int blocks,
                            int first, int recent, int32_t* sel_table, int sel_pages,
                            int32_t* sel_lengths, cudaStream_t stream);

/* Device workspace of mla_sparse_latent and mla_sparse_decode (H = 64); 0 for invalid arguments. */
size_t mla_sparse_workspace_size(int n_seqs, int64_t total_nodes, int H, int max_pages);

/*
 * mla_sparse_latent -- mla_block_scores, mla_block_select and mla_tree_latent over the selection in
 * one call.  keys is the layer's [n_pages, 576]; scores, sel_table and sel_lengths are caller-owned and
 * hold what those calls write; workspace: at least mla_sparse_workspace_size() bytes.  A call without nodes
 * (total_nodes = 0) launches nothing: z, scores, sel_table and sel_lengths stay as they were
 * (mla_block_select, on its own, then writes empty rows).
 */
kda_status mla_sparse_latent(const void* q_cat, int H, const void* pool, const void* keys,
                             int n_pages, int page_size, const int32_t* page_table, int max_pages,
                             const int32_t* lengths, const int32_t* cu_nodes, int n_seqs,
                             int64_t total_nodes, const int64_t* mask, float scale, int blocks,
                             int first, int recent, float* scores, int64_t scores_stride,
                             int32_t* sel_table, int sel_pages, int32_t* sel_lengths, void* z,
                             kda_dtype z_dtype, void* workspace, size_t ws_bytes,
                             cudaStream_t stream);

/*
 * mla_sparse_decode -- mla_tree_decode with mla_sparse_latent (H = 64, fp32 z) for mla_tree_latent.
 */
kda_status mla_sparse_decode(const void* q_nope, const void* q_rope, const void* w_uk,
                             const void* w_uv, const void* pool, const void* keys, int n_pages,
                             int page_size, const int32_t* page_table, int max_pages,
                             const int32_t* lengths, const int32_t* cu_nodes, int n_seqs,
                             int64_t total_nodes, const int64_t* mask, const void* gate_logit,
                             float scale, int blocks, int first, int recent, float* scores,
                             int64_t scores_stride, int32_t* sel_table, int sel_pages,
                             int32_t* sel_lengths, void* q_cat, float* z, void* out,
                             void* workspace, size_t ws_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif  /* MLA_H_ */
