// mla_pages.cu -- the paged latent cache of the absorbed gated-MLA decode: rows written and
// compacted, pages reserved, shared, copied and released.
//
// Each cached position of a sequence is one 576-wide bf16 row ("Ling-3.1-flash: Grouped Routing
// and Two Different MLA Caches", section "MLA's expanded reference path": latent 512 and
// positional key 64), 1,152 bytes, in every latent layer.  A pool holds pages of page_size rows;
// a sequence's table row names its pages in order, the same pages in every layer, and refs
// counts the table rows that name a page (0: free).  Sequences that share a prefix share its
// full pages ("Ling-3.1-flash: What 63 Linear-Attention Layers Do to the KV Budget", section
// "Where the hybrid makes serving harder", on prefix reuse); a partly filled one is copied.
//
// The copies are bound by memory: every kernel moves 16 bytes a thread and access, with all of a
// thread's loads issued before its first store (64 sequences forked to 256 children, freed, and given
// room, nine layers of up to 63 rows each: 35 us, of which the copies of 154 MB are 18).  The
// bookkeeping is bound by latency: one CTA keeps each call to one or two launches, each overlapping
// the one before (the same 46 us without that), and free pages are found by a scan of the counts in
// page order (so the lowest free page is always taken next, whatever was freed when; it grows with the pool:
// reserve and free for 256 sequences take 16 us in 20,000 pages of which the first 18,000 are held, 39 in
// 300,000 of which 270,000 are).  Drafted rows written and compacted, 256 sequences x 8 x 9 layers: 12 us on
// the device for both calls; prompts of 65,536 rows x 9 layers written at the copy rate (200 us).
#include "kda_common.cuh"
#include "kda_internal.h"

#include <climits>

namespace kda {
namespace {

constexpr int ROW16 = 576 * 2 / 16;  // 16-byte pieces of a row

__device__ __forceinline__ uint4 *pool_row(const PagedCache &c, int layer, int page, int row) {
  return reinterpret_cast<uint4 *>(c.pool) +
         (((size_t)layer * c.n_pages + page) * c.page_size + row) * ROW16;
}
// The page of a sequence's position, or -1 (outside the table, or no page there).
__device__ __forceinline__ int page_of(const PagedCache &c, int n, int64_t pos) {
  const int64_t j = pos / c.page_size;
  if (pos < 0 || j >= c.max_pages) return -1;
  const int p = c.table[(size_t)n * c.max_pages + j];
  return p >= 0 && p < c.n_pages ? p : -1;
}
__device__ __forceinline__ void flag(int *err, int bit) {
  if (err) atomicOr(err, bit);
}
// These calls follow one another in a step and are short, so each kernel is launched while the one
// before it runs, and waits here until that one is complete.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

// ---- rows ------------------------------------------------------------------------------------

// Row t of sequence n's new rows goes to position lengths[n] + t.  A CTA takes four rows: 72 threads
// read a row's 72 pieces of up to nine layers while a warp looks up where the row goes (32 sequences'
// offsets at a step), then write them.  A sequence whose offsets are bad must not lead the search away
// from the others' rows: a row that it finds no sequence for is looked for in all of them (so are rows of
// no sequence).
constexpr int AP_ROWS = 4, AP_NT = AP_ROWS * ROW16, AP_LAYERS = 9;
__global__ void __launch_bounds__(AP_NT) cache_append_kernel(const PagedCache c, const int32_t *cu,
                                                             int n_seqs, int64_t total,
                                                             const uint4 *rows) {
  __shared__ int s_page[AP_ROWS], s_row[AP_ROWS];
  after_previous();
  if (blockIdx.x == 0)
    for (int n = threadIdx.x; n < n_seqs; n += AP_NT)
      if (cu[n] < 0 || cu[n + 1] < cu[n] || cu[n + 1] > total) flag(c.err, ERR_BAD_SEQLEN);
  const int64_t t = (int64_t)blockIdx.x * AP_ROWS + threadIdx.x / ROW16;
  const int piece = threadIdx.x % ROW16;
  uint4 x[AP_LAYERS];
#pragma unroll
  for (int y = 0; y < AP_LAYERS; ++y)
    if (t < total && y < c.n_layers) x[y] = __ldcs(rows + ((size_t)y * total + t) * ROW16 + piece);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t mine = (int64_t)blockIdx.x * AP_ROWS + warp;
  if (warp < AP_ROWS && mine < total) {
    // the last sequence whose first row is at most this one, among lo .. hi - 1
    int lo = 0, hi = n_seqs;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, at = lo + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, at < hi && (int64_t)cu[at] <= mine);
      const int k = m ? 31 - __clz(m) : 0;  // offsets that do not rise give some place, inside all the same
      hi = lo + (k + 1) * step < hi ? lo + (k + 1) * step : hi;
      lo += k * step;
    }
    auto holds = [&](int n) {
      const int64_t first = cu[n], end = cu[n + 1];
      return first >= 0 && mine >= first && mine < end && end <= total;
    };
    bool found = holds(lo);
    for (int n0 = 0; !found && n0 < n_seqs; n0 += 32) {
      const unsigned m = __ballot_sync(0xffffffffu, n0 + lane < n_seqs && holds(n0 + lane));
      if (m) found = true, lo = n0 + __ffs((int)m) - 1;
    }
    if (lane == 0) {
      int page = -2, row = 0;  // no sequence's row: not written
      if (found) {
        const int len = c.lengths[lo];
        const int64_t pos = (int64_t)len + (mine - cu[lo]);
        page = len < 0 ? -1 : page_of(c, lo, pos);
        row = (int)(pos % c.page_size);
        if (page < 0) flag(c.err, ERR_BAD_INDEX);
      }
      s_page[warp] = page;
      s_row[warp] = row;
    }
  }
  __syncthreads();
  if (t >= total) return;
  const int page = s_page[threadIdx.x / ROW16], row = s_row[threadIdx.x / ROW16];
  if (page < 0) return;
#pragma unroll
  for (int y = 0; y < AP_LAYERS; ++y)
    if (y < c.n_layers) pool_row(c, y, page, row)[piece] = x[y];
  for (int l = AP_LAYERS; l < c.n_layers; ++l)
    pool_row(c, l, page, row)[piece] = __ldcs(rows + ((size_t)l * total + t) * ROW16 + piece);
}

// The accepted path's rows moved up to lengths[n], lengths[n] + 1, ..: step d of the path is
// node path[d] >= d, so a thread that takes the steps in order never overwrites a row that one
// of its later steps still has to read.  The pages of all drafted positions are looked up beside the
// parents: a path that needs one that is not there is refused whole, before a row is moved.
constexpr int AC_LAYERS = 9, AC_NT = AC_LAYERS * ROW16;
__global__ void __launch_bounds__(AC_NT)
    cache_accept_kernel(const PagedCache c, const int32_t *cu, int64_t total, const int32_t *parent,
                        const int32_t *accept, int32_t *new_lengths) {
  __shared__ int s_par[64], s_path[64], s_page[64], s_m;
  after_previous();
  const int n = blockIdx.x, tid = threadIdx.x;
  const int lo = cu[n], hi = cu[n + 1], last = accept[n], len = c.lengths[n];
  int W = hi - lo;
  if (lo < 0 || hi < lo || hi > total || W > 64) {
    if (tid == 0) flag(c.err, ERR_BAD_SEQLEN);
    W = 0;
  }
  const bool ok = last >= -1 && last < W && len >= 0 && len <= INT_MAX - 64;
  if (tid == 0 && !ok) flag(c.err, ERR_BAD_INDEX);
  const int nodes = ok ? last + 1 : 0;
  for (int i = tid; i < nodes; i += AC_NT) {
    int p = parent[lo + i];
    if (p < -1 || p >= i) {
      flag(c.err, ERR_BAD_INDEX);
      p = -1;
    }
    s_par[i] = p;
    s_page[i] = page_of(c, n, (int64_t)len + i);
  }
  __syncthreads();
  if (tid == 0) {
    int steps = 0, missing = 0;
    for (int j = nodes - 1; j >= 0; j = s_par[j]) ++steps;
    for (int j = nodes - 1, d = steps; j >= 0; j = s_par[j]) {
      s_path[--d] = j;
      missing |= s_page[j] | s_page[d];  // a page that is not there is -1
    }
    s_m = missing < 0 ? 0 : steps;
    if (missing < 0) flag(c.err, ERR_BAD_INDEX);
  }
  __syncthreads();
  const int m = s_m, piece = tid % ROW16;
  int same = 0;  // the path's first steps are already in place
  while (same < m && s_path[same] == same) ++same;
  for (int l = tid / ROW16; l < c.n_layers; l += AC_LAYERS)
    for (int d0 = same; d0 < m; d0 += 8) {
      uint4 x[8];
#pragma unroll
      for (int y = 0; y < 8; ++y)
        if (d0 + y < m) {
          const int from = s_path[d0 + y];
          x[y] = pool_row(c, l, s_page[from], (len + from) % c.page_size)[piece];
        }
#pragma unroll
      for (int y = 0; y < 8; ++y)
        if (d0 + y < m) pool_row(c, l, s_page[d0 + y], (len + d0 + y) % c.page_size)[piece] = x[y];
    }
  if (tid == 0) new_lengths[n] = ok ? len + m : len;
}

// ---- pages -----------------------------------------------------------------------------------

// `count` 16-byte pieces from one page to another, by the whole CTA, eight in flight a thread.
__device__ __forceinline__ void copy_pieces(uint4 *dst, const uint4 *src, int count) {
  for (int i0 = threadIdx.x; i0 < count; i0 += 8 * blockDim.x) {
    uint4 x[8];
#pragma unroll
    for (int y = 0; y < 8; ++y)
      if (i0 + y * (int)blockDim.x < count) x[y] = src[i0 + y * blockDim.x];
#pragma unroll
    for (int y = 0; y < 8; ++y)
      if (i0 + y * (int)blockDim.x < count) dst[i0 + y * blockDim.x] = x[y];
  }
}

// Page src[i] to page dst[i] in every layer.  An entry whose target is named by an earlier entry,
// or is a source of any entry, is flagged and skipped, so no copy reads what another writes.
constexpr int CP_NT = 256;
__global__ void __launch_bounds__(CP_NT) pages_copy_kernel(const PagedCache c, const int32_t *src,
                                                           const int32_t *dst, int n) {
  after_previous();
  const int i = blockIdx.x, layer = blockIdx.y;
  const int a = src[i], b = dst[i];
  if (a < 0 || a >= c.n_pages || b < 0 || b >= c.n_pages) {
    if (threadIdx.x == 0 && layer == 0) flag(c.err, ERR_BAD_INDEX);
    return;
  }
  int clash = 0;
  for (int j = threadIdx.x; j < n; j += CP_NT)
    clash |= (src[j] == b && !(j == i && a == b)) || (j < i && dst[j] == b);
  if (__syncthreads_or(clash)) {
    if (threadIdx.x == 0 && layer == 0) flag(c.err, ERR_BAD_INDEX);
    return;
  }
  if (a != b) copy_pieces(pool_row(c, layer, b, 0), pool_row(c, layer, a, 0), c.page_size * ROW16);
}

// All pages of the listed sequences released; a sequence listed twice is released once.
__global__ void __launch_bounds__(128) pages_free_kernel(PagedCache c, int32_t *table, int32_t *lengths,
                                                         int32_t *refs, int32_t *held, int n_slots,
                                                         const int32_t *slots) {
  __shared__ int s_held;
  after_previous();
  const int slot = slots[blockIdx.x];
  if (slot < 0 || slot >= n_slots) {
    if (threadIdx.x == 0) flag(c.err, ERR_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) {
    const int h = atomicExch(&held[slot], 0);
    if (h < 0 || h > c.max_pages) flag(c.err, ERR_BAD_INDEX);
    s_held = h < 0 ? 0 : (h > c.max_pages ? c.max_pages : h);
    lengths[slot] = 0;
  }
  __syncthreads();
  for (int j = threadIdx.x; j < s_held; j += 128) {
    int32_t *e = table + (size_t)slot * c.max_pages + j;
    const int p = *e;
    if (p < 0 || p >= c.n_pages) {
      flag(c.err, ERR_BAD_INDEX);
    } else if (atomicSub(&refs[p], 1) <= 0) {  // held by nobody: the count goes back to 0
      atomicAdd(&refs[p], 1);
      flag(c.err, ERR_BAD_INDEX);
    }
    *e = -1;
  }
}

constexpr int BK = 1024;    // threads of the bookkeeping CTA
constexpr int KEEP = 2048;  // entries whose notes fit its shared memory

// Exclusive sum over the CTA; s holds 33 ints.
__device__ __forceinline__ int block_scan(int v, int *s, int &all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s[lane], z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    s[lane] = z - w;
    if (lane == 31) s[32] = z;
  }
  __syncthreads();
  all = s[32];
  return s[warp] + x - v;
}

// Which of the 16 pages from `base` on are free.
__device__ __forceinline__ uint32_t free_bits(const int32_t *refs, int base, int n_pages) {
  uint32_t bits = 0;
  if (base + 16 <= n_pages) {
    int4 v[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = reinterpret_cast<const int4 *>(refs + base)[y];
#pragma unroll
    for (int y = 0; y < 4; ++y)
      bits |= (uint32_t)((v[y].x <= 0) | (v[y].y <= 0) << 1 | (v[y].z <= 0) << 2 | (v[y].w <= 0) << 3) << (4 * y);
  } else {
    for (int y = 0; y < 16 && base + y < n_pages; ++y) bits |= (uint32_t)(refs[base + y] <= 0) << y;
  }
  return bits;
}

// The first `want` free pages in page order to list[]; returns how many there are (at most want).
__device__ __forceinline__ int find_free(const int32_t *refs, int n_pages, int want, int32_t *list, int *s) {
  int found = 0;
  for (int p0 = 0; p0 < n_pages && found < want; p0 += BK * 16) {
    const int base = p0 + threadIdx.x * 16;
    uint32_t bits = free_bits(refs, base, n_pages);
    int all, at = found + block_scan(__popc(bits), s, all);
    for (; bits && at < want; bits &= bits - 1, ++at) list[at] = base + __ffs((int)bits) - 1;
    found += all;
  }
  __syncthreads();  // list[] is complete
  return found < want ? found : want;
}

// Fork: claims, lengths and the new pages (one CTA); plan[f] = (parent or -1, child, new page or
// -1, length).  held[child] carries the claim f - n < 0 until the child is settled, so the
// earliest entry that names a child has it.
__global__ void __launch_bounds__(BK) pages_fork_plan_kernel(const PagedCache c, int32_t *table, int32_t *lengths,
                                                             int32_t *refs, int32_t *held, int n_slots,
                                                             const int32_t *src, const int32_t *dst, int n,
                                                             int4 *plan, int32_t *list) {
  __shared__ int s[33];
  after_previous();
  const int tid = threadIdx.x;
  auto inside = [&](int f) {
    return src[f] >= 0 && src[f] < n_slots && dst[f] >= 0 && dst[f] < n_slots;
  };
  for (int f = tid; f < n; f += BK)
    if (inside(f) && atomicAdd(&held[dst[f]], 0) <= 0) atomicMin(&held[dst[f]], f - n);
  __syncthreads();
  int want = 0;
  for (int f0 = 0; f0 < n; f0 += BK) {
    const int f = f0 + tid;
    int4 p = make_int4(-1, -1, -1, 0);
    int part = 0;
    if (f < n) {
      bool ok = inside(f);
      if (ok && held[dst[f]] == f - n) {
        p.y = dst[f];
        const int h = held[src[f]], len = lengths[src[f]];
        const int full = len >= 0 ? len / c.page_size : 0;
        part = len >= 0 && len % c.page_size ? 1 : 0;
        ok = h >= 0 && len >= 0 && full + part <= h && h <= c.max_pages;  // h < 0: a child of this call
        if (ok) p.x = src[f], p.w = len;
        else part = 0;
      } else {
        ok = false;  // held pages, or an earlier entry has the child
      }
      if (!ok) flag(c.err, ERR_BAD_INDEX);
    }
    int all;
    const int rank = want + block_scan(part, s, all);
    if (f < n) {
      p.z = part ? rank : -1;
      plan[f] = p;
    }
    want += all;
  }
  const int got = want ? find_free(refs, c.n_pages, want, list, s) : 0;
  __syncthreads();
  for (int f = tid; f < n; f += BK) {
    int4 p = plan[f];
    if (p.y < 0) continue;
    if (p.x >= 0 && p.z >= got) {  // no page left: the child stays empty
      flag(c.err, ERR_NO_PAGES);
      p.x = -1;
    }
    if (p.x < 0) {
      held[p.y] = 0;
    } else {
      const int full = p.w / c.page_size;
      if (p.z >= 0) {
        p.z = list[p.z];
        refs[p.z] = 1;
        table[(size_t)p.y * c.max_pages + full] = p.z;
      }
      held[p.y] = full + (p.z >= 0);
      lengths[p.y] = p.w;
    }
    plan[f] = p;
  }
}

// Fork: the shared pages (y = n_layers) and the copies of the partly filled ones (a layer each).
__global__ void __launch_bounds__(CP_NT) pages_fork_kernel(const PagedCache c, int32_t *table, int32_t *refs,
                                                           const int4 *plan) {
  after_previous();
  const int4 p = plan[blockIdx.x];
  if (p.x < 0 || p.y < 0) return;
  const int full = p.w / c.page_size, layer = blockIdx.y;
  const int32_t *from = table + (size_t)p.x * c.max_pages;
  if (layer == c.n_layers) {
    for (int j = threadIdx.x; j < full; j += CP_NT) {
      const int g = from[j];
      if (g >= 0 && g < c.n_pages) atomicAdd(&refs[g], 1);
      else flag(c.err, ERR_BAD_INDEX);
      table[(size_t)p.y * c.max_pages + j] = g;
    }
  } else if (p.z >= 0) {
    const int g = from[full];
    if (g >= 0 && g < c.n_pages)
      copy_pieces(pool_row(c, layer, p.z, 0), pool_row(c, layer, g, 0), p.w % c.page_size * ROW16);
    else if (threadIdx.x == 0 && layer == 0) flag(c.err, ERR_BAD_INDEX);
  }
}

// Reserve: room for extra[i] positions past lengths[slots[i]]; pages go to the entries in order
// while they last.  While the call runs, held[] of a named sequence carries the claim i - n < 0
// of the earliest entry that names it; saved[i] keeps its value (-1: entry refused), and
// first[i] .. first[i + 1] are the ranks of the entry's pages among the free ones.
__global__ void __launch_bounds__(BK) pages_reserve_kernel(const PagedCache c, int32_t *table, int32_t *refs,
                                                           int32_t *held, int n_slots, const int32_t *slots,
                                                           const int32_t *extra, int n, int32_t *saved,
                                                           int32_t *first) {
  __shared__ int s[33];
  __shared__ int32_t s_saved[KEEP], s_first[KEEP + 1];
  after_previous();
  if (n <= KEEP) saved = s_saved, first = s_first;
  const int tid = threadIdx.x;
  auto inside = [&](int i) { return slots[i] >= 0 && slots[i] < n_slots; };
  for (int i = tid; i < n; i += BK) saved[i] = inside(i) ? held[slots[i]] : -1;
  __syncthreads();
  for (int i = tid; i < n; i += BK)
    if (inside(i)) atomicMin(&held[slots[i]], i - n);
  __syncthreads();
  int64_t want = 0;  // max_pages <= 2^20: one block_scan's sum fits 32 bits
  for (int i0 = 0; i0 < n; i0 += BK) {
    const int i = i0 + tid;
    int need = 0;
    if (i < n) {
      const bool mine = inside(i) && held[slots[i]] == i - n;
      bool ok = mine;
      if (mine) {
        const int len = c.lengths[slots[i]], e = extra[i], h = saved[i];
        const int64_t pages = ((int64_t)len + e + c.page_size - 1) / c.page_size;
        ok = len >= 0 && e >= 0 && h >= 0 && h <= c.max_pages && pages <= c.max_pages;
        if (ok && pages > h) need = (int)pages - h;
        if (!ok) held[slots[i]] = h;  // refused: as it was
      }
      if (!ok) {
        saved[i] = -1;
        flag(c.err, ERR_BAD_INDEX);
      }
    }
    int all;
    const int64_t at = want + block_scan(need, s, all);
    if (i < n) first[i] = (int)(at < INT_MAX ? at : INT_MAX);
    want += all;
  }
  __syncthreads();
  const int most = want < c.n_pages ? (int)want : c.n_pages;
  if (tid == 0) first[n] = (int)(want < INT_MAX ? want : INT_MAX);
  __syncthreads();
  // the free pages in page order, each to the entry whose ranks hold its own
  int found = 0;
  for (int p0 = 0; p0 < c.n_pages && found < most; p0 += BK * 16) {
    const int base = p0 + tid * 16;
    uint32_t bits = free_bits(refs, base, c.n_pages);
    int all, at = found + block_scan(__popc(bits), s, all);
    for (; bits && at < most; bits &= bits - 1, ++at) {
      const int p = base + __ffs((int)bits) - 1, i = seq_of_token(first, n, at);
      refs[p] = 1;
      table[(size_t)slots[i] * c.max_pages + saved[i] + (at - first[i])] = p;
    }
    found += all;
  }
  const int got = found < most ? found : most;
  __syncthreads();
  for (int i = tid; i < n; i += BK) {
    if (saved[i] < 0) continue;
    const int need = first[i + 1] - first[i];
    if (need > 0 && first[i + 1] > got) {  // not all of its pages were there: none are taken
      flag(c.err, ERR_NO_PAGES);
      for (int r = first[i]; r < got; ++r) {
        int32_t *e = table + (size_t)slots[i] * c.max_pages + saved[i] + (r - first[i]);
        refs[*e] = 0;
        *e = -1;
      }
      held[slots[i]] = saved[i];
    } else {
      held[slots[i]] = saved[i] + need;
    }
  }
}

// Bit j of mask[i]: node j is node i or one of its ancestors.  A warp per sequence.
__global__ void __launch_bounds__(32) tree_mask_kernel(const int32_t *parent, const int32_t *cu, int64_t total,
                                                       int64_t *mask, int *err) {
  __shared__ int s_par[64];
  after_previous();
  const int n = blockIdx.x, lo = cu[n], hi = cu[n + 1];
  if (lo < 0 || hi < lo || hi > total || hi - lo > 64) {
    if (threadIdx.x == 0) flag(err, ERR_BAD_SEQLEN);
    return;
  }
  const int W = hi - lo;
  for (int i = threadIdx.x; i < W; i += 32) {
    int p = parent[lo + i];
    if (p < -1 || p >= i) {
      flag(err, ERR_BAD_INDEX);
      p = -1;
    }
    s_par[i] = p;
  }
  __syncwarp();
  for (int i = threadIdx.x; i < W; i += 32) {
    unsigned long long m = 0;
    for (int j = i; j >= 0; j = s_par[j]) m |= 1ull << j;
    mask[lo + i] = (int64_t)m;
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.stream = s;
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early, cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

cudaError_t launch_cache_append(const PagedCache &c, const int32_t *cu, int n_seqs, int64_t total,
                                const void *rows, cudaStream_t s) {
  return launch(cache_append_kernel, dim3((unsigned)((total + AP_ROWS - 1) / AP_ROWS)), AP_NT, s, c, cu, n_seqs, total,
                static_cast<const uint4 *>(rows));
}

cudaError_t launch_cache_accept(const PagedCache &c, const int32_t *cu, int n_seqs, int64_t total,
                                const int32_t *parent, const int32_t *accept, int32_t *new_lengths,
                                cudaStream_t s) {
  return launch(cache_accept_kernel, dim3(n_seqs), AC_NT, s, c, cu, total, parent, accept, new_lengths);
}

cudaError_t launch_pages_copy(const PagedCache &c, const int32_t *src, const int32_t *dst, int n,
                              cudaStream_t s) {
  return launch(pages_copy_kernel, dim3(n, c.n_layers), CP_NT, s, c, src, dst, n);
}

cudaError_t launch_pages_free(const PagedCache &c, int32_t *refs, int32_t *held, int n_slots,
                              const int32_t *slots, int n, cudaStream_t s) {
  return launch(pages_free_kernel, dim3(n), 128, s, c, const_cast<int32_t *>(c.table), const_cast<int32_t *>(c.lengths),
                refs, held, n_slots, slots);
}

// fork: plan and list; reserve: saved and first (which has an entry more)
size_t pages_ws_bytes(int n) { return (size_t)n * (sizeof(int4) + sizeof(int32_t)) + 16; }

cudaError_t launch_pages_fork(const PagedCache &c, int32_t *refs, int32_t *held, int n_slots,
                              const int32_t *src, const int32_t *dst, int n, void *ws, cudaStream_t s) {
  int4 *plan = static_cast<int4 *>(ws);
  int32_t *list = reinterpret_cast<int32_t *>(plan + n);
  int32_t *table = const_cast<int32_t *>(c.table);
  cudaError_t e = launch(pages_fork_plan_kernel, dim3(1), BK, s, c, table, const_cast<int32_t *>(c.lengths), refs, held,
                         n_slots, src, dst, n, plan, list);
  if (e != cudaSuccess) return e;
  return launch(pages_fork_kernel, dim3(n, c.n_layers + 1), CP_NT, s, c, table, refs, plan);
}

cudaError_t launch_pages_reserve(const PagedCache &c, int32_t *refs, int32_t *held, int n_slots,
                                 const int32_t *slots, const int32_t *extra, int n, void *ws, cudaStream_t s) {
  int32_t *saved = static_cast<int32_t *>(ws);
  return launch(pages_reserve_kernel, dim3(1), BK, s, c, const_cast<int32_t *>(c.table), refs, held, n_slots, slots, extra,
                n, saved, saved + n);
}

cudaError_t launch_tree_mask(const int32_t *parent, const int32_t *cu, int n_seqs, int64_t total,
                             int64_t *mask, int *err, cudaStream_t s) {
  return launch(tree_mask_kernel, dim3(n_seqs), 32, s, parent, cu, total, mask, err);
}

}  // namespace kda
