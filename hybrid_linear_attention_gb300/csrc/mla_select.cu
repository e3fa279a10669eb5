// mla_select.cu -- what of a long cache is read, and what of it is kept: the keys of full blocks, the
// selection of the largest values of a row, the compaction of an evicted sequence's rows.
//
// A block is a page of the latent cache: sequences that share a prefix share its full pages, and so
// the pages' keys.  The pages of the hybrid's sources name sparse reads without an interface ("Kimi
// K3.1 Pro: Sparse Reads ...", the index that picks positions); what is computed here:
//   key of a page      the mean of its rows, summed in fp32, rounded once to bf16;
//   selection          of `count` values: the first and the most recent are always taken, of the
//                      others the largest, among equals the lower index first, ascending;
//   eviction           a sequence keeps the selected positions; its rows move up in every layer.
// A selection is bound by latency: a CTA or a cluster of them takes a row of values, finds the value that the
// last one taken has by up to three passes of 11 bits over order-preserving keys (counts in shared memory,
// added up across the cluster), and writes what is taken by prefix sums.  Every sum is of whole numbers, so
// the result does not depend on the order.  Blocks' scores are summed up right before, by the same CTA or, where
// they are many, by a launch of their own.
// The moves are bound by memory.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_tc_ptx.cuh"

#include <atomic>
#include <climits>

namespace kda {
namespace {

using tc::cluster_rank;
using tc::cluster_sync;

constexpr int ROW16 = 576 * 2 / 16;  // 16-byte pieces of a row

__device__ __forceinline__ void flag(int *err, int bit) {
  if (err) atomicOr(err, bit);
}
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ bool page_known(const PagedCache &c, int page) { return page >= 0 && page < c.n_pages; }

// ---- block keys -------------------------------------------------------------------------------

// Units (page, layer) of the pages that filled up, CTA b taking every gridDim.x-th page.  A warp brings the
// pages in, 16 rows a bulk copy, through a ring in shared memory; 72 threads take a row's pieces, four rows
// at a time, and their four sums meet in shared memory.
constexpr int BK_ROWS = 4, BK_SUM = BK_ROWS * ROW16, BK_NT = BK_SUM + 32, BK_SEQS = BK_NT, BK_U = 4, BK_RING = 3;
constexpr int BK_SLOT = BK_U * BK_SUM * 16, BK_SMEM = BK_RING * BK_SLOT;
__global__ void __launch_bounds__(BK_NT, 3) block_keys_kernel(const PagedCache c, const int32_t *from, int n_seqs, bf16 *keys) {
  extern __shared__ __align__(128) uint4 ring[];  // [BK_RING][16 rows]
  __shared__ int s_end[BK_SEQS], s_first[BK_SEQS], s_warp[BK_NT / 32];
  __shared__ __align__(16) float s_sum[BK_ROWS][576];
  __shared__ __align__(8) uint64_t s_full[BK_RING], s_empty[BK_RING];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, layer = blockIdx.y;
  const int steps = c.page_size / (BK_U * BK_ROWS);
  const bool loads = warp == BK_SUM / 32;
  if (tid < BK_RING) {
    tc::mbar_init(tc::smem_u32(&s_full[tid]), 1);
    tc::mbar_init(tc::smem_u32(&s_empty[tid]), BK_SUM / 32);
    tc::mbar_fence_init();
  }
  int slot = 0;
  uint32_t par = 0;  // of the slot's next filling
  bool ok = true;    // no wait has run out
  after_previous();
  const int64_t room = (int64_t)c.max_pages * c.page_size;
  int64_t before = 0;  // pages of the sequences before n0
  for (int n0 = 0; n0 < n_seqs; n0 += BK_SEQS) {
    const int n = n0 + tid;
    int first = 0, count = 0;
    if (n < n_seqs) {
      const int f = from[n], t = c.lengths[n];
      if (f < 0 || t < 0 || t > room) {
        if (blockIdx.x == 0 && layer == 0) flag(c.err, ERR_BAD_INDEX);
      } else if (t > f) {
        first = f / c.page_size, count = t / c.page_size - first;
      }
    }
    int x = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < BK_NT / 32; ++w) {
      if (w < warp) x += s_warp[w];
      all += s_warp[w];
    }
    s_end[tid] = x, s_first[tid] = first;  // at most 320 x 2^20 pages
    __syncthreads();
    // page of unit u; past the last unit, or where there is none: -1
    auto look = [&](int u) {
      if (u >= all) return -1;
      int lo = 0, hi = BK_SEQS - 1;  // the first sequence whose pages end behind u
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > u) hi = mid;
        else lo = mid + 1;
      }
      return c.table[(size_t)(n0 + lo) * c.max_pages + s_first[lo] + u - (lo > 0 ? s_end[lo - 1] : 0)];
    };
    const uint4 *pool = reinterpret_cast<const uint4 *>(c.pool) + (size_t)layer * c.n_pages * c.page_size * ROW16;
    const int begin = (int)((blockIdx.x + gridDim.x - before % gridDim.x) % gridDim.x);
    int page = look(begin);
    for (int u = begin; u < all; u += gridDim.x) {
      const int mine = page;
      page = look(u + gridDim.x);
      if (!page_known(c, mine)) {
        if (tid == 0 && layer == 0) flag(c.err, ERR_BAD_INDEX);
        continue;
      }
      if (loads) {
        if (lane == 0)
          for (int s = 0; s < steps; ++s) {
            const uint32_t full = tc::smem_u32(&s_full[slot]);
            if (ok) ok = tc::mbar_wait(tc::smem_u32(&s_empty[slot]), par ^ 1);
            if (ok) {
              tc::mbar_expect_tx(full, BK_SLOT);
              asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                               tc::smem_u32(ring) + slot * BK_SLOT),
                           "l"(__cvta_generic_to_global(pool + ((size_t)mine * c.page_size + s * (BK_U * BK_ROWS)) * ROW16)),
                           "r"(BK_SLOT), "r"(full)
                           : "memory");
            }
            if (++slot == BK_RING) slot = 0, par ^= 1;
          }
        __syncwarp();
        continue;
      }
      float sum[8] = {};
#pragma unroll 1
      for (int s = 0; s < steps; ++s) {
        if (ok) ok = tc::mbar_wait(tc::smem_u32(&s_full[slot]), par);
#pragma unroll
        for (int x = 0; x < BK_U; ++x) {
          const uint4 v = ring[(slot * BK_U + x) * BK_SUM + tid];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) sum[2 * y] += __uint_as_float(w[y] << 16), sum[2 * y + 1] += __uint_as_float(w[y] & 0xffff0000u);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(tc::smem_u32(&s_empty[slot]));
        if (++slot == BK_RING) slot = 0, par ^= 1;
      }
      const int group = tid / ROW16, piece = tid - group * ROW16;
      asm volatile("bar.sync 1, %0;" ::"n"(BK_SUM) : "memory");  // the sums of the page before are read
      store4(&s_sum[group][8 * piece], make_float4(sum[0], sum[1], sum[2], sum[3]));
      store4(&s_sum[group][8 * piece + 4], make_float4(sum[4], sum[5], sum[6], sum[7]));
      asm volatile("bar.sync 1, %0;" ::"n"(BK_SUM) : "memory");
      // two channels a thread
      const float2 g0 = load2(&s_sum[0][2 * tid]), g1 = load2(&s_sum[1][2 * tid]), g2 = load2(&s_sum[2][2 * tid]), g3 = load2(&s_sum[3][2 * tid]);
      const float f = 1.f / c.page_size;  // a power of two
      if (ok)
        store2(keys + ((size_t)layer * c.n_pages + mine) * 576 + 2 * tid,
               make_float2(((g0.x + g1.x) + (g2.x + g3.x)) * f, ((g0.y + g1.y) + (g2.y + g3.y)) * f));
    }
    before += all;
    __syncthreads();
  }
  if (!ok) {  // let the copies in flight land
    flag(c.err, ERR_MBAR_TIMEOUT);
    for (int y = 0; y < 100; ++y) __nanosleep(10000);
  }
}

// ---- selection --------------------------------------------------------------------------------

// A number whose order is the values': NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}

constexpr int SEL_NT = 512, SEL_W = SEL_NT / 32, BINS = 2048;
constexpr int SC_ROWS = 1024, SC_GROUP = 128;  // rows, blocks at a time
constexpr int FEW = 16;                        // parts of a row's sum that a thread takes
constexpr int MAX_CS = 8;                      // CTAs of a cluster
static_assert(SEL_W == 16, "the groups' warps are counted in powers of two");

// The scores of blocks begin .. end - 1 of a sequence with `rows` rows from row0 on: each row's softmax over
// all of its blocks, U of them on their way, summed over the rows, to `out` and, where given, to `here`.
struct ScoreSpace {
  float lse[SC_ROWS];  // of rows, in units of log 2
  float part[SEL_W][SC_GROUP];
};
template <int U>
__device__ __forceinline__ void block_scores(const SelectArgs &a, int row0, int rows, int count, int begin, int end, float *out, float *here,
                                             ScoreSpace &s) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int groups = (end - begin + SC_GROUP - 1) / SC_GROUP, pieces = (count + 31) / 32;
  const int log_gp = groups <= 1 ? 0 : groups <= 2 ? 1 : groups <= 4 ? 2 : groups <= 8 ? 3 : 4;  // groups side by side
  const int share = SEL_W >> log_gp, sub = warp & (share - 1);                                    // warps of a group
  for (int r0 = 0; r0 < rows; r0 += SC_ROWS) {
    const int n = rows - r0 < SC_ROWS ? rows - r0 : SC_ROWS;
    const float *at = a.rows + (int64_t)(row0 + r0) * a.rows_stride;
    // U rows' scores of this thread's blocks (up to three more are read inside a row's stride, and not used)
    auto load = [&](int r, int b, float4 (&x)[U]) {
#pragma unroll
      for (int y = 0; y < U; ++y)
        x[y] = r + y * share < n && b < end ? load4(at + (int64_t)(r + y * share) * a.rows_stride + b)
                                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    };
    float4 ahead[U];  // the first of them are on their way while the log-sums are merged
    load(sub, begin + (warp >> (4 - log_gp)) * SC_GROUP + 4 * lane, ahead);
    const float2 *part = a.parts + (int64_t)(row0 + r0) * a.parts_stride;
    // a row's log-sum by a thread where its parts are few, all of them on their way (16 x 4 rows of 64 heads,
    // 256 to 512 blocks: the scores 22 -> 17 us) ...
    for (int r = tid; pieces <= FEW && r < n; r += SEL_NT) {
      float2 x[FEW];
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int p = 0; p < FEW; ++p) x[p] = p < pieces ? part[(int64_t)r * a.parts_stride + p] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int p = 0; p < FEW; ++p) M = fmaxf(M, x[p].x);
      const float t = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int p = 0; p < FEW; ++p) L = fmaf(exp2f(x[p].x - t), x[p].y, L);
      s.lse[r] = M == -INFINITY && L == 0.f ? 0.f : M + log2f(L);
    }
    // ... else by a warp, U rows on their way
    for (int r = warp; pieces > FEW && r < n; r += U * SEL_W) {
      float M[U], L[U];
#pragma unroll
      for (int k = 0; k < U; ++k) M[k] = -INFINITY, L[k] = 0.f;
      for (int p = lane; p < pieces; p += 32) {
        float2 x[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
          x[k] = r + k * SEL_W < n ? part[(int64_t)(r + k * SEL_W) * a.parts_stride + p] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const float top = fmaxf(M[k], x[k].x), t = top == -INFINITY ? 0.f : top;
          L[k] = L[k] * exp2f(M[k] - t) + exp2f(x[k].x - t) * x[k].y, M[k] = top;
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float top = warp_max(M[k]);
        const float sum = warp_sum(L[k] * exp2f(M[k] - (top == -INFINITY ? 0.f : top)));
        if (lane == 0 && r + k * SEL_W < n) s.lse[r + k * SEL_W] = top == -INFINITY && sum == 0.f ? 0.f : top + log2f(sum);
      }
    }
    __syncthreads();
    for (int g0 = 0; g0 < groups; g0 += 1 << log_gp) {
      const int b = begin + (g0 + (warp >> (4 - log_gp))) * SC_GROUP + 4 * lane;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b < end)
        for (int r = sub; r < n; r += U * share) {
          float4 x[U];
          if (g0 == 0 && r == sub) {
#pragma unroll
            for (int y = 0; y < U; ++y) x[y] = ahead[y];
          } else {
            load(r, b, x);
          }
#pragma unroll
          for (int y = 0; y < U; ++y) {
            const float e = r + y * share < n ? s.lse[r + y * share] : 0.f;
            acc.x += exp2f(x[y].x - e), acc.y += exp2f(x[y].y - e), acc.z += exp2f(x[y].z - e), acc.w += exp2f(x[y].w - e);
          }
        }
      store4(&s.part[warp][4 * lane], acc);
      __syncthreads();
      for (int t = tid; t < SC_GROUP << log_gp; t += SEL_NT) {
        const int g = t / SC_GROUP, o = begin + g0 * SC_GROUP + t;
        if (o >= end) break;
        float sum = r0 == 0 ? 0.f : out[o];
        for (int w = 0; w < share; ++w) sum += s.part[g * share + w][t % SC_GROUP];
        out[o] = sum;
        if (here) here[o] = sum;
      }
      __syncthreads();
    }
  }
}

// The step of a sequence as the two kernels of blocks see it; false: nothing is done for it (told once).
struct BlockStep {
  int lo, W, len, full;
};
__device__ __forceinline__ bool step_of(const SelectArgs &a, int n, bool tell, BlockStep &s) {
  s.lo = a.cu_nodes[n], s.len = a.c.lengths[n];
  const int hi = a.cu_nodes[n + 1];
  s.W = hi - s.lo, s.full = s.len / a.c.page_size;
  if (s.lo < 0 || hi < s.lo || hi > a.total || s.W > 64) {
    if (tell) flag(a.c.err, ERR_BAD_SEQLEN);
    return false;
  }
  if (s.W == 0) return false;  // nothing to attend from, and no error
  if (s.len < 0 || (int64_t)s.len + s.W > (int64_t)a.c.max_pages * a.c.page_size) {
    if (tell) flag(a.c.err, ERR_BAD_INDEX);
    return false;
  }
  return true;
}

// Scores of `width` blocks a CTA, where a sequence may have more than one CTA takes along with its selection.
constexpr int SC_WIDE = 4 * SC_GROUP;
template <int U>
__global__ void __launch_bounds__(SEL_NT, U > 4 ? 1 : 2) block_scores_kernel(const SelectArgs a, int width) {
  __shared__ __align__(16) ScoreSpace s_space;
  after_previous();
  const int n = blockIdx.y, begin = blockIdx.x * width;
  BlockStep s;
  if (!step_of(a, n, blockIdx.x == 0 && threadIdx.x == 0, s) || begin >= s.full) return;
  block_scores<U>(a, s.lo * a.H, s.W * a.H, s.full, begin, s.full < begin + width ? s.full : begin + width,
               a.scores + (size_t)n * a.stride, nullptr, s_space);
}

// p in CTA r of the cluster
template <typename T>
__device__ __forceinline__ const T *of_cta(const T *p, int r, int cs) {
  return cs > 1 ? reinterpret_cast<const T *>(tc::map_rank(p, r)) : p;
}

// What a CTA tells the others of its cluster.
struct __align__(16) SelectEnd {
  unsigned long long taken;  // taken for sure << 32 | equal to the threshold
  int gap, bad;              // the first value that is not taken; the last page that may not be read or written
};

template <bool EVICT>
__global__ void __launch_bounds__(SEL_NT, 2) select_kernel(const SelectArgs a) {
  constexpr int HELD = EVICT ? 16 : 4;  // values of a thread that stay in registers
  __shared__ __align__(16) union {
    ScoreSpace scores;
    int hist[2][BINS];
  } s_u;
  __shared__ uint32_t s_digit;
  __shared__ int s_need, s_equal, s_sums[SEL_W];
  __shared__ unsigned long long s_warp[SEL_W];
  __shared__ SelectEnd s_end;
  __shared__ int s_gap, s_refuse;
  __shared__ __align__(16) float s_scores[EVICT ? 4 : SC_WIDE];  // computed here
  after_previous();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = (int)cluster_ctas(), rank = (int)cluster_rank(), n = blockIdx.x / cs;
  const int page_size = a.c.page_size;
  const int64_t room = (int64_t)a.c.max_pages * page_size;
  const int len = a.c.lengths[n];
  const float *value = a.values + (size_t)n * a.stride;
  const int32_t *table = a.c.table + (size_t)n * a.c.max_pages;
  int count, tail = 0;  // values; pages behind the full blocks
  bool ok, fits = true;
  if (EVICT) {
    ok = len >= 0 && len <= room && len <= a.stride;
    count = len;
  } else {
    BlockStep s;
    ok = step_of(a, n, rank == 0 && tid == 0, s);
    count = s.full;
    if (ok) {
      tail = (int)(((int64_t)len + s.W + page_size - 1) / page_size) - count;
      fits = (count < a.most ? count : a.most) + tail <= a.out_stride;
      if (!fits && rank == 0 && tid == 0) flag(a.c.err, ERR_BAD_INDEX);
      if (a.rows) {  // (a cluster of one CTA then)
        block_scores<4>(a, s.lo * a.H, s.W * a.H, count, 0, count, a.scores + (size_t)n * a.stride, s_scores, s_u.scores);
        value = s_scores;
      }
    }
  }
  // this CTA's values
  const int width = ok ? ((count + cs - 1) / cs + 3) & ~3 : 0;
  const int64_t c0 = (int64_t)rank * width;
  const int cta_begin = c0 < count ? (int)c0 : count, cta_end = c0 + width < count ? (int)c0 + width : count;
  int32_t *out = a.out + (size_t)n * a.out_stride;
  if (!ok || !fits) {
    for (int64_t j = rank * SEL_NT + tid; j < a.out_stride; j += cs * SEL_NT) out[j] = -1;
    if (EVICT && a.new_values && a.new_values != a.values)  // how many of them count is not known: the whole row
      for (int64_t j = rank * SEL_NT + tid; j < a.stride; j += cs * SEL_NT) a.new_values[(size_t)n * a.stride + j] = value[j];
    if (rank == 0 && tid == 0) {
      if (EVICT) flag(a.c.err, ERR_BAD_INDEX);
      a.out_lengths[n] = EVICT ? len : 0;
    }
    return;
  }
  const int most = a.most, take = count < most ? count : most;
  const int lo = a.first, hi = count - a.recent;  // where values decide (count > most)
  uint32_t threshold = 0;
  int need = 0;  // of the values equal to it
  const int per0 = (width + SEL_NT - 1) / SEL_NT, per = per0 > 1 ? (per0 + 3) & ~3 : per0;
  const int begin = cta_begin + tid * per < cta_end ? cta_begin + tid * per : cta_end;
  const int end = begin + per < cta_end ? begin + per : cta_end;
  const bool choose = count > most;
  const int page_ahead = EVICT && choose && rank * SEL_NT + tid <= (count - 1) / page_size ? table[rank * SEL_NT + tid] : 0;
  // the keys of this thread's values in order, from registers where they fit
  uint32_t held[HELD] = {};
  const bool fit = per <= HELD;
  if (choose && fit) {
    float x[HELD];
    if (per > 1 && (reinterpret_cast<uintptr_t>(value) & 15) == 0) {  // begin is a multiple of four then
#pragma unroll
      for (int y = 0; y < HELD; y += 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (begin + y + 3 < end) v = load4(value + begin + y);
        else if (begin + y < end) {
          v.x = value[begin + y];
          if (begin + y + 1 < end) v.y = value[begin + y + 1];
          if (begin + y + 2 < end) v.z = value[begin + y + 2];
        }
        x[y] = v.x, x[y + 1] = v.y, x[y + 2] = v.z, x[y + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int y = 0; y < HELD; ++y) x[y] = begin + y < end ? value[begin + y] : 0.f;
    }
#pragma unroll
    for (int y = 0; y < HELD; ++y) held[y] = order_key(x[y]);
  }
  int named[EVICT ? 1 : HELD];  // blocks: their pages
  if (!EVICT && fit) {
#pragma unroll
    for (int y = 0; y < HELD; ++y) named[EVICT ? 0 : y] = begin + y < end ? table[begin + y] : -1;
  }
  auto each = [&](auto &&f) {
    if (fit) {
#pragma unroll
      for (int y = 0; y < HELD; ++y)
        if (begin + y < end) f(begin + y, held[y]);
    } else {
#pragma unroll 4
      for (int j = begin; j < end; ++j) f(j, order_key(value[j]));
    }
  };
  // eviction: a page of the sequence's and its count, asked for now and looked at behind the counting
  const int last_page = EVICT && choose ? (count - 1) / page_size : -1, first_look = rank * SEL_NT + tid;
  const int page0 = first_look <= last_page ? page_ahead : 0;
  const int ref0 = first_look <= last_page && a.refs && page_known(a.c, page0) ? a.refs[page0] : 0;
  if (tid == 0) s_end.taken = 0, s_end.gap = INT_MAX, s_end.bad = -1, s_gap = INT_MAX, s_refuse = 0;
  if (choose) {
    need = most - a.first - a.recent;
    if (need > 0) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        // bits 31 .. 21, 20 .. 10 and 9 .. 0; the bits above them are known
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, up = pass == 2 ? 10 : 21, mask = pass == 2 ? 1023 : BINS - 1;
        int *hist = s_u.hist[pass & 1];
        for (int b = tid; b < BINS; b += SEL_NT) hist[b] = 0;
        __syncthreads();
        each([&](int j, uint32_t k) {
          if (j >= lo && j < hi && (pass == 0 || k >> up == threshold >> up)) atomicAdd(&hist[k >> shift & mask], 1);
        });
        if (cs > 1) cluster_sync();
        else __syncthreads();
        // this thread's four bins, from the top
        const int top = BINS - 1 - 4 * tid;
        int v[4] = {}, sum = 0;
        int4 bins[MAX_CS];
#pragma unroll
        for (int r = 0; r < MAX_CS; ++r)
          bins[r] = r < cs ? *of_cta(reinterpret_cast<const int4 *>(hist + top - 3), r, cs) : make_int4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < MAX_CS; ++r) v[0] += bins[r].w, v[1] += bins[r].z, v[2] += bins[r].y, v[3] += bins[r].x;
#pragma unroll
        for (int y = 0; y < 4; ++y) sum += v[y];
        int x = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (lane == 31) s_sums[warp] = x;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < SEL_W; ++w)
          if (w < warp) x += s_sums[w];
        int above = x - sum;
        if (above < need && x >= need) {
          int y = 0;
          while (above + v[y] < need) above += v[y], ++y;
          s_digit = top - y, s_need = need - above, s_equal = v[y];
        }
        __syncthreads();
        threshold |= s_digit << shift;
        need = s_need;
        if (need == s_equal && threshold > 0) {  // all that begin so are taken
          --threshold, need = 0;
          break;
        }
      }
    } else {
      threshold = 0xffffffffu;  // no key reaches it
      __syncthreads();
    }
  }
  // 2: taken, 1: equal to the threshold (the first `need` of these are taken), 0: not
  auto sort_of = [&](int j, uint32_t k) { return !choose || j < lo || j >= hi || k > threshold ? 2 : k == threshold && need > 0 ? 1 : 0; };
  // how many are taken, and equal, before this thread's values
  unsigned long long mine = 0;
  if (choose) {
    int gap = INT_MAX;  // the first that is not taken for sure
    each([&](int j, uint32_t k) {
      const int s = sort_of(j, k);
      mine += s == 2 ? 1ull << 32 : s;
      if (s == 0 && gap == INT_MAX) gap = j;
    });
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    if (EVICT) {
      // the last page that is not there, or is shared and would be written
      int last_bad = -1;
      for (int j = first_look, p = page0, r = ref0; j <= last_page; j += cs * SEL_NT) {
        if (j != first_look) p = table[j], r = a.refs && page_known(a.c, p) ? a.refs[p] : 0;
        if (!page_known(a.c, p) || (r > 1 && j <= (most - 1) / page_size)) last_bad = j;
      }
      gap = __reduce_min_sync(0xffffffffu, gap), last_bad = __reduce_max_sync(0xffffffffu, last_bad);
      if (lane == 0 && gap != INT_MAX) atomicMin(&s_end.gap, gap);
      if (lane == 0 && last_bad >= 0) atomicMax(&s_end.bad, last_bad);
    }
    __syncthreads();
    unsigned long long all = 0;
#pragma unroll
    for (int w = 0; w < SEL_W; ++w) {
      if (w < warp) x += s_warp[w];
      all += s_warp[w];
    }
    if (tid == 0) s_end.taken = all;
    mine = x - mine;
    if (cs > 1) cluster_sync();
    else __syncthreads();
    gap = INT_MAX;
    int last_bad = -1;
    SelectEnd ends[MAX_CS];
#pragma unroll
    for (int r = 0; r < MAX_CS; ++r)
      if (r < cs) ends[r] = *of_cta(&s_end, r, cs);
#pragma unroll
    for (int r = 0; r < MAX_CS; ++r)
      if (r < cs) {
        if (r < rank) mine += ends[r].taken;
        if (EVICT) gap = min(gap, ends[r].gap), last_bad = max(last_bad, ends[r].bad);
      }
    if (EVICT && need > 0) {  // of the equal ones the first behind those that are taken
      int equal = (int)(uint32_t)mine, here = INT_MAX;
      each([&](int j, uint32_t k) {
        if (sort_of(j, k) == 1 && equal++ >= need && here == INT_MAX) here = j;
      });
      if (here != INT_MAX) atomicMin(&s_gap, here);
      if (cs > 1) cluster_sync();
      else __syncthreads();
#pragma unroll
      for (int r = 0; r < MAX_CS; ++r)
        if (r < cs) gap = min(gap, *of_cta(&s_gap, r, cs));
    }
    // Rows behind the first gap move: their pages have to be there, and nobody else's where they go.  A page that is
    // not there, or shared, behind the gap is seldom, and only then it is asked whether such a row needs it: from
    // positions `gap` .. on where the rows go, and from each kept one behind it.
    bool refused = false;
    if (EVICT && last_bad >= gap / page_size) {
      bool bad = false;
      for (int j = gap / page_size + first_look; gap < most && j <= (most - 1) / page_size; j += cs * SEL_NT) {
        const int p = table[j];
        bad |= !page_known(a.c, p) || (a.refs && a.refs[p] > 1);
      }
      int equal = (int)(uint32_t)mine;
      each([&](int j, uint32_t k) {
        const int s = sort_of(j, k);
        if (j > gap && (s == 2 || (s == 1 && equal < need))) bad |= !page_known(a.c, table[j / page_size]);
        equal += s == 1;
      });
      if (bad) s_refuse = 1;
      if (cs > 1) cluster_sync();
      else __syncthreads();
#pragma unroll
      for (int r = 0; r < MAX_CS; ++r)
        if (r < cs) refused |= *of_cta(&s_refuse, r, cs) != 0;
    }
    if (refused) {  // the sequence stays as it is
      for (int64_t j = rank * SEL_NT + tid; j < a.out_stride; j += cs * SEL_NT) out[j] = -1;
      if (a.new_values && a.new_values != a.values)
        for (int j = rank * SEL_NT + tid; j < count; j += cs * SEL_NT) a.new_values[(size_t)n * a.stride + j] = value[j];
      if (rank == 0 && tid == 0) {
        flag(a.c.err, ERR_BAD_INDEX);
        a.out_lengths[n] = len;
      }
      if (cs > 1) cluster_sync();
      return;
    }
  } else {
    mine = (unsigned long long)begin << 32;
  }
  int taken = (int)(mine >> 32), equal = (int)(uint32_t)mine;
  const bool aside = EVICT && a.new_values && a.new_values != a.values;
  float *fresh = EVICT && a.new_values ? a.new_values + (size_t)n * a.stride : nullptr;
  auto put = [&](int j, uint32_t k, int page) {
    const int s = sort_of(j, k);
    if (s == 2 || (s == 1 && equal < need)) {
      const int at = taken + (equal < need ? equal : need);
      out[at] = EVICT ? j : page;
      // the value again from its key, but for zeros, of which there are two, and NaN
      if (aside) fresh[at] = !choose || k == 0 || k == 0x80000000u ? value[j] : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
    }
    if (s == 2) ++taken;
    else equal += s;
  };
  if (fit) {
#pragma unroll
    for (int y = 0; y < HELD; ++y)
      if (begin + y < end) put(begin + y, held[y], named[EVICT ? 0 : y]);
  } else {
    for (int j = begin; j < end; ++j) put(j, choose ? order_key(value[j]) : 0, EVICT ? 0 : table[j]);
  }
  for (int64_t j = take + rank * SEL_NT + tid; j < a.out_stride; j += cs * SEL_NT)
    out[j] = !EVICT && j < take + tail ? table[count + (j - take)] : -1;
  if (EVICT) {
    if (aside) {
      for (int j = take + rank * SEL_NT + tid; j < count; j += cs * SEL_NT) fresh[j] = 0.f;
    } else if (fresh && choose) {
      // in place: a batch is read before it is written, and no later one reads what it wrote (a kept
      // position is never before its new one)
      if (cs > 1) cluster_sync();
      else __syncthreads();
      if (rank == 0) {
        for (int b = 0; b < take; b += 4 * SEL_NT) {
          float x[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int j = b + y * SEL_NT + tid;
            if (j < take) x[y] = value[__ldcg(out + j)];
          }
          __syncthreads();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int j = b + y * SEL_NT + tid;
            if (j < take) fresh[j] = x[y];
          }
          __syncthreads();
        }
        for (int j = take + tid; j < count; j += SEL_NT) fresh[j] = 0.f;
      }
    }
  }
  if (rank == 0 && tid == 0) a.out_lengths[n] = EVICT ? take : (int)((int64_t)take * page_size + len % page_size);
  if (cs > 1) cluster_sync();  // its shared memory is not read by the others any more
}

// Row kept[j] of each sequence moves to row j, in every layer.  A CTA takes 128 bytes of the rows (64 or 32
// where the GPU has room for as many CTAs at once: one sequence of 1024, nine layers, 15.0 us, with 128 17.1), 144
// rows at a time (288, 576), through a ring in shared memory of which all but one batch are on their way: a batch is
// written once all of its reads, and so those of the batches before, are done.  kept[j] >= j and both
// rise, so no later batch reads a row that an earlier one wrote.  A thread writes what it read itself; the
// places of a batch are looked up two ahead of its reads.  (64 sequences of 2048 to 4096 positions cut to 2048,
// nine layers: 430 us with the selection, 6.3 TB/s, 93 % of the copy rate; with the lookups on the way 540.  Wider
// slices leave long sequences to fewer CTAs: 4 sequences cut to 16384 250 us, with 384 bytes 436, whole rows 819.)
constexpr int MV_NT = 288, MV_U = 4, MV_STAGES = 4, MV_SMEM = MV_STAGES * MV_U * MV_NT * 16;
template <int MV_PIECES>
__global__ void __launch_bounds__(MV_NT, 3) evict_rows_kernel(const PagedCache c, const int32_t *kept_all, int budget) {
  constexpr int MV_ROWS = MV_NT / MV_PIECES, MV_BATCH = MV_ROWS * MV_U;
  extern __shared__ uint4 ring[];  // [stage][MV_U][MV_NT]
  after_previous();
  const int n = blockIdx.z, layer = blockIdx.y, tid = threadIdx.x, r = tid / MV_PIECES;
  const int piece = blockIdx.x * MV_PIECES + tid % MV_PIECES;
  const int32_t *kept = kept_all + (size_t)n * budget;
  const int last = kept[budget - 1];
  const int32_t *table = c.table + (size_t)n * c.max_pages;
  uint4 *rows = reinterpret_cast<uint4 *>(c.pool) + (size_t)layer * c.n_pages * c.page_size * ROW16 + piece;
  const int lp = 31 - __clz(c.page_size), in_page = c.page_size - 1;
  const int batches = (budget + MV_BATCH - 1) / MV_BATCH;
  // The places are looked up ahead, without a wait in between: `at` and `page` of the next batch to read, `then`
  // of the one behind it, `to` of the next batch to write.  at: kept position, -1 where the row stays.
  int at[MV_U], page[MV_U], then[MV_U], to[MV_U];
  auto row_of = [&](int b, int y) { return b * MV_BATCH + y * MV_ROWS + r; };
  auto look = [&](int b, int (&k)[MV_U]) {
#pragma unroll
    for (int y = 0; y < MV_U; ++y) k[y] = row_of(b, y) < budget ? kept[row_of(b, y)] : -1;
  };
  auto look_pages = [&](int b) {  // of `then`, which becomes the next batch
#pragma unroll
    for (int y = 0; y < MV_U; ++y) {
      at[y] = then[y] > row_of(b, y) ? then[y] : -1;
      page[y] = at[y] >= 0 ? table[at[y] >> lp] : 0;
    }
  };
  auto look_to = [&](int b) {
#pragma unroll
    for (int y = 0; y < MV_U; ++y) to[y] = row_of(b, y) < budget ? table[row_of(b, y) >> lp] : 0;
  };
  uint32_t moves = 0;  // MV_U bits a batch of the ring, the next one to be written lowest
  auto read = [&](int b) {
    uint4 *slot = ring + (b % MV_STAGES) * (MV_U * MV_NT) + tid;
#pragma unroll
    for (int y = 0; y < MV_U; ++y)
      if (at[y] >= 0) {
        moves |= 1u << ((MV_STAGES - 1) * MV_U + y);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(slot + y * MV_NT)),
                     "l"(__cvta_generic_to_global(rows + (((int64_t)page[y] << lp) + (at[y] & in_page)) * ROW16))
                     : "memory");
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  {  // the first batches' places all at once
    int k[MV_STAGES + 1][MV_U], p[MV_STAGES][MV_U];
#pragma unroll
    for (int b = 0; b <= MV_STAGES; ++b) look(b, k[b]);
    if (last < budget) return;  // nothing moves (or the sequence is refused)
#pragma unroll
    for (int b = 0; b < MV_STAGES; ++b)
#pragma unroll
      for (int y = 0; y < MV_U; ++y) {
        if (k[b][y] <= row_of(b, y)) k[b][y] = -1;
        p[b][y] = k[b][y] >= 0 ? table[k[b][y] >> lp] : 0;
      }
#pragma unroll
    for (int b = 0; b < MV_STAGES; ++b) {
#pragma unroll
      for (int y = 0; y < MV_U; ++y) at[y] = k[b][y], page[y] = p[b][y];
      if (b < MV_STAGES - 1) {
        read(b);
        moves >>= MV_U;
      }
    }
#pragma unroll
    for (int y = 0; y < MV_U; ++y) then[y] = k[MV_STAGES][y];
  }
  look_to(0);
#pragma unroll 1
  for (int b = 0; b < batches; ++b) {
    read(b + MV_STAGES - 1);
    look_pages(b + MV_STAGES);
    look(b + MV_STAGES + 1, then);
    asm volatile("cp.async.wait_group %0;" ::"n"(MV_STAGES - 1) : "memory");
    __syncthreads();
    const uint4 *x = ring + (b % MV_STAGES) * (MV_U * MV_NT) + tid;
#pragma unroll
    for (int y = 0; y < MV_U; ++y)
      if (moves >> y & 1) __stcs(rows + (((int64_t)to[y] << lp) + (row_of(b, y) & in_page)) * ROW16, x[y * MV_NT]);
    moves >>= MV_U;
    look_to(b + 1);
  }
}

// The weights of an accepted path's nodes to the places of its steps, those of the other nodes to 0.
__global__ void __launch_bounds__(64) weights_accept_kernel(float *weights, int64_t stride, const int32_t *lengths, const int32_t *cu,
                                                            int64_t total, const int32_t *parent, const int32_t *accept, int *err) {
  __shared__ int s_par[64], s_path[64], s_m;
  after_previous();
  const int n = blockIdx.x, tid = threadIdx.x, lo = cu[n], hi = cu[n + 1], W = hi - lo, last = accept[n], len = lengths[n];
  if (lo < 0 || hi < lo || hi > total || W > 64) {
    if (tid == 0) flag(err, ERR_BAD_SEQLEN);
    return;
  }
  if (last < -1 || last >= W || len < 0 || (int64_t)len + W > stride) {
    if (tid == 0) flag(err, ERR_BAD_INDEX);
    return;
  }
  if (tid <= last) {
    int p = parent[lo + tid];
    if (p < -1 || p >= tid) {
      flag(err, ERR_BAD_INDEX);
      p = -1;
    }
    s_par[tid] = p;
  }
  float *w = weights + (size_t)n * stride + len;
  __syncthreads();
  if (tid == 0) {
    int steps = 0;
    for (int j = last; j >= 0; j = s_par[j]) ++steps;
    s_m = steps;
    for (int j = last; j >= 0; j = s_par[j]) s_path[--steps] = j;
  }
  __syncthreads();
  const float x = tid < s_m ? w[s_path[tid]] : 0.f;
  __syncthreads();
  if (tid < W) w[tid] = x;
}

// The pages of the listed sequences that lie wholly behind their lengths released.
__global__ void __launch_bounds__(128) pages_trim_kernel(PagedCache c, int32_t *table, int32_t *refs, int32_t *held, int n_slots,
                                                         const int32_t *slots) {
  __shared__ int s_held, s_keep;
  after_previous();
  const int slot = slots[blockIdx.x];
  if (slot < 0 || slot >= n_slots) {
    if (threadIdx.x == 0) flag(c.err, ERR_BAD_INDEX);
    return;
  }
  if (threadIdx.x == 0) {
    const int len = c.lengths[slot];
    int keep = len < 0 ? INT_MAX : (int)(((int64_t)len + c.page_size - 1) / c.page_size);
    const int h = atomicMin(&held[slot], keep);  // a sequence listed twice is cut once
    if (len < 0 || h < 0 || h > c.max_pages || h < keep) flag(c.err, ERR_BAD_INDEX);
    s_held = h < 0 ? 0 : (h > c.max_pages ? c.max_pages : h), s_keep = keep;
  }
  __syncthreads();
  for (int j = s_keep < s_held ? s_keep + (int)threadIdx.x : s_held; j < s_held; j += 128) {
    int32_t *e = table + (size_t)slot * c.max_pages + j;
    const int p = *e;
    if (!page_known(c, p)) {
      flag(c.err, ERR_BAD_INDEX);
    } else if (atomicSub(&refs[p], 1) <= 0) {  // held by nobody: the count goes back to 0
      atomicAdd(&refs[p], 1);
      flag(c.err, ERR_BAD_INDEX);
    }
    *e = -1;
  }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int cluster, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster, at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at, cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Lets a kernel use that much shared memory on this device; done[device] once it may (idempotent if raced).
template <typename K>
cudaError_t opt_in(K kernel, int smem, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done[dev].load())) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev < 64) done[dev].store(true);
  return e;
}

// CTAs of a selection: one for up to 16 values a thread (an exchange between the CTAs of a cluster costs
// about as much as 16 values: 64 x 4096 take 10 us by one CTA each and 13 by four; 4 x 65536 by clusters of eight
// 18), as long as the GPU has room for the clusters (two CTAs an SM).
int select_ctas(int n_seqs, int64_t most_values) {
  int cs = 1;
  while (cs < MAX_CS && most_values > (int64_t)cs * SEL_NT * 16 && (int64_t)n_seqs * cs * 2 <= 304) cs *= 2;
  return cs;
}

}  // namespace

cudaError_t launch_block_keys(const PagedCache &c, const int32_t *from, int n_seqs, void *keys, cudaStream_t s) {
  static std::atomic<bool> opted[64];
  const cudaError_t e = opt_in(block_keys_kernel, BK_SMEM, opted);
  if (e != cudaSuccess) return e;
  const int ctas = 456 / c.n_layers;  // three an SM
  return launch(block_keys_kernel, dim3(ctas < 1 ? 1 : ctas, c.n_layers), 1, BK_NT, BK_SMEM, s, c, from, n_seqs, static_cast<bf16 *>(keys));
}

cudaError_t launch_block_select(const SelectArgs &args, int *launches, cudaStream_t s) {
  SelectArgs a = args;
  // one CTA takes its sequence's scores along where they are few
  const double scores = (double)a.total * a.H * a.c.max_pages / a.n_seqs;
  if (a.rows && (a.c.max_pages > SC_WIDE || scores > 16384. || !a.out)) {
    // as narrow as one wave of CTAs allows: of one an SM with eight rows on their way (16 x 4 nodes, 512 blocks: the
    // step 68 us, with four 71), else of two with four (256 x 1, 64 blocks: the call 18 us, with eight 23)
    auto ctas = [&](int w) { return (double)((a.c.max_pages + w - 1) / w) * a.n_seqs; };
    const bool few = ctas(SC_WIDE) <= 152.;
    int width = SC_GROUP;
    while (width < SC_WIDE && ctas(width) > (few ? 152. : 304.)) width *= 2;
    const cudaError_t e = launch(few ? block_scores_kernel<8> : block_scores_kernel<4>,
                                 dim3((a.c.max_pages + width - 1) / width, a.n_seqs), 1, SEL_NT, 0, s, a, width);
    if (e != cudaSuccess) return e;
    ++*launches;
    if (!a.out) return e;
    a.rows = nullptr;  // the scores are there
  }
  const int cs = select_ctas(a.n_seqs, a.c.max_pages);
  ++*launches;
  return launch(select_kernel<false>, dim3(a.n_seqs * cs), cs, SEL_NT, 0, s, a);
}

cudaError_t launch_cache_evict(const SelectArgs &a, int *launches, cudaStream_t s) {
  const int64_t room = (int64_t)a.c.max_pages * a.c.page_size;
  const int cs = select_ctas(a.n_seqs, room < a.stride ? room : a.stride);
  cudaError_t e = launch(select_kernel<true>, dim3(a.n_seqs * cs), cs, SEL_NT, 0, s, a);
  if (e != cudaSuccess) return e;
  ++*launches;
  static std::atomic<bool> opted[3][64];
  auto move = [&](auto kernel, int pieces, std::atomic<bool> (&done)[64]) {
    const cudaError_t e = opt_in(kernel, MV_SMEM, done);
    return e != cudaSuccess ? e : launch(kernel, dim3(ROW16 / pieces, a.c.n_layers, a.n_seqs), 1, MV_NT, MV_SMEM, s, a.c, a.out, a.most);
  };
  const int64_t units = (int64_t)a.n_seqs * a.c.n_layers;  // three CTAs an SM
  e = units * (ROW16 / 2) <= 456   ? move(evict_rows_kernel<2>, 2, opted[0])
      : units * (ROW16 / 4) <= 456 ? move(evict_rows_kernel<4>, 4, opted[1])
                                   : move(evict_rows_kernel<8>, 8, opted[2]);
  ++*launches;
  return e;
}

cudaError_t launch_weights_accept(float *weights, int64_t stride, const int32_t *lengths, const int32_t *cu, int n_seqs,
                                  int64_t total, const int32_t *parent, const int32_t *accept, int *err, cudaStream_t s) {
  return launch(weights_accept_kernel, dim3(n_seqs), 1, 64, 0, s, weights, stride, lengths, cu, total, parent, accept, err);
}

cudaError_t launch_pages_trim(const PagedCache &c, int32_t *refs, int32_t *held, int n_slots, const int32_t *slots, int n,
                              cudaStream_t s) {
  return launch(pages_trim_kernel, dim3(n), 1, 128, 0, s, c, const_cast<int32_t *>(c.table), refs, held, n_slots, slots);
}

}  // namespace kda
