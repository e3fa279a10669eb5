// mla_sums.cu -- the attention that cached positions, or the keys of blocks, receive from all query
// rows of a sequence's step.
//
// With the absorbed form's scores ("Ling-3.1-flash: Grouped Routing and Two Different MLA Caches",
// section "Why weight absorption keeps the same attention function") s_rt = scale q_r . [c_t ; r_t]
// of the rows r (nodes x heads) and lse_r = ln sum_t exp(s_rt) over what row r sees,
//     weights_t += sum_r u_r exp(s_rt - lse_r)        (positions; u_r: the weight of r's node);
// of blocks, whose keys are the pages' mean rows, the scores s_rb themselves are left for the selection
// (mla_select.cu), with each row's maximum and sum over every 32 of them.
//
// The keys are the product's M side, D[256 keys x rows] = K Q^T on a pair of CTAs (cta_group::2, 128
// keys each), so a thread owns a key: the sum over rows runs along its own columns of tensor memory,
// in registers, in a fixed order, and what comes out is a number per key.  A key's garbage (no page, a
// row past the end) stays in its own lane and is never used.  A tile's keys stay in shared memory,
// 147 KB a CTA in nine blocks of 64 channels, while the step's rows pass by: up to 128 rows are
// resident for a whole sequence, more come in chunks of 128; chunks of nodes that do not count are
// passed over.
//
// What bounds it.  One node a sequence: the cache's bytes, which stream through once, block by block, as
// the products free the blocks (256 sequences of 2048 to 4096 positions, 64 heads: 137 us, 6.8 TB/s, the copy
// rate).  Many nodes: rows x positions x 1152 flop on the tensor cores; a chunk's 36 products of 64 cycles take
// about 2,900, with the epilogue beside them (8 sequences x 22 to 32 nodes x 8192 to 16384 positions: 150 us where
// all count, 1.40 PFLOP/s; chunks of 256 rows, whose products fill a buffer of tensor memory each and so are one
// sum over all channels, took 147 us and were up to 1.4e-6 off).  Few positions: latency, a launch of 8 us.
#include "batch_sums.h"
#include "kda_common.cuh"
#include "kda_internal.h"
#include "mla_pair.cuh"

#include <atomic>
#include <cstring>

namespace kda {
namespace {

using namespace tc;

constexpr int TK = 576, KB = TK / 64;
constexpr int CHUNK = 128;             // rows of a product: as many are resident, more are streamed
constexpr int NQ = KB, QK = 3;         // rows' slots, a block each; resident rows come by threes of blocks
constexpr int DCOLS = 256;             // columns of tensor memory of a product (two of them)
// Keys: positions 128 a CTA (M = 256), in one buffer of nine blocks; blocks 64 (M = 128: each CTA's lanes 64 ..
// hold the upper half of the rows' columns), in two, as their tiles are few and their latency counts
template <bool BLOCKS>
struct Keys {
  static constexpr int KC = BLOCKS ? 64 : 128, TILE = 2 * KC, BUFS = BLOCKS ? 2 : 1;
  static constexpr uint32_t SLOT = KC * 128;
};
constexpr uint32_t OFF_K = 0, OFF_Q = KB * 128 * 128;
constexpr uint32_t QSLOT = (CHUNK / 2) * 128, QBYTES = KB * (CHUNK / 2) * 128;
constexpr uint32_t SMEM = OFF_Q + QBYTES + 1024;
static_assert(NQ * QSLOT <= QBYTES && KB % QK == 0, "a chunk fits the resident rows' place");
// warps 0-7 sum, 8 loads keys, 9 rows, 10 and 11 issue the products of the even and of the odd blocks of
// channels; of blocks, the last three load keys too, of positions the last two rows.  A thread issues a product in
// 80 cycles at best, waits come on top; a load costs its thread some 450 (the window above: 181 us with one
// issuing warp, 200 with two and one for the rows' loads, 150 so).
constexpr int W_KEYS = 8, W_ROWS = 9, W_MMA = 10, W_MORE = 12, NTP = 448, NTB = 480;
constexpr int MAX_CLUSTERS = 80;  // of two CTAs (152 SMs: 76)
constexpr int KNOWN = 32;         // sequences of a run that are looked at once

// barriers; L: the leading CTA's are used by both
enum {
  B_KFULL = 0,                  // L  a key block is there in both CTAs; of blocks, a buffer of them
  B_KEMPTY = B_KFULL + KB,      //    the products have read it
  B_QFULL = B_KEMPTY + KB,      // L  a slot of streamed rows
  B_QEMPTY = B_QFULL + NQ,
  B_RFULL = B_QEMPTY + NQ,      // L  the resident rows (two)
  B_REMPTY = B_RFULL + 2,
  B_DFULL = B_REMPTY + 2,       //    a product is done (two buffers)
  B_DFREE = B_DFULL + 2,        // L  and read
  B_DRAIN = B_DFREE + 2, B_N = B_DRAIN + 2
};

struct SumMaps {
  CUtensorMap k, q[4], q3[4];  // query rows in boxes of 16, 32, 48 and 64, one and three blocks of channels each
};

struct Seq {
  int lo, rows, len, keys, tiles;
  unsigned long long live;  // chunks that hold a node that counts (8192 rows: 64 at most)
  // of a tile, in chunks' products: its keys' way into shared memory takes as long as three
  __device__ __forceinline__ int cost() const { return max(__popcll(live), 3); }
};
// the live chunk behind chunk ch (-1: the first), or -1
__device__ __forceinline__ int next_chunk(const Seq &s, int ch) { return __ffsll((long long)(ch < 0 ? s.live : s.live & (~1ull << ch))) - 1; }
template <bool BLOCKS>
__device__ __forceinline__ Seq seq_of(const KeySumArgs &a, int n, bool tell) {
  Seq s;
  s.lo = a.cu_nodes[n];
  const int hi = a.cu_nodes[n + 1];
  int W = hi - s.lo;
  if (s.lo < 0 || hi < s.lo || hi > a.total || W > 64) {
    if (tell && a.err) atomicOr(a.err, ERR_BAD_SEQLEN);
    W = 0;
  }
  s.len = a.c.lengths[n];
  const int64_t room = (int64_t)a.c.max_pages * a.c.page_size;
  const int64_t last = (int64_t)s.len + W;
  if (W > 0 && (s.len < 0 || last > room || (!BLOCKS && last > a.out_stride))) {
    if (tell && a.err) atomicOr(a.err, ERR_BAD_INDEX);
    s.len = 0, W = 0;
  }
  s.rows = W * a.H;
  s.keys = W == 0 ? 0 : BLOCKS ? s.len / a.c.page_size : s.len + W;
  const int chunks = s.rows <= CHUNK ? 1 : (s.rows + CHUNK - 1) / CHUNK;
  s.live = ~0ull >> (64 - chunks);
  if (!BLOCKS && a.node_weight) {
    s.live = 0;
    for (int i0 = 0; i0 < W; i0 += 16) {  // sixteen on their way
      float u[16];
#pragma unroll
      for (int y = 0; y < 16; ++y) u[y] = i0 + y < W ? a.node_weight[s.lo + i0 + y] : 0.f;
#pragma unroll
      for (int y = 0; y < 16; ++y) {
        const int i = i0 + y;
        if (u[y] != 0.f) s.live |= chunks == 1 ? 1ull : (~0ull << (i * a.H / CHUNK)) & (~0ull >> (63 - ((i + 1) * a.H - 1) / CHUNK));
      }
    }
    if (s.live == 0) s.keys = 0;
  }
  s.tiles = (s.keys + Keys<BLOCKS>::TILE - 1) / Keys<BLOCKS>::TILE;
  return s;
}

// This cluster's run of the batch's units, a tile's cost each; a tile belongs to the run that its first unit falls in.
template <bool BLOCKS>
struct Walk {
  int n, t;          // the next tile
  int64_t at, stop;  // its first unit; where the run ends
  bool fresh = true;
  const Seq *known;      // of sequences n0 .. in shared memory (a look at global memory takes longer than a tile)
  int n0, knowns;
  Seq s;
  int tile;
  bool first, last;  // of the sequence's tiles in this run
  __device__ __forceinline__ bool next(const KeySumArgs &a) {
    while (at < stop) {
      if (fresh) s = n - n0 < knowns ? known[n - n0] : seq_of<BLOCKS>(a, n, false), first = true, fresh = false;
      else first = false;
      if (t >= s.tiles) {
        if (++n >= a.n_seqs) return false;
        t = 0, fresh = true;
        continue;
      }
      tile = t++;
      at += s.cost();
      last = t >= s.tiles || at >= stop;
      return true;
    }
    return false;
  }
};

// The first unit of cluster c's run (a 64-bit division costs hundreds of cycles: only where needed).
__device__ __forceinline__ long long run_start(long long units, int c, int clusters) {
  return units < (1 << 24) ? (long long)((uint32_t)units * (uint32_t)c / (uint32_t)clusters) : units * c / clusters;
}

template <bool BLOCKS>
__host__ __device__ __forceinline__ int columns(const Seq &s, int chunk) {  // of a chunk's product, padded
  constexpr int pad = BLOCKS ? 63 : 31;
  const int r = s.rows - CHUNK * chunk;
  return r >= CHUNK ? CHUNK : (r + pad) & ~pad;
}
// The products drop bits of every partial sum (measured: weights up to 1.4e-6 off), so a score is the sum of two
// or, where tensor memory has room, four of them over a part of the channels each, added in fp32.
template <bool BLOCKS>
__device__ __forceinline__ int parts_of(int columns) {
  const int wide = BLOCKS ? columns / 2 : columns;  // of tensor memory
  return wide <= DCOLS / 4 ? 4 : 2;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(__cvta_generic_to_global(src)) : "memory");
}
// The CTA as sum_pass sees it.
struct Threads {
  int w, lane;
  __device__ __forceinline__ int warp() const { return w; }
  __device__ __forceinline__ bool last_lane() const { return lane == 31; }
  __device__ __forceinline__ void barrier() const { __syncthreads(); }
  __device__ __forceinline__ long long inclusive(long long x) const {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  }
};
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Sums over the warp's lanes of 16 columns: lane l gets column l & 15's.
__device__ __forceinline__ float columns_sum(float (&v)[16], int lane) {
#pragma unroll
  for (int c = 0; c < 16; ++c) v[c] += __shfl_xor_sync(0xffffffffu, v[c], 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int c = 0; c < o; ++c) {
      const bool up = lane & o;
      const float keep = up ? v[c + o] : v[c], give = up ? v[c] : v[c + o];
      v[c] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  return v[0];
}
__device__ __forceinline__ float lanes_max(float x) {  // (a NaN may be passed over: it shows in the sum)
  const int i = __float_as_int(x);
  const int m = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7fffffff));
  return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

template <bool BLOCKS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(BLOCKS ? NTB : NTP, 1)
    key_sums_kernel(const KeySumArgs a, const __grid_constant__ SumMaps maps) {
  constexpr int NT = BLOCKS ? NTB : NTP, KC = Keys<BLOCKS>::KC, TILE = Keys<BLOCKS>::TILE, BUFS = Keys<BLOCKS>::BUFS;
  constexpr uint32_t SLOT = Keys<BLOCKS>::SLOT;
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t s_bar[B_N];
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_abort;
  __shared__ PassSums<NT / 32> s_scan;
  __shared__ int s_n, s_t;
  __shared__ Seq s_known[KNOWN];
  __shared__ long long s_at;
  __shared__ __align__(16) float2 s_col[2][BLOCKS ? 2 : CHUNK];  // rows' (lse, weight)
  __shared__ __align__(16) uint8_t s_node[2][BLOCKS ? 16 : CHUNK];
  __shared__ uint32_t s_counts[2][CHUNK / 32];  // bits of the rows that count
  __shared__ float s_half[2][BLOCKS ? 1 : KC];
  const uint32_t raw = smem_u32(dyn);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int cid = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  auto bar = [&](int i) { return smem_u32(&s_bar[i]); };
  if (tid < B_N) {
    int n = 1;
    if (tid < B_KEMPTY) n = BLOCKS ? 8 : 2;              // the loaders of both CTAs
    else if (tid < B_QFULL) n = BLOCKS ? 2 : 1;          // the issuing warps that read it
    else if (tid < B_QEMPTY) n = 2;
    else if (tid < B_RFULL) n = 1;
    else if (tid < B_DFREE) n = 2;
    if (tid == B_DFREE || tid == B_DFREE + 1) n = 16;                                 // the sums' warps
    mbar_init(bar(tid), n);
    mbar_fence_init();
  }
  if (tid == 64) s_abort = 0, s_n = 0, s_t = 0, s_at = 0;
  if (tid >= 96 && (tid == 96 ? !BLOCKS : tid < 105 && a.total * a.H > CHUNK))  // the maps that there are
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.k + (tid - 96)) : "memory");
  if (warp == W_MMA) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  // launched while the kernel before runs out: nothing of global memory is read or written above
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // barriers and tensor memory are there in this CTA; waited for below

  // ---- this cluster's run of the batch's units: sequences' units summed up, a thread each --------
  Seq mine = {};       // of the first NT sequences
  long long at = 0;    // units before this thread's sequence
  int passes = 0;
  auto sum_up = [&](const Seq &s, long long &before) {  // returns the units before it, adds all to `before`
    return sum_pass(Threads{warp, lane}, s_scan, passes, (long long)s.tiles * s.cost(), before);
  };
  long long total = 0;
  for (int n0 = 0; n0 < a.n_seqs; n0 += NT) {
    Seq s = {};
    if (n0 + tid < a.n_seqs) s = seq_of<BLOCKS>(a, n0 + tid, blockIdx.x == 0);
    const long long x = sum_up(s, total);
    if (n0 == 0) mine = s, at = x;
  }
  const long long begin = run_start(total, cid, clusters), stop = run_start(total, cid + 1, clusters);
  if (stop > begin) {  // the first tile whose first unit is at or behind `begin`
    auto claim = [&](const Seq &s, long long at, int n) {
      const int cost = s.cost();
      if (at <= begin && begin < at + (long long)s.tiles * cost) {
        const int t = (int)(begin - at + cost - 1) / cost;  // (a sequence has at most 2^26 units)
        s_n = n, s_t = t, s_at = at + (long long)t * cost;
      }
    };
    claim(mine, at, tid);
    if (a.n_seqs > NT) {
      long long before = 0;
      for (int n0 = 0; n0 < a.n_seqs && before <= begin; n0 += NT) {
        Seq s = {};
        if (n0 + tid < a.n_seqs) s = seq_of<BLOCKS>(a, n0 + tid, false);
        const long long x = sum_up(s, before);
        if (n0 > 0) claim(s, x, n0 + tid);
      }
    }
  }
  __syncthreads();
  if (tid >= s_n && tid < s_n + KNOWN) s_known[tid - s_n] = mine;
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  Walk<BLOCKS> walk;
  walk.known = s_known, walk.n0 = s_n, walk.knowns = s_n + KNOWN <= NT ? KNOWN : s_n < NT ? NT - s_n : 0;
  walk.n = s_n, walk.t = s_t, walk.at = s_at, walk.stop = stop > begin ? stop : s_at;
  // A wait that runs out raises s_abort; from then on waits fail at once.  The warps of the sums walk
  // on to the end without waiting (they meet on a named barrier), the others issue nothing more.
  auto wait = [&](int i, uint32_t parity) {
#pragma unroll 1
    for (long it = 0; it < kWaitLimit; ++it) {
      if (mbar_try_wait(bar(i), parity & 1)) return true;
      if (s_abort) return false;
    }
    s_abort = 1;
    return false;
  };
  auto warp_wait = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };
  // the leading CTA's barrier expects both CTAs' bytes; the other CTA only arrives (its bytes cannot
  // come before the phase they belong to: its place was freed by that phase's products)
  auto announce = [&](int i, uint32_t bytes) {
    if (rank == 0) mbar_expect_tx(bar(i), 2 * bytes);
    else arrive_pair(map_shared_rank(bar(i), 0));
  };
  const int lp = 31 - __clz(a.c.page_size);

  if (warp == W_KEYS || (BLOCKS && warp >= W_MORE)) {
    // ---- key blocks: positions by tile loads, a lane each; blocks by 16-byte copies of their keys, 16 a
    //      warp, the next tile's pages looked up meanwhile (gathers by TMA, four rows each, took
    //      three times as long)
    auto known = [&](int page) { return page >= 0 && page < a.c.n_pages; };
    int tiles = 0;
    if constexpr (BLOCKS) {
      const int mine = 16 * (warp == W_KEYS ? 0 : warp - W_MORE + 1), piece = lane & 7;
      int page = 0, rows = 0;  // of the next tile: this lane's page, the warp's keys (may be below 0)
      auto look = [&]() {
        const int b = TILE * walk.tile + KC * (int)rank + mine;
        rows = walk.s.keys - b;
        page = lane < 16 && lane < rows ? a.c.table[(size_t)walk.n * a.c.max_pages + b + lane] : 0;
      };
      bool more = walk.next(a), ok = true;
      if (more) look();
      while (more) {
        if (!known(page)) {  // no page: any key stands for it
          if (a.err) atomicOr(a.err, ERR_BAD_INDEX);
          page = 0;
        }
        const char *key[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          key[y] = reinterpret_cast<const char *>(a.c.pool) + (size_t)__shfl_sync(0xffffffffu, page, 4 * y + (lane >> 3)) * (TK * 2) +
                   16 * piece;
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb) {
          if (tiles > 1 && kb == 0) ok = ok && warp_wait(B_KEMPTY + (tiles & 1), (uint32_t)((tiles >> 1) - 1));
          const uint32_t dst = sb + OFF_K + ((tiles & 1) * KB + kb) * SLOT + mine * 128;
          if (ok)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int r = 4 * y + (lane >> 3);
              if (r < rows) copy16(dst + r * 128 + ((piece ^ (r & 7)) << 4), key[y] + 128 * kb);
            }
          asm volatile("cp.async.commit_group;" ::: "memory");
        }
        more = walk.next(a);
        if (more) look();
        if (ok) {
          copies_wait<0>();
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) arrive_pair(map_shared_rank(bar(B_KFULL + (tiles & 1)), 0));
        }
        ++tiles;
      }
    } else {
      const int box = a.c.page_size < 64 ? a.c.page_size : 64, lb = 31 - __clz(box), in_page = a.c.page_size - 1;
      uint64_t policy;  // the cache's rows are read once
      asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
      while (walk.next(a)) {
        const int p = TILE * walk.tile + KC * (int)rank + (lane << lb);
        const bool here = (lane << lb) < KC && p < walk.s.keys;
        int page = here ? a.c.table[(size_t)walk.n * a.c.max_pages + (p >> lp)] : a.c.n_pages;
        if (!known(page)) {  // past the pool, where loads give zeros
          if (here && a.err) atomicOr(a.err, ERR_BAD_INDEX);
          page = a.c.n_pages;
        }
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb) {
          if (tiles > 0 && !warp_wait(B_KEMPTY + kb, (uint32_t)(tiles - 1))) continue;
          if (lane == 0) announce(B_KFULL + kb, SLOT);
          __syncwarp();
          if ((lane << lb) < KC)
            tma_pair_3d(sb + OFF_K + kb * SLOT + (lane << lb) * 128, &maps.k, 64 * kb, p & in_page, page,
                        map_shared_rank(bar(B_KFULL + kb), 0), policy);
        }
        ++tiles;
      }
    }
    // read before the CTA may end
    if (BLOCKS)
      for (int t = tiles > 2 ? tiles - 2 : 0; t < tiles; ++t) wait(B_KEMPTY + (t & 1), (uint32_t)(t >> 1));
    else if (tiles > 0)
      for (int kb = 0; kb < KB; ++kb) wait(B_KEMPTY + kb, (uint32_t)(tiles - 1));
    if (s_abort)  // a wait ran out: let the copies in flight land
      for (int y = 0; y < 100; ++y) __nanosleep(10000);
  } else if (warp == W_ROWS || (!BLOCKS && warp >= W_MORE)) {
    // ---- query rows: resident for a sequence, or a chunk's blocks of channels one by one.  Up to 64 resident
    //      rows take half of the place, so that the next sequence's are loaded meanwhile; the k-th
    //      resident sequence uses the barriers k & 1.
    const int which = warp == W_ROWS ? 0 : warp - W_MORE + 1, loaders = BLOCKS ? 1 : 3;
    int segs = 0, streamed = 0;
    bool wide = false;  // the last one took the whole place
    bool ring = false;  // a chunk's slots hold what was read last
    auto seg_done = [&](int k) {
      if (k >= 0) warp_wait(B_REMPTY + (k & 1), (uint32_t)(k >> 1));
    };
    while (walk.next(a)) {
      const int64_t row0 = (int64_t)walk.s.lo * a.H;
      if (walk.s.rows <= CHUNK) {
        if (!walk.first) continue;
        if (which > 0) {
          ring = false;
          ++segs;
          continue;
        }
        const int half = columns<BLOCKS>(walk.s, 0) / 2;
        const bool whole = 2 * half > CHUNK / 2;
        seg_done(segs - 2);
        if (whole || wide) seg_done(segs - 1);
        wide = whole;
        if (ring)
          for (int g = 0; g < NQ; ++g) warp_wait(B_QEMPTY + g, (uint32_t)(streamed - 1));
        ring = false;
        const int b = segs & 1;
        const uint32_t place = sb + OFF_Q + (whole || b == 0 ? 0 : QBYTES / 2);
        if (!s_abort) {
          if (lane == 0) {
            announce(B_RFULL + b, (uint32_t)(KB * half * 128));
            for (int kb = 0; kb < KB; kb += QK)
              tma_pair_3d(place + kb * half * 128, &maps.q3[half / 16 - 1], 0, (int)(row0 + half * (int)rank), kb,
                          map_shared_rank(bar(B_RFULL + b), 0));
          }
          __syncwarp();
        }
        ++segs;
      } else {
        if (!ring) seg_done(segs - 1);
        ring = true;
        for (int ch = next_chunk(walk.s, -1); ch >= 0; ch = next_chunk(walk.s, ch), ++streamed) {
          const int half = columns<BLOCKS>(walk.s, ch) / 2;
#pragma unroll 1
          for (int kb = which; kb < KB; kb += loaders)
            if (streamed == 0 || warp_wait(B_QEMPTY + kb, (uint32_t)(streamed - 1))) {
              if (lane == 0) {
                announce(B_QFULL + kb, (uint32_t)half * 128);
                tma_pair_3d(sb + OFF_Q + kb * QSLOT, &maps.q[half / 16 - 1], 0, (int)(row0 + CHUNK * ch + half * (int)rank), kb,
                            map_shared_rank(bar(B_QFULL + kb), 0));
              }
              __syncwarp();
            }
        }
      }
    }
    seg_done(segs - 2);
    seg_done(segs - 1);
    if (streamed > 0)
      for (int g = 0; g < NQ; ++g) wait(B_QEMPTY + g, (uint32_t)(streamed - 1));
    if (s_abort)
      for (int y = 0; y < 100; ++y) __nanosleep(10000);
  } else if (warp == W_MMA || warp == W_MMA + 1) {
    // ---- products (a thread each of two warps of the leading CTA: their partial sums are apart) ----
    if (rank == 0 && elect()) {
      const int which = warp - W_MMA, blocks = which == 0 ? 5 : 4;
      int i = 0, tiles = 0, segs = 0, streamed = 0;
      bool ok = true;
      while (ok && walk.next(a)) {
        const bool res = walk.s.rows <= CHUNK;
        if (res && walk.first && !(ok = wait(B_RFULL + (segs & 1), (uint32_t)(segs >> 1)))) break;
        const uint32_t place = sb + OFF_Q + (!res || columns<BLOCKS>(walk.s, 0) > CHUNK / 2 || !(segs & 1) ? 0 : QBYTES / 2);
        if (BLOCKS && !(ok = wait(B_KFULL + (tiles & 1), (uint32_t)(tiles >> 1)))) break;
        bool fill = !BLOCKS;  // the tile's keys are waited for
        for (int ch = next_chunk(walk.s, -1), then; ch >= 0 && ok; ch = then, ++i) {
          then = next_chunk(walk.s, ch);
          const int N = columns<BLOCKS>(walk.s, ch), parts = parts_of<BLOCKS>(N);
          const uint32_t id = idesc(1, TILE, (uint32_t)N, 0, 0), d = tm + DCOLS * (i & 1);
          if (i >= 2 && !(ok = wait(B_DFREE + (i & 1), (uint32_t)((i >> 1) - 1)))) break;
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < blocks; ++x) {
            const int kb = 2 * x + which;
            if (fill && !(ok = wait(B_KFULL + kb, (uint32_t)tiles))) break;
            if (!res && !(ok = wait(B_QFULL + kb, (uint32_t)streamed))) break;
            // its part of the sum: half of them are each warp's, which takes three blocks or two to one of two
            const int part = which * (parts >> 1) + (parts == 4 && x >= 3 - which ? 1 : 0);
            const bool fresh = x == 0 || (parts == 4 && x == 3 - which);
            const uint64_t ad = sdesc_sw128(sb + OFF_K + (tiles % BUFS * KB + kb) * SLOT, 16, 1024);
            const uint64_t bd = sdesc_sw128(place + kb * (res ? (N / 2) * 128 : QSLOT), 16, 1024);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma2(d + part * (DCOLS / parts), ad + 2 * ks, bd + 2 * ks, id, !fresh || ks > 0);
            if (!res) commit2(bar(B_QEMPTY + kb));
            if (!BLOCKS && then < 0) commit2(bar(B_KEMPTY + kb));
          }
          fill = false;
          if (!ok) break;
          if (BLOCKS && then < 0) commit2(bar(B_KEMPTY + (tiles & 1)));
          commit2(bar(B_DFULL + (i & 1)));
          if (!res) ++streamed;
        }
        if (ok && res && walk.last) {
          commit2(bar(B_REMPTY + (segs & 1)));
          ++segs;
        }
        ++tiles;
      }
      if (!ok) {  // a wait ran out: let the products in flight end
        commit2(bar(B_DRAIN + which));
        mbar_wait(bar(B_DRAIN + which), 0);
      }
    }
  } else {
    // ---- sums: lane l of tensor memory is the CTA's key l; warp w reads lanes 32 (w & 3) .. and
    //      half w >> 2 of the columns
    const int qw = warp & 3, hf = warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * qw) << 16;
    const uint32_t lead = map_shared_rank(bar(0), 0);
    int i = 0, loads = 0, tiles = 0;
    float2 ahead = {};    // the next chunk's row of this thread
    int ahead_node = 0;
    auto row_of = [&](const Seq &s, int ch) {  // (lse in units of log 2, weight)
      float2 x = make_float2(0.f, 0.f);
      const int r = CHUNK * ch + tid;
      if (tid >= CHUNK || r >= s.rows) return x;
      ahead_node = r / a.H;
      x.x = a.lse[(int64_t)s.lo * a.H + r] * 1.4426950408889634f;
      x.y = a.node_weight ? a.node_weight[s.lo + ahead_node] : 1.f;
      if (x.x == -INFINITY) x.y = 0.f;  // a row that sees nothing
      return x;
    };
    while (walk.next(a)) {
      const Seq s = walk.s;
      const int p = TILE * walk.tile + KC * (int)rank + (BLOCKS ? 32 * (qw & 1) : 32 * qw) + lane;
      // the nodes that see this thread's key, as bits
      unsigned long long vis = 0;
      if (p < s.keys) {
        const int page = a.c.table[(size_t)walk.n * a.c.max_pages + (BLOCKS ? p : p >> lp)];
        if (page >= 0 && page < a.c.n_pages) {
          if (BLOCKS || p < s.len) {
            vis = ~0ull;
          } else {  // a drafted row
            const int jn = p - s.len, W = s.keys - s.len;
            for (int x = 0; x < W; ++x)
              vis |= (unsigned long long)(a.mask ? (a.mask[s.lo + x] >> jn) & 1 : jn <= x) << x;
          }
        }
      }
      const bool none = __all_sync(0xffffffffu, BLOCKS ? p >= s.keys : vis == 0), whole = __all_sync(0xffffffffu, vis == ~0ull);
      float *out = nullptr;
      float old = 0.f;
      if (!BLOCKS && hf == 0 && vis != 0) {
        out = a.out + (size_t)walk.n * a.out_stride + p;
        old = *out;
      }
      float acc = 0.f;
      const int head = next_chunk(s, -1);
      for (int ch = head, then; ch >= 0; ch = then, ++i) {
        then = next_chunk(s, ch);
        const int N = columns<BLOCKS>(s, ch), parts = parts_of<BLOCKS>(N), share = BLOCKS ? N / 4 : N / 2, c0 = hf * share, c1 = c0 + share;
        if (!BLOCKS && (s.rows > CHUNK || walk.first)) {
          if (walk.first && ch == head) ahead = row_of(s, ch);
          const float2 x = ahead;
          const int b = loads & 1;
          if (tid < CHUNK) {
            s_col[b][tid] = x;
            s_node[b][tid] = (uint8_t)ahead_node;
            const uint32_t counts = __ballot_sync(0xffffffffu, x.y != 0.f);
            if (lane == 0) s_counts[b][warp] = counts;
          }
          ++loads;
          bar_sync(1, 256);  // two buffers: the next but one is written behind the next barrier
          if (s.rows > CHUNK) ahead = row_of(s, then >= 0 ? then : head);  // asked for while this one is summed
        }
        const int b = (loads - 1) & 1;
        wait(B_DFULL + (i & 1), (uint32_t)(i >> 1));
        tc_fence_after();
        const uint32_t d = tm + lanes + DCOLS * (i & 1);
        // 16 columns' scores, in `parts` parts: asked for, and added up once they are there
        auto ask = [&](int c, int part, float (&v)[16]) { tmem_ld16(d + part * (DCOLS / parts) + c, v); };
        auto add = [&](float (&v)[16], const float (&w)[16]) {
#pragma unroll
          for (int y = 0; y < 16; ++y) v[y] += w[y];
        };
        auto all_of_four = [&](int c, float (&v)[16]) {
          float w[3][16];
          ask(c, 0, v), ask(c, 1, w[0]), ask(c, 2, w[1]), ask(c, 3, w[2]);
          tmem_wait_ld();
          add(v, w[0]), add(w[1], w[2]), add(v, w[1]);
        };
        if (!BLOCKS) {
          if (!none) {
            auto sum = [&](const float (&v)[16], int c) {
              const float4 *col = reinterpret_cast<const float4 *>(&s_col[b][c]);
              const uint32_t counts = s_counts[b][c >> 5] >> (c & 16) & 0xffff;
              if (counts == 0) return;
              if (whole && counts == 0xffff) {
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  const float4 x = col[y];
                  acc = fmaf(x.y, ex2(fmaf(v[2 * y], a.scale_log2, -x.x)), acc);
                  acc = fmaf(x.w, ex2(fmaf(v[2 * y + 1], a.scale_log2, -x.z)), acc);
                }
              } else if (whole) {
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const float2 x = s_col[b][c + y];
                  const float e = ex2(fmaf(v[y], a.scale_log2, -x.x));
                  if (counts >> y & 1) acc = fmaf(x.y, e, acc);
                }
              } else {
                const uint4 nodes = *reinterpret_cast<const uint4 *>(&s_node[b][c]);
                const uint32_t word[4] = {nodes.x, nodes.y, nodes.z, nodes.w};
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const float4 x = col[y >> 1];
                  const float lse = y & 1 ? x.z : x.x, u = y & 1 ? x.w : x.y;
                  const float e = ex2(fmaf(v[y], a.scale_log2, -lse));
                  const uint32_t node = word[y >> 2] >> (8 * (y & 3)) & 63;
                  const uint32_t bit = (node & 32 ? (uint32_t)(vis >> 32) : (uint32_t)vis) >> (node & 31) & 1;
                  if ((counts >> y & 1) && bit) acc = fmaf(u, e, acc);
                }
              }
            };
            if (parts == 4) {
#pragma unroll 1
              for (int c = c0; c < c1; c += 16) {
                float v[16];
                all_of_four(c, v);
                sum(v, c);
              }
            } else {
              float v[2][16], w[2][16];
              ask(c0, 0, v[0]), ask(c0, 1, v[1]);
#pragma unroll 1
              for (int c = c0; c < c1; c += 32) {  // 16 columns are read while 16 are summed
                tmem_wait_ld();
                if (c + 16 < c1) ask(c + 16, 0, w[0]), ask(c + 16, 1, w[1]);
                add(v[0], v[1]);
                sum(v[0], c);
                if (c + 16 < c1) {
                  tmem_wait_ld();
                  if (c + 32 < c1) ask(c + 32, 0, v[0]), ask(c + 32, 1, v[1]);
                  add(w[0], w[1]);
                  sum(w[0], c + 16);
                }
              }
            }
          }
        } else if (!none) {
#pragma unroll 1
          for (int c = c0; c < c1; c += 16) {
            float v[16];  // (never more than 128 rows: four parts)
            all_of_four(c, v);
            const int r = CHUNK * ch + (qw >> 1) * (N / 2) + c;
            const int64_t row = (int64_t)s.lo * a.H + r;
            float *to = a.out + row * a.out_stride + p;
            float top = 0.f;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const float x = vis ? v[y] * a.scale_log2 : -INFINITY;
              if (r + y < s.rows && p < s.keys) to[y * a.out_stride] = x;
              const float m = lanes_max(x);
              if ((lane & 15) == y) top = m;
              v[y] = ex2(x - (m == -INFINITY ? 0.f : m));
            }
            const float sum = columns_sum(v, lane);
            if (lane < 16 && r + lane < s.rows) a.part[(row + lane) * a.part_stride + (p >> 5)] = make_float2(top, sum);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(lead + 8 * (B_DFREE + (i & 1)));
      }
      if (!BLOCKS) {
        if (hf == 1) s_half[tiles & 1][32 * qw + lane] = acc;
        bar_sync(1, 256);  // two buffers here too
        if (out) *out = old + (acc + s_half[tiles & 1][32 * qw + lane]);
      }
      ++tiles;
    }
  }
  if (lane == 0 && s_abort && a.err) atomicOr(a.err, ERR_MBAR_TIMEOUT);
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == W_MMA)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
}

template <bool BLOCKS>
cudaError_t launch_sums(const KeySumArgs &a, const SumMaps &maps, cudaStream_t s) {
  int dev = 0, nsm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> sms[64];  // SMs of a device once the kernel is opted in there (idempotent if raced)
  if (dev < 64) nsm = sms[dev].load();
  if (nsm == 0) {
    e = cudaFuncSetAttribute(key_sums_kernel<BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) sms[dev].store(nsm);
  }
  const int clusters = nsm / 2 < 1 ? 1 : (nsm / 2 < MAX_CLUSTERS ? nsm / 2 : MAX_CLUSTERS);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;  // each launch overlaps the end of the kernel before
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early, cfg.numAttrs = 1, cfg.stream = s;
  cfg.gridDim = dim3(2 * clusters), cfg.blockDim = dim3(BLOCKS ? NTB : NTP), cfg.dynamicSmemBytes = SMEM;
  return cudaLaunchKernelEx(&cfg, key_sums_kernel<BLOCKS>, a, maps);
}

// query rows as [9 blocks of 64 channels][rows], so that a load brings several blocks; a batch of few rows needs the
// small boxes alone (each map costs the host some 0.2 us)
template <bool BLOCKS>
bool row_maps(const KeySumArgs &a, SumMaps *maps) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const int64_t rows = a.total * a.H;
  const bool streams = rows > CHUNK;
  Seq all = {};
  all.rows = streams ? CHUNK : (int)rows;
  for (int i = 0; i < 8; ++i) {
    if (i < 4 ? !streams : 16 * (i - 3) > columns<BLOCKS>(all, 0) / 2) continue;
    cuuint64_t dims[3] = {64, (cuuint64_t)rows, KB}, strides[2] = {TK * 2, 128};
    cuuint32_t bx[3] = {64, (cuuint32_t)(16 * (i % 4 + 1)), (cuuint32_t)(i < 4 ? 1 : QK)}, es[3] = {1, 1, 1};
    if (fn(i < 4 ? &maps->q[i] : &maps->q3[i - 4], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, bx, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

}  // namespace

cudaError_t launch_cache_weights(const KeySumArgs &a, cudaStream_t s) {
  SumMaps maps;
  memset(&maps, 0, sizeof maps);
  const int box = a.c.page_size < 64 ? a.c.page_size : 64;
  if (!row_maps<false>(a, &maps) || !tree_map(&maps.k, a.c.pool, true, TK, a.c.page_size, a.c.n_pages, 64, box))
    return cudaErrorInvalidValue;
  return launch_sums<false>(a, maps, s);
}

cudaError_t launch_block_products(const KeySumArgs &a, cudaStream_t s) {
  SumMaps maps;
  memset(&maps, 0, sizeof maps);
  if (!row_maps<true>(a, &maps)) return cudaErrorInvalidValue;  // (no map of the keys: they come by copies)
  return launch_sums<true>(a, maps, s);
}

}  // namespace kda
