// mla_tree.cu -- latent attention of a tree of drafted tokens over the paged cache.
//
// The absorbed form's function ("Ling-3.1-flash: Grouped Routing and Two Different MLA Caches",
// section "Why weight absorption keeps the same attention function") for several query nodes of
// a sequence at once: node i, head h has the 576-wide query [q~ ; q^R], every cached position t
// < len the key [c_t ; r_t] and the value c_t, and drafted node j, whose row is at position
// len + j, is a key of node i where bit j of i's mask is set:
//     s_t = scale q . [c_t ; r_t],  z = sum_t softmax(s)_t c_t  over the visible positions
// (z = 0 where none is).
//
// What bounds it: a sequence of len positions and R = nodes x heads query rows costs 2176 R len
// flop over 1152 len bytes, so beyond two nodes of 64 heads the tensor cores are the floor, not
// the cache's bytes.  z of R rows is 512 fp32 wide: tensor memory (256 KB) holds 64 rows of it
// beside the scores, and a 64-row product runs the tensor cores at half rate on one SM
// (measured: 2048 of 4096 multiply-adds a cycle).  So a pair of CTAs works on 128 rows with
// cta_group::2 products, M = 128 (64 rows each) and N = 256, which run at the full rate
// (measured: 64 cycles a K = 16 step; N = 128 takes 44 instead of 32):
//     S[128 x 256 positions] = Q C^T    each CTA holds its 64 query rows and 128 of the
//                                       positions, all 576 channels, in nine 64-channel blocks;
//     Z[128 x 512 latents] += P C       each CTA holds its 64 rows of weights and all 256
//                                       positions of its half of the latents, in eight
//                                       [64 positions x 128 latents] chunks.
// Blocks and chunks stream through a ring of 16 KB slots each (four and three), with a loading and
// an issuing warp each: while the softmax of tile t runs, S of t + 1 and Z of t - 1 are built side
// by side.  One thread's products leave gaps (measured: with a wait and a commit every four of
// them, 101 to 149 cycles a product instead of 64), two threads' fill each other's (64 cycles); one
// thread's loads cost it about 450 cycles a slot, so two load, a slot's loads in a row without a lookup
// between them (with one, pages of 16 positions were bound by it: 422 us for 283, pages of 64 278 for 266).
// That brings 272 KB to a CTA for 256 positions, 64 bytes a cycle at the products' full rate; TMA moves 41
// to 48 bytes a cycle and SM from L2, so L2 is the bound where the cache is read by several row tiles:
// 4 sequences x 11 to 16 nodes x 65536 positions 266 us in bursts of ten, 1.60 PFLOP/s, 83 % of the measured bf16
// peak; 290 to 304 us where calls follow one another for long (1.40 to 1.47 PFLOP/s: the power limit).
// The rings' depth is what that rate needs: a slot less in either costs 11 to 35 %, one more (weights of
// 128 positions at a time) gives back only what the smaller place for the weights costs.  With one node a
// sequence the same loop streams the cache: 256 sequences of 2048 to 4096 positions 198 us, 4.8 TB/s, and 202 to
// 211 among other calls (asking L2 for coming tiles, by bulk prefetches or by threads, measured slower: 247 to
// 272 us).  There every byte of the cache still comes into shared memory 1.85 times, for the scores and for the
// values, and with 64 heads half of the products' rows are empty.
//
// Work is dealt in tiles of 256 positions: clusters form groups of G that take G row tiles of a
// sequence side by side (they read the same positions at the same time, so HBM sees them once),
// and every group takes an equal run of the batch's tiles.  A run that begins or ends inside a
// sequence leaves partial sums, which tree_combine_kernel merges in a fixed order.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_tc_ptx.cuh"

#include <atomic>
#include <cstring>
#include <type_traits>

namespace kda {
namespace {

using namespace tc;

constexpr int TL = 512, TK = 576, KB = TK / 64;
constexpr int TILE = 256;            // positions of a tile
constexpr int RC = 64;               // query rows of a CTA (a pair: 128)
constexpr int NS = 4, NZ = 3;        // slots of the score and value operands' rings
constexpr uint32_t SLOT = 16384;
constexpr uint32_t OFF_Q = 0;                        // [KB][64 rows][128 B]
constexpr uint32_t OFF_P = KB * RC * 128;            // [4][64 rows][128 B]: 64 positions each
constexpr uint32_t OFF_S = OFF_P + 4 * RC * 128;     // score blocks [128 positions][128 B]
constexpr uint32_t OFF_Z = OFF_S + NS * SLOT;        // value chunks [2][64 positions][128 B]
constexpr uint32_t SMEM = OFF_Z + NZ * SLOT + 1024;
constexpr uint32_t TM_Z = 0, TM_S = 256;  // Z: two products of 128 columns; S: two buffers of 128
// warps 0-7 softmax and output, 8 and 9 load score blocks and value chunks, 10 loads the queries
// and looks over a sequence's last chunks, 11 arrives for the softmax warps of a CTA without rows, 12
// and 13 issue the score and the value products
constexpr int W_LOAD_S = 8, W_LOAD_Z = 9, W_HELP = 10, W_TELL = 11, W_SCORE = 12, W_VALUE = 13, NT = 448;
constexpr int MAX_CLUSTERS = 80;     // of two CTAs (152 SMs: 76)
constexpr float LAZY = 8.f;          // log2 of how far a row's scores may rise above its reference

// barriers; L: the leading CTA's are used by both
enum {
  B_FULL_S = 0,                 // L  a slot's data is there in both CTAs
  B_FULL_Z = B_FULL_S + NS,     // L
  B_EMPTY_S = B_FULL_Z + NZ,    //    the products have read a slot
  B_EMPTY_Z = B_EMPTY_S + NS,
  B_QFULL = B_EMPTY_Z + NZ, B_QEMPTY,  // L, -: the queries
  B_SFULL,                  //    a score buffer is written (two)
  B_SFREE = B_SFULL + 2,    // L  and read (two)
  B_SCALED = B_SFREE + 2,   // L  Z is scaled to a tile's reference
  B_PFULL,                  // L  64 positions' weights are written (four)
  B_PFREE = B_PFULL + 4,    //    and read (four)
  B_ZFULL = B_PFREE + 4,    //    a tile's value product is done
  B_ZFREE,                  // L  the output has read Z
  B_TAIL,                   //    a value slot that threads have to look over has landed
  B_DRAIN = B_TAIL + NZ, B_N = B_DRAIN + 2
};

struct TreeMaps {
  CUtensorMap q, c, z, part;
};
// What the clusters leave for the combine kernel: partial sums [2 x clusters][128][512], their
// (reference, normaliser) [..][128][2], and for every cluster the row tile that its run begins inside.
struct Merge {
  int row0, rows;           // the row tile (0 rows: the run begins with one)
  int first, last;          // workers that hold parts of it
  int group, pad[3];
};

__device__ __forceinline__ bool elect() {  // one lane of the (whole) warp
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float ex2(float x) {  // 2^x, relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc));
}
// arrive on this barrier in both CTAs once the products issued so far are done
__device__ __forceinline__ void commit2(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// tile load into this CTA, completing on a barrier of the pair (shared::cluster address)
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// the same with an L2 eviction policy
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
// Arrive n times on a barrier of the pair (shared::cluster address).  What a thread wrote before is
// in its own SM's shared and tensor memory, where the products read it: a CTA-scope release is
// enough (a cluster-scope one costs the thread a fence of about a thousand cycles).
__device__ __forceinline__ void arrive_pair(uint32_t cluster_bar, uint32_t n = 1) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(n) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// the stores before the last one have read their shared memory
__device__ __forceinline__ void bulk_wait_read1() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// A sequence as the kernel sees it: rows of its nodes, visible positions, tiles.
struct Seq {
  int lo, W, len, end, tiles, row_tiles;
};
__device__ __forceinline__ Seq seq_of(const TreeAttnArgs &a, int n, bool tell) {
  Seq s;
  s.lo = a.cu_nodes[n];
  const int hi = a.cu_nodes[n + 1];
  s.W = hi - s.lo;
  if (s.lo < 0 || hi < s.lo || hi > a.total || s.W > 64) {
    if (tell && a.err) atomicOr(a.err, ERR_BAD_SEQLEN);
    s.W = 0;
  }
  s.len = a.c.lengths[n];
  if (s.W > 0 && (s.len < 0 || (int64_t)s.len + s.W > (int64_t)a.c.max_pages * a.c.page_size)) {
    if (tell && a.err) atomicOr(a.err, ERR_BAD_INDEX);
    s.len = s.end = 0;  // nothing visible
  } else {
    s.end = s.len + s.W;
  }
  s.tiles = s.W > 0 ? (s.end > 0 ? (s.end - 1) / TILE + 1 : 1) : 0;
  s.row_tiles = (s.W * a.H + 2 * RC - 1) / (2 * RC);
  return s;
}

// This cluster's run of tiles, cut at the sequences' ends; every warp role walks it on its own.
struct Walk {
  int n, off;    // place in sequence n's (pass, tile) order (at most 2^26 tiles)
  int64_t left;  // tiles left
  int log_group, member;
  Seq s;
  int rt, t0, t1;     // the current segment: row tile, tiles t0 .. t1 - 1
  __device__ __forceinline__ bool next(const TreeAttnArgs &a) {
    while (left > 0) {
      s = seq_of(a, n, false);
      if (off >= ((s.row_tiles + (1 << log_group) - 1) >> log_group) * s.tiles) {
        ++n;
        off = 0;
        continue;
      }
      const int pass = off / s.tiles;
      t0 = off - pass * s.tiles;
      rt = (pass << log_group) + member;
      t1 = s.tiles - t0 < left ? s.tiles : t0 + (int)left;
      off += t1 - t0;
      left -= t1 - t0;
      if (rt < s.row_tiles) return true;
    }
    return false;
  }
};

// The first tile of worker w's run (a 64-bit division costs hundreds of cycles: only where needed).
__device__ __forceinline__ int64_t run_start(int64_t tiles, int w, int workers) {
  return tiles < (1 << 24) ? (int64_t)((uint32_t)tiles * (uint32_t)w / (uint32_t)workers) : tiles * w / workers;
}
// The worker whose run holds tile t: the last that starts at or before it.
__device__ __forceinline__ int worker_of(int64_t tiles, int64_t t, int workers) {
  const int64_t x = (t + 1) * workers - 1;
  return ((x | tiles) >> 32) == 0 ? (int)((uint32_t)x / (uint32_t)tiles) : (int)(x / tiles);
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NT, 1)
    tree_attn_kernel(const TreeAttnArgs a, const __grid_constant__ TreeMaps maps, float *part, float *part_ml,
                     Merge *merge) {
  extern __shared__ uint8_t dyn[];
  __shared__ __align__(8) uint64_t s_bar[B_N];
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_abort;
  __shared__ unsigned long long s_cost[4];
  __shared__ uint32_t s_scan[NT / 32];
  __shared__ int s_n, s_off, s_page[2][16];
  __shared__ float s_max[2][4][RC], s_sum[4][RC];
  const uint32_t raw = smem_u32(dyn);
  const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
  uint8_t *sm = dyn + pad;
  const uint32_t sb = raw + pad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int cid = blockIdx.x >> 1, clusters = gridDim.x >> 1;
  auto bar = [&](int i) { return smem_u32(&s_bar[i]); };
  if (tid < B_N) {
    const int i = tid;
    int n = 1;
    if (i < B_EMPTY_S || i == B_QFULL) n = 2;                                        // a loader of each CTA
    if (i == B_SFREE || i == B_SFREE + 1 || i == B_SCALED || i == B_ZFREE) n = 16;  // the softmax warps
    if (i >= B_PFULL && i < B_PFREE) n = 4;                                         // two of each CTA
    mbar_init(bar(i), n);
    mbar_fence_init();
  }
  if (tid == 64) s_abort = 0, s_n = 0, s_off = 0;
  if (tid >= 96 && tid < 100) s_cost[tid - 96] = 0;
  if (tid >= 128 && tid < 132)
    asm volatile("prefetch.tensormap [%0];" ::"l"(&maps.q + (tid - 128)) : "memory");
  if (warp == W_SCORE) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  // launched while the kernel before runs out: nothing of global memory is read or written above
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Seq mine = {};
  if (tid < a.n_seqs) mine = seq_of(a, tid, blockIdx.x == 0);
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // barriers and tensor memory are there in this CTA; waited for below

  // ---- the batch's tiles for groups of 1, 2, 4 and 8 clusters, and this cluster's run ----------
  for (int n0 = 0; n0 < a.n_seqs; n0 += NT) {
    Seq s = mine;
    if (n0 > 0) {
      s.row_tiles = s.tiles = 0;
      if (n0 + tid < a.n_seqs) s = seq_of(a, n0 + tid, blockIdx.x == 0);
    }
#pragma unroll 1  // (run once: its instructions come from L2, so few of them)
    for (int g = 0; g < 4; ++g) {  // at most 64 x 2^20 tiles each: a warp's sum fits 32 bits
      const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)((s.row_tiles + (1 << g) - 1) >> g) * (uint32_t)s.tiles);
      if (lane == 0 && c) atomicAdd(&s_cost[g], (unsigned long long)c);
    }
  }
  __syncthreads();
  // The group whose run takes the least time.  A larger one idles where row tiles do not divide by
  // it, but its clusters' tiles take less: they share HBM's reads (measured: 0.86 to 0.96 of a lone
  // cluster's time for two, 0.73 to 0.83 for four; 64 sequences x 6 to 8 nodes x 4096: 190 us alone, 193 in
  // twos, 165 in fours; 100 x 3 to 4 nodes: 169, 148, 235; 100 x 4 to 5 nodes: 204, 228, 241).
  int log_group = lane & 3;
  {
    float cost = (clusters >> log_group)
                     ? __fdividef((float)s_cost[log_group] * (log_group == 0 ? 1.f : log_group == 1 ? 0.93f : 0.82f),
                                  (float)(clusters >> log_group))
                     : INFINITY;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float c = __shfl_xor_sync(0xffffffffu, cost, o);
      const int g = __shfl_xor_sync(0xffffffffu, log_group, o);
      if (c < cost || (c == cost && g > log_group)) cost = c, log_group = g;
    }
  }
  const int group = 1 << log_group;
  const int64_t tiles = (int64_t)s_cost[log_group];
  // every worker has a run
  const int workers = tiles < (clusters >> log_group) ? (int)tiles : clusters >> log_group;
  const int worker = cid >> log_group, member = cid & (group - 1);
  int64_t begin = 0, stop = 0;
  if (worker < workers) {
    const int64_t x = run_start(tiles, worker + (lane & 1), workers);
    begin = __shfl_sync(0xffffffffu, x, 0), stop = __shfl_sync(0xffffffffu, x, 1);
  }
  if (stop > begin) {  // the sequence that tile `begin` falls in
    int64_t before = 0;
    for (int n0 = 0; n0 < a.n_seqs && before <= begin; n0 += NT) {
      uint32_t cost = 0;
      Seq s = mine;
      if (n0 + tid < a.n_seqs) {
        if (n0 > 0) s = seq_of(a, n0 + tid, false);
        cost = (uint32_t)((s.row_tiles + group - 1) >> log_group) * (uint32_t)s.tiles;
      }
      uint32_t x = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_scan[warp] = x;
      __syncthreads();
      const uint32_t v = lane < NT / 32 ? s_scan[lane] : 0, v0 = lane < warp ? v : 0;  // sums in two halves: past 32 bits
      const int64_t at = before + __reduce_add_sync(0xffffffffu, v0 & 0xffff) +
                         ((int64_t)__reduce_add_sync(0xffffffffu, v0 >> 16) << 16) + (x - cost);
      if (at <= begin && begin < at + cost) {
        const int off = (int)(begin - at);
        s_n = n0 + tid, s_off = off;
        if (rank == 0) {  // what the combine kernel merges with this worker's blocks
          const int t0 = off % s.tiles, left = s.W * a.H - 2 * RC * (off / s.tiles * group + member);
          Merge g;
          g.group = group;
          g.first = worker_of(tiles, begin - t0, workers), g.last = worker_of(tiles, begin - t0 + s.tiles - 1, workers);
          g.row0 = (s.lo + s.W) * a.H - left;
          g.rows = t0 == 0 || left <= 0 ? 0 : left < 2 * RC ? left : 2 * RC;
          merge[cid] = g;
        }
      }
      before += __reduce_add_sync(0xffffffffu, v & 0xffff) + ((int64_t)__reduce_add_sync(0xffffffffu, v >> 16) << 16);
      __syncthreads();
    }
  }
  if (stop <= begin && rank == 0 && tid == 0) merge[cid].rows = 0;
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tm = s_tmem;
  Walk walk;
  walk.n = s_n, walk.off = s_off, walk.left = stop - begin, walk.log_group = log_group, walk.member = member;
  // A wait that runs out raises s_abort; from then on waits fail at once.  The softmax and load
  // warps then walk on to the end without waiting (they meet on named barriers, which all of them
  // have to reach), and the loader issues nothing more.
  auto wait = [&](int i, uint32_t parity) {
#pragma unroll 1
    for (long it = 0; it < kWaitLimit; ++it) {
      if (mbar_try_wait(bar(i), parity & 1)) return true;
      if (s_abort) return false;
    }
    s_abort = 1;
    return false;
  };
  const int box = a.c.page_size < 64 ? a.c.page_size : 64;  // rows of a tile load

  auto warp_wait = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, wait(i, parity)) != 0; };

  if (warp == W_LOAD_S || warp == W_LOAD_Z) {
    // ---- the rings, a tile at a time; one thread loads, s_page[which][e] is the page of the
    //      positions 256 t + e box ..
    const bool scores = warp == W_LOAD_S;
    const int which = scores ? 0 : 1, full = scores ? B_FULL_S : B_FULL_Z, empty = scores ? B_EMPTY_S : B_EMPTY_Z;
    const int slots = scores ? NS : NZ;
    const uint32_t full0 = map_shared_rank(bar(full), 0), tail0 = map_shared_rank(bar(B_TAIL), rank);
    const uint32_t ring = sb + (scores ? OFF_S : OFF_Z);
    // A lone cluster reads a position's row twice, its scores' loads and one or two tiles later its
    // values'; then L2 may drop it.  (By default L2 kept rows that were done with: 1.35 GB came from
    // HBM for 0.95 GB of cache at 256 sequences x 1 node, 252 us; so, 212.)  In a group the others
    // still need it.
    uint64_t policy;
    if (group > 1) asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    else if (scores) asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
    else asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    const int lb = 31 - __clz(box), lp = 31 - __clz(a.c.page_size), in_page = a.c.page_size - 1;
    const int per = 64 >> lb;  // tile loads of 64 positions
    int j = 0;                 // the next slot
    uint32_t par = 1;          // parity that its last use ends (a fresh barrier counts as ended)
    auto step = [&]() {
      if (++j == slots) j = 0, par ^= 1;
    };
    // the leading CTA's barrier expects both CTAs' bytes; the other CTA only arrives (its bytes
    // cannot come before the phase they belong to: its slot was freed by that phase's products)
    auto announce = [&]() {
      if (rank == 0) mbar_expect_tx(bar(full + j), 2 * SLOT);
      else arrive_pair(full0 + 8 * j);
    };
    int limit = 0;  // tiles that begin before it have a position for this lane to look up
    auto lookup = [&](int t) {
      return TILE * t < limit ? a.c.table[(size_t)walk.n * a.c.max_pages + ((TILE * t + lane * box) >> lp)] : -2;
    };
    while (walk.next(a)) {
      limit = lane * box < TILE ? walk.s.end - lane * box : 0;
      int ahead = lookup(walk.t0);
      for (int t = walk.t0; t < walk.t1; ++t) {
        const int page = ahead;
        if (t + 1 < walk.t1) ahead = lookup(t + 1);
        if (scores && (page < 0 || page >= a.c.n_pages) && TILE * t < limit && a.err) atomicOr(a.err, ERR_BAD_INDEX);
        // no page, or behind the last node: past the pool, where loads give zeros
        if (lane < 16) s_page[which][lane] = page >= 0 && page < a.c.n_pages ? page : a.c.n_pages;
        __syncwarp();
        if (elect()) {
          const int p0 = TILE * t;
          // a tile's loads, 64 positions in PER boxes
          auto load = [&](auto PER) {
            constexpr int per = decltype(PER)::value, rows = 64 / per;
            if (scores) {
              const int e0 = 2 * per * (int)rank;
              int page[2 * per];
#pragma unroll
              for (int y = 0; y < 2 * per; ++y) page[y] = s_page[0][e0 + y];
#pragma unroll 1
              for (int kb = 0; kb < KB; ++kb) {
                if (wait(empty + j, par)) {
                  announce();
#pragma unroll
                  for (int y = 0; y < 2 * per; ++y)
                    tma_pair_3d(ring + j * SLOT + y * rows * 128, &maps.c, 64 * kb,
                                per == 1 ? (p0 + 64 * (e0 + y)) & in_page : 0, page[y], full0 + 8 * j, policy);
                }
                step();
              }
            } else {
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                const int g0 = p0 + 64 * (c >> 1), e0 = per * (c >> 1), ch = 256 * (int)rank + 128 * (c & 1);
                const bool tail = g0 + 64 > walk.s.len && g0 < walk.s.end;  // warp 10 looks it over
                if (wait(empty + j, par)) {
                  if (!tail) announce();
                  else mbar_expect_tx(bar(B_TAIL + j), SLOT);
                  const uint32_t done = (tail ? tail0 : full0) + 8 * j;
                  const int row = per == 1 ? g0 & in_page : 0;
#pragma unroll
                  for (int y = 0; y < per; ++y) {
                    const int page = s_page[1][e0 + y];
                    tma_pair_3d(ring + j * SLOT + y * rows * 128, &maps.c, ch, row, page, done, policy);
                    tma_pair_3d(ring + j * SLOT + 8192 + y * rows * 128, &maps.c, ch + 64, row, page, done, policy);
                  }
                }
                step();
              }
            }
          };
          if (per == 1) load(std::integral_constant<int, 1>{});
          else if (per == 2) load(std::integral_constant<int, 2>{});
          else load(std::integral_constant<int, 4>{});
        } else {
          for (int y = 0; y < (scores ? KB : 8); ++y) step();
        }
        __syncwarp();
      }
    }
    // every slot read before the CTA may end
    for (int y = 0; y < slots; ++y) {
      wait(empty + j, par);
      step();
    }
    if (s_abort)  // a wait ran out: let the copies in flight land
      for (int y = 0; y < 100; ++y) __nanosleep(10000);
  } else if (warp == W_HELP) {
    // ---- the queries of a segment, and the chunks of Z's operand that reach past the cached
    //      positions: rows behind the last drafted node and drafted rows with a value that is not
    //      finite become zeros there before the products may use them (their weight is 0 or NaN,
    //      and 0 x NaN must not reach the rows that do not see them).  In short contexts every other
    //      tile waits for this: eight rows' reads at a time (two took 194 us for 155 sequences x 25 nodes
    //      x 32 heads, 526 positions, now 173).
    const uint32_t qfull0 = map_shared_rank(bar(B_QFULL), 0);
    int segs = 0, j0 = 0;      // the tile's first value slot
    uint32_t looked = 0;       // parity of B_TAIL + j
    int len1 = -1, end1 = 0, t1 = 0;
    auto look = [&](int len, int end, int t) {
      const int first = j0;
      j0 = (j0 + 8) % NZ;
      if (TILE * (t + 1) <= len) return;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        const int g0 = TILE * t + 64 * (c >> 1), j = (first + c) % NZ;
        if (g0 + 64 <= len || g0 >= end) continue;
        const bool ok = warp_wait(B_TAIL + j, (looked >> j) & 1);
        looked ^= 1u << j;
        uint8_t *slot = sm + OFF_Z + j * SLOT;
        const int piece = lane & 15, half = lane >> 4;  // 16 lanes a row
        uint8_t *column = slot + (piece >> 3) * 8192;
        auto place = [&](int r) { return reinterpret_cast<uint4 *>(column + r * 128 + (((piece & 7) ^ (r & 7)) << 4)); };
        auto odd = [](uint32_t u) { return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u; };
        const int first = len > g0 ? len - g0 : 0, stop = end - g0 < 64 ? end - g0 : 64;  // drafted rows
        const uint32_t row_lanes = lane < 16 ? 0xffffu : 0xffff0000u;
        for (int r0 = first; r0 < stop; r0 += 8) {  // eight of them at a time
          uint4 v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) v[y] = *place((r0 + 2 * y + half) & 63);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = r0 + 2 * y + half;
            const bool bad = odd(v[y].x) || odd(v[y].y) || odd(v[y].z) || odd(v[y].w);
            if ((__ballot_sync(0xffffffffu, bad) & row_lanes) && r < stop) *place(r) = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll 4
        for (int r = stop + half; r < 64; r += 2) *place(r) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && ok) arrive_pair(map_shared_rank(bar(B_FULL_Z + j), 0));
      }
    };
    while (walk.next(a)) {
      if (segs == 0 || warp_wait(B_QEMPTY, (uint32_t)(segs - 1))) {
        const int64_t row = (int64_t)walk.s.lo * a.H + 2 * RC * walk.rt + RC * (int)rank;
        const int rows = a.total * a.H < RC ? (int)(a.total * a.H) : RC;  // of a box
        if (lane == 0) {
          if (rank == 0) mbar_expect_tx(bar(B_QFULL), 2 * KB * rows * 128);
          else arrive_pair(qfull0);
        }
        __syncwarp();
        if (lane < KB) tma_pair_3d(sb + OFF_Q + lane * RC * 128, &maps.q, 64 * lane, (int)row, 0, qfull0);
      }
      ++segs;
      for (int t = walk.t0; t < walk.t1; ++t) {
        if (len1 >= 0) look(len1, end1, t1);  // a tile late: a segment's queries go first
        len1 = walk.s.len, end1 = walk.s.end, t1 = t;
      }
    }
    if (len1 >= 0) look(len1, end1, t1);
    if (segs > 0) wait(B_QEMPTY, (uint32_t)(segs - 1));
  } else if (warp == W_SCORE) {
    // ---- score products (one thread of the leading CTA) ---------------------------------------
    if (rank == 0 && elect()) {
      constexpr uint32_t ID_S = idesc(1, 128, 256, 0, 0);
      int segs = 0, i = 0, j = 0;
      uint32_t par = 0;
      bool ok = true;
      while (ok && walk.next(a)) {
        for (int t = walk.t0; t < walk.t1 && ok; ++t, ++i) {
          if (t == walk.t0 && !(ok = wait(B_QFULL, (uint32_t)segs))) break;
          // this buffer's scores (tile i - 2) are read
          if (i >= 2 && !(ok = wait(B_SFREE + (i & 1), (uint32_t)((i >> 1) - 1)))) break;
          tc_fence_after();
          const uint32_t d = tm + TM_S + 128 * (i & 1);
#pragma unroll 1
          for (int kb = 0; kb < KB; ++kb) {
            if (!(ok = wait(B_FULL_S + j, par))) break;
            const uint64_t ad = sdesc_sw128(sb + OFF_Q + kb * RC * 128, 16, 1024);
            const uint64_t bd = sdesc_sw128(sb + OFF_S + j * SLOT, 16, 1024);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma2(d, ad + 2 * ks, bd + 2 * ks, ID_S, kb > 0 || ks > 0);
            commit2(bar(B_EMPTY_S + j));
            if (++j == NS) j = 0, par ^= 1;
          }
          if (!ok) break;
          commit2(bar(B_SFULL + (i & 1)));
          if (t == walk.t1 - 1) commit2(bar(B_QEMPTY));
        }
        ++segs;
      }
      if (!ok) {  // a wait ran out: let the products in flight end
        commit2(bar(B_DRAIN));
        mbar_wait(bar(B_DRAIN), 0);
      }
    }
  } else if (warp == W_VALUE) {
    // ---- value products (one thread of the leading CTA) ---------------------------------------
    if (rank == 0 && elect()) {
      constexpr uint32_t ID_Z = idesc(1, 128, 256, 0, 1);
      int segs = 0, i = 0, j = 0;
      uint32_t par = 0;
      bool ok = true;
      while (ok && walk.next(a)) {
        for (int t = walk.t0; t < walk.t1 && ok; ++t, ++i) {
          const bool first = t == walk.t0;
          if (!(ok = wait(B_SCALED, (uint32_t)i))) break;
          if (first && segs > 0 && !(ok = wait(B_ZFREE, (uint32_t)(segs - 1)))) break;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {  // 64 positions, one half of the latents and then the other
            const int pc = c >> 1, h = c & 1;
            if (h == 0 && !(ok = wait(B_PFULL + pc, (uint32_t)i))) break;
            if (!(ok = wait(B_FULL_Z + j, par))) break;
            tc_fence_after();
            const uint64_t ad = sdesc_sw128(sb + OFF_P + pc * RC * 128, 16, 1024);
            const uint64_t bd = sdesc_sw128(sb + OFF_Z + j * SLOT, 8192, 1024);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma2(tm + TM_Z + 128 * h, ad + 2 * ks, bd + 128 * ks, ID_Z, !(first && pc == 0 && ks == 0));
            commit2(bar(B_EMPTY_Z + j));
            if (h == 1) commit2(bar(B_PFREE + pc));
            if (++j == NZ) j = 0, par ^= 1;
          }
          if (!ok) break;
          commit2(bar(B_ZFULL));
        }
        ++segs;
      }
      if (!ok) {
        commit2(bar(B_DRAIN + 1));
        mbar_wait(bar(B_DRAIN + 1), 0);
      }
    }
  } else if (warp == W_TELL) {
    // ---- the softmax warps' arrivals where this CTA has no rows (the upper half of a row tile)
    int i = 0;
    const uint32_t lead = map_shared_rank(bar(0), 0);
    while (walk.next(a)) {
      if (walk.s.W * a.H <= 2 * RC * walk.rt + RC * (int)rank) {
        for (int t = walk.t0; t < walk.t1; ++t, ++i) {
          wait(B_SFULL + (i & 1), (uint32_t)(i >> 1));
          if (lane == 0) arrive_pair(lead + 8 * (B_SFREE + (i & 1)), 8);
          for (int q = 0; q < 4; ++q) {
            if (i > 0) wait(B_PFREE + q, (uint32_t)(i - 1));
            if (lane == 0 && q == 0) arrive_pair(lead + 8 * B_SCALED, 8);
            if (lane == 0) arrive_pair(lead + 8 * (B_PFULL + q), 2);
          }
          __syncwarp();
        }
        wait(B_ZFULL, (uint32_t)(i - 1));
        if (lane == 0) arrive_pair(lead + 8 * B_ZFREE, 8);
      } else {
        i += walk.t1 - walk.t0;
      }
      // in step with the softmax warps: a barrier's phases are told apart by parity only
      bar_sync(2, 288);
    }
  } else {
    // ---- softmax and output: TMEM lane l of S and Z is row l % 64; lanes 64-127 hold the upper
    //      128 positions of S and the upper 256 latents of Z.  Warp w reads lanes 32 (w & 3) ..,
    //      and of their 128 columns (positions; of Z's two products the one) half w >> 2.
    const int qw = warp & 3, hf = warp >> 2, ph = qw >> 1;
    const int row = (32 * qw + lane) & 63, quarter = 2 * ph + hf;  // this thread's 64 positions of a tile
    const uint32_t lanes = (uint32_t)(32 * qw) << 16;
    const int lp = 31 - __clz(a.c.page_size);
    const uint32_t lead = map_shared_rank(bar(0), 0);
    const uint32_t prow = sb + OFF_P + quarter * RC * 128 + row * 128;
    int i = 0;
    while (walk.next(a)) {
      const int r0 = 2 * RC * walk.rt + RC * (int)rank;  // this CTA's first row of the sequence
      const int rows = walk.s.W * a.H - r0;              // and how many are there (may be <= 0)
      const Seq s = walk.s;
      unsigned long long seen = 0;
      if (row < rows) {
        const int node = (r0 + row) / a.H;
        seen = a.mask ? (unsigned long long)a.mask[s.lo + node] : (2ull << node) - 1;
        if (s.W < 64) seen &= (1ull << s.W) - 1;
        if (s.end == 0) seen = 0;  // a bad length: nothing is there
      }
      float ref = -INFINITY, sum = 0.f;
      if (rows <= 0) i += walk.t1 - walk.t0;  // a row tile of one CTA: this one's products are not used
      for (int t = walk.t0; t < walk.t1 && rows > 0; ++t, ++i) {
        const int buf = i & 1;
        const int p0 = TILE * t + 64 * quarter;  // this thread's first position
        // the visible ones of its 64 positions, as bits
        unsigned long long vis = ~0ull;
        if (p0 + 64 > s.len) {
          const int d = s.len - p0;  // cached ones among them
          vis = d >= 0 ? (((1ull << d) - 1) | (seen << d)) : (d > -64 ? seen >> -d : 0ull);
        }
        for (int x = 0; x < 64; x += box) {
          if (p0 + x >= s.end) break;
          const int p = a.c.table[(size_t)walk.n * a.c.max_pages + ((p0 + x) >> lp)];
          if (__builtin_expect(p < 0 || p >= a.c.n_pages, 0)) vis &= ~((box == 64 ? ~0ull : ((1ull << box) - 1)) << x);
        }
        wait(B_SFULL + buf, (uint32_t)(i >> 1));
        tc_fence_after();
        float v[64];
        {
          float x[32], y[32];
          tmem_ld32(tm + lanes + TM_S + 128 * buf + 64 * hf, x);
          tmem_ld32(tm + lanes + TM_S + 128 * buf + 64 * hf + 32, y);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = x[c], v[32 + c] = y[c];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(lead + 8 * (B_SFREE + buf));
        if (vis != ~0ull) {
#pragma unroll
          for (int c = 0; c < 64; ++c) v[c] = (vis >> c) & 1 ? v[c] : -INFINITY;
        }
        float m = fmaxf(v[0], v[1]);
#pragma unroll
        for (int c = 2; c < 64; c += 2) m = fmaxf(m, fmaxf(v[c], v[c + 1]));
        s_max[buf][quarter][row] = m;  // two buffers: this barrier is a tile's only one
        bar_sync(1, 256);
        m = fmaxf(fmaxf(s_max[buf][0][row], s_max[buf][1][row]), fmaxf(s_max[buf][2][row], s_max[buf][3][row])) *
            a.scale_log2;
        // the reference follows the maximum only when it is passed by 2^8: the weights keep their
        // relative precision up to there, and Z is rescaled seldom
        float al = 1.f;
        if (m > ref + LAZY || ref == -INFINITY) {
          al = ref == -INFINITY ? 1.f : ex2(ref - m);
          ref = m;
        }
        const float base = ref == -INFINITY ? 0.f : ref;
        float ls = 0.f;
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float e0 = ex2(fmaf(v[2 * c], a.scale_log2, -base)), e1 = ex2(fmaf(v[2 * c + 1], a.scale_log2, -base));
          const __nv_bfloat162 b = __floats2bfloat162_rn(e0, e1);
          w[c] = *reinterpret_cast<const uint32_t *>(&b);
          // weights are rounded to bf16, the product's operands (two parts each would double its time): 2^-8 of a
          // weight at most, which averages out over the positions (a bf16 z is 1.7e-3 to 2.0e-3 off in RMS, where
          // its own rounding is 1.7e-3).  The normaliser sums the weights that the product uses: they add up to one.
          ls += __uint_as_float(w[c] << 16) + __uint_as_float(w[c] & 0xffff0000u);
        }
        sum = sum * al + ls;
        // the last tile's first products are done, so both CTAs have scaled Z for it: this tile's turn
        if (i > 0) wait(B_PFREE, (uint32_t)(i - 1));
        if (__any_sync(0xffffffffu, al != 1.f)) {
          wait(B_ZFULL, (uint32_t)(i - 1));
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float z[32];
            const uint32_t at = tm + lanes + TM_Z + 128 * hf + 32 * c;
            tmem_ld32(at, z);
            tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 32; ++y) z[y] *= al;
            tmem_st32(at, z);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
        }
        if (lane == 0) arrive_pair(lead + 8 * B_SCALED);
        if (i > 0) wait(B_PFREE + quarter, (uint32_t)(i - 1));  // the last tile's weights are read
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(prow + ((c ^ (row & 7)) << 4)), "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3]) : "memory");
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_pair(lead + 8 * (B_PFULL + quarter));
      }
      // the segment's output
      const bool whole = walk.t0 == 0 && walk.t1 == s.tiles;
      const int slot = 2 * cid + (walk.t0 == 0 ? 1 : 0);
      if (rows > 0) {
        wait(B_ZFULL, (uint32_t)(i - 1));
        s_sum[quarter][row] = sum;
        bar_sync(1, 256);
        const float l = (s_sum[0][row] + s_sum[1][row]) + (s_sum[2][row] + s_sum[3][row]);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        tc_fence_after();
        // the warp's [32 rows][128 latents], 64 bytes of each row at a time: through shared memory
        // (the weights' place, free now) in two buffers, from where tile stores take them; threads
        // where a store would pass the sequence's last row
        uint8_t *stage = sm + OFF_P + warp * 4096;
        const bool bits = whole && a.z_bf16;
        const int col0 = 256 * ph + 128 * hf, first = 32 * (qw & 1);  // of the warp: latents, rows
        const int width = bits ? 2 : 4, cols = 64 / width;
        const bool by_tile = !whole || first + 32 <= rows;
        const int64_t row0 = whole ? (int64_t)s.lo * a.H + r0 + first : (int64_t)slot * 2 * RC + RC * rank + first;
        const CUtensorMap *map = whole ? &maps.z : &maps.part;
        auto put = [&](int half, int c, const uint4 (&v)[4]) {
          if (lane == 0) bulk_wait_read1();
          __syncwarp();
          uint8_t *buf = stage + 2048 * half;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            *reinterpret_cast<uint4 *>(buf + lane * 64 + ((x ^ (lane >> 1 & 3)) << 4)) = v[x];
          if (by_tile) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(map, col0 + c, (int)row0, 0, smem_u32(buf));
              bulk_commit();
            }
          } else {
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = 8 * x + (lane >> 2), piece = lane & 3;
              const uint4 y = *reinterpret_cast<const uint4 *>(buf + r * 64 + ((piece ^ (r >> 1 & 3)) << 4));
              if (first + r < rows)
                *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(a.z) + ((row0 + r) * TL + col0 + c) * width + 16 * piece) = y;
            }
          }
        };
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          float z[32];
          tmem_ld32(tm + lanes + TM_Z + 128 * hf + c, z);
          tmem_wait_ld();
          if (bits) {
            auto pack = [&](float lo, float hi) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(lo * inv, hi * inv);
              return *reinterpret_cast<const uint32_t *>(&b);
            };
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              v[x] = make_uint4(pack(z[8 * x], z[8 * x + 1]), pack(z[8 * x + 2], z[8 * x + 3]),
                                pack(z[8 * x + 4], z[8 * x + 5]), pack(z[8 * x + 6], z[8 * x + 7]));
            put(c >> 5 & 1, c, v);
          } else {
            const float f = whole ? inv : 1.f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint4 v[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                v[x] = make_uint4(__float_as_uint(z[16 * y + 4 * x] * f), __float_as_uint(z[16 * y + 4 * x + 1] * f),
                                  __float_as_uint(z[16 * y + 4 * x + 2] * f), __float_as_uint(z[16 * y + 4 * x + 3] * f));
              put(y, c + cols * y, v);
            }
          }
        }
        if (!whole && quarter == 0) {
          float *ml = part_ml + ((size_t)slot * 2 * RC + RC * rank + row) * 2;
          ml[0] = ref;
          ml[1] = l;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_pair(lead + 8 * B_ZFREE);
          bulk_wait_read0();  // the weights' place is free again
        }
      }
      bar_sync(2, 288);  // (see warp 11)
    }
    if (lane == 0) bulk_wait0();
  }
  if (lane == 0 && s_abort && a.err) atomicOr(a.err, ERR_MBAR_TIMEOUT);
  __syncwarp();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == W_SCORE)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512u));
}

// z = sum_w 2^(m_w - M) Z_w / sum_w 2^(m_w - M) l_w over the workers w that hold parts of a row.  The blocks
// of all workers but the first share a row tile's rows: with two workers a warp merges a row, with more
// (a long sequence alone is cut into as many parts as there are workers) two to eight warps take a row's
// parts in turn and add up in a fixed order (one sequence x 4 nodes x 16384 positions, 64 parts: 41 us
// for both kernels with a warp a row by the last worker's blocks, 29 so; one x 1 x 65536 59 and 36).
constexpr int CNT = 256, CW = CNT / 32, CY = 2 * RC / CW;
__global__ void __launch_bounds__(CNT) tree_combine_kernel(const TreeAttnArgs a, const float *part, const float *part_ml,
                                                           const Merge *merge) {
  __shared__ __align__(16) float s_z[CW][TL];
  __shared__ float s_l[CW];
  // launched while the attention kernel runs out: its results are there once this returns
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
  const Merge g = merge[blockIdx.x];
  if (g.rows == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = g.first, last = g.last;
  const int log_group = 31 - __clz(g.group), member = blockIdx.x & (g.group - 1);
  const int sharers = last - first, mine = ((int)blockIdx.x >> log_group) - first - 1;
  const int log_k = sharers >= 8 ? 3 : sharers >= 4 ? 2 : sharers >= 2 ? 1 : 0, k = 1 << log_k;  // warps a row
  const int row = (((int)blockIdx.y * sharers + mine) << (3 - log_k)) + (warp >> log_k), slice = warp & (k - 1);
  float4 z[4] = {};
  float L = 0.f;
  if (row < g.rows) {
    // the first worker's part is the end of its run, the others' the beginning of theirs
    auto slot = [&](int w) { return (size_t)(2 * (w * g.group + member) + (w == first ? 1 : 0)) * 2 * RC + row; };
    float M = -INFINITY;
    for (int w = first + lane; w <= last; w += 32) M = fmaxf(M, part_ml[slot(w) * 2]);
    M = warp_max(M);
#pragma unroll 2
    for (int w = first + slice; w <= last; w += k) {
      const size_t s = slot(w);
      const float m = part_ml[s * 2], l = part_ml[s * 2 + 1];
      float4 x[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) x[y] = load4(part + s * TL + 128 * y + 4 * lane);
      const float f = m == -INFINITY ? (l == 0.f ? 0.f : l) : exp2f(m - M);  // l NaN: the row is NaN
      L = fmaf(f, l, L);
#pragma unroll
      for (int y = 0; y < 4; ++y)
        z[y].x = fmaf(f, x[y].x, z[y].x), z[y].y = fmaf(f, x[y].y, z[y].y), z[y].z = fmaf(f, x[y].z, z[y].z),
        z[y].w = fmaf(f, x[y].w, z[y].w);
    }
  }
  if (k > 1) {
    if (slice > 0) {
#pragma unroll
      for (int y = 0; y < 4; ++y) *reinterpret_cast<float4 *>(&s_z[warp][128 * y + 4 * lane]) = z[y];
      if (lane == 0) s_l[warp] = L;
    }
    __syncthreads();
    if (slice > 0) return;
    for (int w = warp + 1; w < warp + k; ++w) {
      L += s_l[w];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float4 x = *reinterpret_cast<const float4 *>(&s_z[w][128 * y + 4 * lane]);
        z[y].x += x.x, z[y].y += x.y, z[y].z += x.z, z[y].w += x.w;
      }
    }
  }
  if (row >= g.rows) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const float4 v = make_float4(z[y].x * inv, z[y].y * inv, z[y].z * inv, z[y].w * inv);
    const int64_t at = ((int64_t)g.row0 + row) * TL + 128 * y + 4 * lane;
    if (a.z_bf16) store4(reinterpret_cast<bf16 *>(a.z) + at, v);
    else store4(reinterpret_cast<float *>(a.z) + at, v);
  }
}

// [d2][d1][cols], the innermost contiguous, in boxes of box_cols x box_rows
bool tree_map(CUtensorMap *m, const void *ptr, bool bits, int cols, int64_t d1, int64_t d2, int box_cols, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const int width = bits ? 2 : 4;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)d1, (cuuint64_t)d2};
  cuuint64_t strides[2] = {(cuuint64_t)cols * width, (cuuint64_t)d1 * cols * width};
  cuuint32_t bx[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, es[3] = {1, 1, 1};
  return fn(m, bits ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(ptr), dims,
            strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            box_cols * width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t PART = (size_t)MAX_CLUSTERS * 2 * 2 * RC * TL * sizeof(float);
constexpr size_t PART_ML = (size_t)MAX_CLUSTERS * 2 * 2 * RC * 2 * sizeof(float);

}  // namespace

size_t mla_tree_ws_bytes(int, int64_t, int) { return PART + PART_ML + MAX_CLUSTERS * sizeof(Merge); }

cudaError_t launch_mla_tree(const TreeAttnArgs &a, int *launches, cudaStream_t s) {
  *launches = 0;
  TreeMaps maps;
  memset(&maps, 0, sizeof maps);
  const int64_t rows = a.total * a.H;
  const int box = a.c.page_size < 64 ? a.c.page_size : 64;
  if (!tree_map(&maps.q, a.q, true, TK, rows, 1, 64, rows < RC ? (int)rows : RC) ||
      !tree_map(&maps.c, a.c.pool, true, TK, a.c.page_size, a.c.n_pages, 64, box) ||
      !tree_map(&maps.z, a.z, a.z_bf16, TL, rows, 1, a.z_bf16 ? 32 : 16, rows < 32 ? (int)rows : 32) ||
      !tree_map(&maps.part, a.ws, false, TL, MAX_CLUSTERS * 2 * 2 * RC, 1, 16, 32))
    return cudaErrorInvalidValue;
  int dev = 0, nsm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  static std::atomic<int> sms[64];  // SMs of a device once the kernel is opted in there (idempotent if raced)
  if (dev < 64) nsm = sms[dev].load();
  if (nsm == 0) {
    e = cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) sms[dev].store(nsm);
  }
  const int clusters = nsm / 2 < 1 ? 1 : (nsm / 2 < MAX_CLUSTERS ? nsm / 2 : MAX_CLUSTERS);
  float *part = reinterpret_cast<float *>(a.ws);
  float *part_ml = reinterpret_cast<float *>(reinterpret_cast<char *>(a.ws) + PART);
  Merge *merge = reinterpret_cast<Merge *>(reinterpret_cast<char *>(a.ws) + PART + PART_ML);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;  // each launch overlaps the end of the kernel before
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early, cfg.numAttrs = 1, cfg.stream = s;
  cfg.gridDim = dim3(2 * clusters), cfg.blockDim = dim3(NT), cfg.dynamicSmemBytes = SMEM;
  e = cudaLaunchKernelEx(&cfg, tree_attn_kernel, a, maps, part, part_ml, merge);
  if (e != cudaSuccess) return e;
  ++*launches;
  cfg.gridDim = dim3(clusters, CY), cfg.blockDim = dim3(CNT), cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, tree_combine_kernel, a, (const float *)part, (const float *)part_ml, (const Merge *)merge);
  ++*launches;
  return e;
}

}  // namespace kda
