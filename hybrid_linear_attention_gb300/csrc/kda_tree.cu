// kda_tree.cu -- the KDA layer over a tree of drafted tokens: the outputs of every node, and the
// accepted path written into the state.
//
// Per head, node i of a sequence's tree has a parent p(i) < i (-1: it follows the sequence
// itself), and its state is the recurrence's ("Ling-3.1-flash: a 560B hybrid-attention MoE,
// counted from its safetensors headers", section "How KDA and MLA split the work", with the
// delta-rule write of "Ling-3.1-flash: Grouped Routing and Two Different MLA Caches", section
// "KDA replaces a token list with a recurrent matrix") applied to its parent's:
//     S_i = Diag(a_i) S_p(i) + k_i u_i^T,  u_i = beta_i (v_i - (Diag(a_i) S_p(i))^T k_i)
// Unrolled along the path from the pool state S, with G_i the sum of the log-retentions over
// the path of i and anc(i) its proper ancestors:
//     u_i = beta_i (v_i - S^T (k_i e^{G_i}) - sum_{j in anc(i)} A_ij u_j)
//     o_i = scale (S^T (q_i e^{G_i}) + sum_{j in anc(i) + i} B_ij u_j)
//     A_ij = sum_c k_ic k_jc e^{G_ic - G_jc},  B_ij = sum_c q_ic k_jc e^{G_ic - G_jc}
// so the 64 KB state of a (sequence, head) is read once for the whole tree and no node's state
// is ever stored; every exponent is a sum of log-retentions, at most 0.  A G behind a past that was
// forgotten is large (64 nodes at the clamp -5: 462 as a power of two), and the small retentions of later
// nodes would be rounded at its size and come out of G_i - G_j wrong (up to 1e-2 of an output with g_min
// near -88).  So G is kept as F - 16 - 32 N, F in fp32 within -16 .. 16 and N a whole number up to 255: a step
// is rounded by 2^-21 at most (half an fp32 step below 16), whatever lies before it, N_i - N_j is exact, and down
// to G = -32 N is 0.  Trees so small that G cannot pass -64 (at the clamp -5: up to 8 nodes) keep one fp32 sum
// G + 32, within -32 .. 32: 7 steps rounded by 2^-20 are no worse than 63 by 2^-21.  The accepted path is replayed
// afterwards (tree_accept_kernel), which reads and writes the state once.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "kda_tc_ptx.cuh"

#include <atomic>
#include <type_traits>

namespace kda {
namespace {

__device__ __forceinline__ void l2_prefetch(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// Launched while the kernel before runs out; waits here until that one is complete.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;" ::: "memory");
}

// 2^x, 1/x and the sigmoid on the special-function unit (relative errors about 2^-22)
__device__ __forceinline__ float ex2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_(float x) { return rcp_(1.f + ex2_(x * -LOG2E)); }
__device__ __forceinline__ float silu_(float x) { return x * sigmoid_(x); }

// fp32 -> tf32 (10 mantissa bits, to nearest), and the warp's 16 x 8 x 8 product
__device__ __forceinline__ uint32_t tf32_(float x) {
  uint32_t y;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_16x8x8(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same of bf16 operands, 16 x 8 x 16, two values a register
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two values as bf16 pairs hi + lo, good to about 2^-17 of each
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  const __nv_bfloat162 l =
      __floats2bfloat162_rn(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xffff0000u));
  lo = *reinterpret_cast<const uint32_t *>(&l);
}
// four 8 x 16-byte blocks: lane l gets the 32-bit word l % 4 of row l / 4 of each
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void *row) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"((uint32_t)__cvta_generic_to_shared(row)));
}

// The nodes of sequence n: first row and count; an offset pair that is out of range, runs
// backwards or holds more than `most` nodes is flagged and treated as empty.
__device__ __forceinline__ int tree_nodes(const TreeArgs &a, int n, int most, int &row0, bool tell) {
  const int lo = a.cu_nodes[n], hi = a.cu_nodes[n + 1];
  row0 = lo;
  if (lo < 0 || hi < lo || hi > a.total || hi - lo > most) {
    if (tell && a.err) atomicOr(a.err, ERR_BAD_SEQLEN);
    return 0;
  }
  return hi - lo;
}

// Raw input of a path position: node j's row for j >= 0, else the conv tail (j = -1 newest).
template <typename IO>
__device__ __forceinline__ const IO *tap_row(const TreeArgs &a, int row0, int slot, int j, size_t C) {
  return j >= 0 ? reinterpret_cast<const IO *>(a.x_raw) + (size_t)(row0 + j) * C
                : reinterpret_cast<const IO *>(a.conv_state) + ((size_t)slot * 3 + (3 + j)) * C;
}

// Four neighbouring channels' weights of the width-4 convolution, and its SiLU for taps t0 (oldest)
// to t3.
struct Conv4 {
  float4 a, b, c, d;
  template <typename IO>
  __device__ __forceinline__ void load(const IO *w, size_t ch) {
    a = load4(w + 4 * ch), b = load4(w + 4 * ch + 4), c = load4(w + 4 * ch + 8), d = load4(w + 4 * ch + 12);
  }
  __device__ __forceinline__ float4 operator()(float4 t0, float4 t1, float4 t2, float4 t3) const {
    return make_float4(silu_(fmaf(a.x, t0.x, fmaf(a.y, t1.x, fmaf(a.z, t2.x, a.w * t3.x)))),
                       silu_(fmaf(b.x, t0.y, fmaf(b.y, t1.y, fmaf(b.z, t2.y, b.w * t3.y)))),
                       silu_(fmaf(c.x, t0.z, fmaf(c.y, t1.z, fmaf(c.z, t2.z, c.w * t3.z)))),
                       silu_(fmaf(d.x, t0.w, fmaf(d.y, t1.w, fmaf(d.z, t2.w, d.w * t3.w)))));
  }
};

// `bytes` (a multiple of 16) from p on into L2, by one instruction
__device__ __forceinline__ void ask_bulk(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// What a CTA will read of heads h .. h + HEADS - 1 of `rows` nodes of sequence n, into L2: the raw
// inputs' streams FIRST .. 2, the retentions, the gates and the conv tail (a line or more a thread).
template <int D, typename IO, int HEADS, int FIRST>
__device__ __forceinline__ void ask_inputs(const TreeArgs &a, int row0, int rows, int slot, int h, int th, int nth) {
  const size_t C = (size_t)3 * a.H * D;
  constexpr int first = FIRST, xl = (HEADS * D * (int)sizeof(IO) + 127) / 128, gl = (HEADS * D * 4 + 127) / 128;  // lines
  constexpr int nx = (3 - FIRST) * xl, per = nx + gl + (FIRST == 0 ? xl : 0);
  const IO *x_raw = reinterpret_cast<const IO *>(a.x_raw);
  for (int x = th; x < rows * per + 3 * nx; x += nth) {
    const char *p;
    if (x < rows * per) {
      const int i = row0 + x / per, y = x % per;
      const size_t at = ((size_t)i * a.H + h) * D;
      if (y < nx) p = reinterpret_cast<const char *>(x_raw + (size_t)i * C + ((size_t)(first + y / xl) * a.H + h) * D) + y % xl * 128;
      else if (y < nx + gl) p = reinterpret_cast<const char *>(a.g + at) + (y - nx) * 128;
      else if (a.gate) p = reinterpret_cast<const char *>(reinterpret_cast<const IO *>(a.gate) + at) + (y - nx - gl) * 128;
      else continue;
    } else {
      const int y = x - rows * per;
      p = reinterpret_cast<const char *>(reinterpret_cast<const IO *>(a.conv_state) + ((size_t)slot * 3 + y / nx) * C +
                                         ((size_t)(first + y % nx / xl) * a.H + h) * D) + y % xl * 128;
    }
    l2_prefetch(p);
  }
}

// shared memory of the verify kernel for at most W nodes (floats): k over q [2 W][D + 4], v, F (then S^T k)
// [W][D] each, the taps [W][4] and, with G split, N (bytes) [W][D], then S^T q [W][D] and A and B of the pairs,
// which take the place of the raw inputs [W + 3][3 D] where those are staged (bf16); parents, first pairs [W + 1],
// strengths and norms [2 W]; the list of the pairs (node, itself or an ancestor), 16 bits each
__host__ __device__ constexpr size_t verify_pairs(int W) { return (size_t)W * (W + 1) / 2; }
__host__ __device__ constexpr size_t verify_late_floats(int W, int D, bool staged) {
  const size_t late = (size_t)W * D + 2 * verify_pairs(W), raw = staged ? ((size_t)(W + 3) * 3 * D + 1) / 2 : 0;
  return late > raw ? late : raw;
}
__host__ __device__ constexpr size_t verify_smem_floats(int W, int D, bool staged, bool split) {
  const size_t all = (size_t)2 * W * (D + 4) + (size_t)2 * W * D + (size_t)W * (4 + (split ? D / 4 : 0)) +
                     verify_late_floats(W, D, staged) + (size_t)5 * W + 1 + (verify_pairs(W) + 1) / 2;
  return (all + 3) / 4 * 4;  // what follows starts on 16 bytes
}
__device__ __forceinline__ void copy_async16(void *smem, const void *global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(global)
               : "memory");
}

// F + 32 n for the n that brings F to -16 or above; returns n, at most 4 at a step (a retention of 0 counts as
// 2^-127)
__device__ __forceinline__ uint32_t wrap(float &f) {
  const float n = fmaxf(floorf(fmaf(f, -0.03125f, 0.5f)), 0.f);
  f = fmaf(n, 32.f, f);
  return (uint32_t)n;
}
// f - 32 n of four channels, n in bytes
__device__ __forceinline__ float4 unwrap(float4 f, uint32_t n) {
  auto whole = [&](uint32_t which) { return __uint_as_float(__byte_perm(n, 0x4b000000u, which)) - 8388608.f; };  // 2^23 + byte
  return make_float4(fmaf(whole(0x7540), -32.f, f.x), fmaf(whole(0x7541), -32.f, f.y), fmaf(whole(0x7542), -32.f, f.z),
                     fmaf(whole(0x7543), -32.f, f.w));
}

// columns of the state that a warp of the verify kernel owns, and its threads: four warps of 32
// columns (one of 16 at D = 16)
template <int D>
struct VerifyShape {
  static constexpr int CW = D < 32 ? D : 32, NT = D / CW * 32, NJ = CW / 8;
};
template <int N>
struct Cols {
  float v[N];
};
__device__ __forceinline__ void load_cols(Cols<4> &c, const float *p) {
  const float4 x = __ldcs(reinterpret_cast<const float4 *>(p));
  c.v[0] = x.x, c.v[1] = x.y, c.v[2] = x.z, c.v[3] = x.w;
}
__device__ __forceinline__ void load_cols(Cols<4> &c, const bf16 *p) {
  const float4 x = load4_stream(p);
  c.v[0] = x.x, c.v[1] = x.y, c.v[2] = x.z, c.v[3] = x.w;
}
template <typename ST>
__device__ __forceinline__ void load_cols(Cols<2> &c, const ST *p) {
  const float2 x = load2(p);
  c.v[0] = x.x, c.v[1] = x.y;
}
template <typename ST>
__device__ __forceinline__ void load_cols_shared(Cols<4> &c, const ST *p) {
  const float4 x = load4(p);
  c.v[0] = x.x, c.v[1] = x.y, c.v[2] = x.z, c.v[3] = x.w;
}
template <typename ST>
__device__ __forceinline__ void load_cols_shared(Cols<2> &c, const ST *p) {
  load_cols(c, p);
}
// floats that a state kept in shared memory takes (rows padded by 16 bytes)
template <int D, typename ST>
constexpr size_t resident_floats() {
  return (size_t)D * (D * sizeof(ST) + 16) / 4;
}

// With X the 2 W rows k_i e^{G_i} and q_i e^{G_i}, the product X S is what the state is read for; it
// runs on the tensor cores (mma.sync, 16 rows of X at a time: there are too few rows for the 128-row
// tcgen05 forms, and the kernel is bound by the state's bytes).  Lane (g, t) = (l / 4, l % 4) of warp
// w loads columns 32 w + 4 g .. + 3 of its rows of S, which are its parts of the products' B operands,
// straight from memory into registers, and gets columns 32 w + 8 t .. + 7 of X S.  With bf16 I/O both
// operands are split into two bf16 parts and three products are added, good to about 2^-16 (an output
// is rounded to 2^-8 of itself); with fp32 I/O into two tf32 parts, about 2^-21.
// A CTA is small (four warps, no state held), so that eight share an SM, each in another of the phases
// that the few barriers of a unit cut.  bf16 inputs come into shared memory by asynchronous copies
// that run while the tree is worked out.
// Forms, of x 64 heads:
// RESIDENT: with few units (no more than fit at a time) the state comes into shared memory the same
// way, all at once; read step by step from L2 it would be most of a lone unit's time (one sequence x
// 12 nodes: 19.7 us so, 16.2 resident, before the pairs were listed; 13.7 since).
// LARGE: where shared memory holds five CTAs or fewer there are registers for the pair loop twice, with N and
// without (32 sequences x up to 64 nodes 1268 us; 1411 with the capped forms' one loop; 128 x 16 406 and 425).
// SHALLOW (one fp32 sum) and MANY: eight CTAs an SM, so 64 registers a thread and one pair loop that looks at N
// only where a unit has one that is not 0 (256 x 8: 321 us SHALLOW, 327 MANY; with the loop twice 330 to 339).
// Measured at 256 sequences x 6 to 8 nodes x 64 heads: 321 us, 4.1 TB/s of what it must move.  What is
// not the state's product takes 186 us on its own (issue and the latencies of its short phases), the
// product's loads from L2 most of the rest: more CTAs hide more of both (seven an SM 334 us, six 346, nine
// spill: 356), which is also why deeper loads cost more than they give (two steps of the state in flight
// through shared memory, five CTAs: 438 us; through registers: 363).  The state is asked of L2 by one bulk
// prefetch a unit (325 us by a line a thread, 341 without).
enum { SHALLOW_FORM, MANY_FORM, RESIDENT_FORM, LARGE_FORM };
template <int D, typename IO, typename ST, int FORM>
__global__ void __launch_bounds__(VerifyShape<D>::NT, D == 128 ? (FORM == RESIDENT_FORM ? 2 : FORM == LARGE_FORM ? 5 : 8) : 1)
    tree_verify_kernel(const TreeArgs a) {
  constexpr bool RESIDENT = FORM == RESIDENT_FORM, SPLIT = FORM != SHALLOW_FORM, CAPPED = FORM == SHALLOW_FORM || FORM == MANY_FORM;
  constexpr float F_TOP = SPLIT ? 16.f : 32.f;
  constexpr int CW = VerifyShape<D>::CW, NT = VerifyShape<D>::NT, NJ = VerifyShape<D>::NJ, NW = NT / 32, XS = D + 4;
  constexpr int CT = 3 * D / 4;  // threads of the convolution, four channels each
  constexpr bool EXACT = sizeof(IO) == 4;
  extern __shared__ __align__(16) float smem[];
  const int WM = a.max_nodes;
  float *s_x = smem, *s_v = s_x + 2 * WM * XS, *s_g = s_v + WM * D;
  int4 *s_tap = reinterpret_cast<int4 *>(s_g + WM * D);  // a node's taps, oldest first: nodes, or -1 (newest) .. -3 of the tail
  uint32_t *s_n = reinterpret_cast<uint32_t *>(s_tap + WM);  // N of G, four channels a word
  float *s_o = reinterpret_cast<float *>(s_n + (SPLIT ? WM * (D / 4) : 0)), *s_A = s_o + WM * D, *s_B = s_A + verify_pairs(WM);
  int *s_par = reinterpret_cast<int *>(s_o + verify_late_floats(WM, D, !EXACT));
  int *s_off = s_par + WM;  // the pairs of node i: s_off[i] .. s_off[i + 1] - 1, itself first
  float *s_beta = reinterpret_cast<float *>(s_off + WM + 1), *s_rn = s_beta + WM;
  uint16_t *s_pair = reinterpret_cast<uint16_t *>(s_rn + 2 * WM);  // node << 6 | ancestor
  IO *s_raw = reinterpret_cast<IO *>(s_o);  // row 3 + i: node i, rows 0 .. 2 the tail
  constexpr int SS = D + 16 / (int)sizeof(ST);
  ST *s_S = reinterpret_cast<ST *>(smem + verify_smem_floats(WM, D, !EXACT, SPLIT));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  after_previous();
  const uint32_t H = a.H, units = (uint32_t)a.n_seqs * H;  // at most 65535 x 21845
  const size_t C = (size_t)3 * H * D;

  for (uint32_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int n = (int)(unit / H), h = (int)(unit % H);
    const int slot = a.slot_idx ? a.slot_idx[n] : n;
    int row0;
    const int W = tree_nodes(a, n, WM, row0, tid == 0 && h == 0);
    if (slot < 0 || slot >= a.n_slots) {
      if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
      continue;
    }
    if (W == 0) continue;
    const ST *src = reinterpret_cast<const ST *>(a.state) + ((size_t)slot * H + h) * (size_t)D * D;
    __syncthreads();  // the previous unit's shared memory has been read
    if (!EXACT) {
      constexpr int P = D * (int)sizeof(IO) / 16;  // pieces of a head's channels
      for (int x = tid; x < (W + 3) * 3 * P; x += NT) {
        const int i = x / (3 * P) - 3, st = x / P % 3, y = x % P * (16 / (int)sizeof(IO));
        copy_async16(s_raw + (size_t)(i + 3) * 3 * D + st * D + y, tap_row<IO>(a, row0, slot, i, C) + ((size_t)st * H + h) * D + y);
      }
    }
    for (int x = tid; x < W * (D / 4); x += NT)
      copy_async16(s_g + 4 * x, a.g + ((size_t)(row0 + x / (D / 4)) * H + h) * D + 4 * (x % (D / 4)));
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (RESIDENT) {
      constexpr int P = 16 / (int)sizeof(ST);
      for (int x = tid; x < D * D / P; x += NT) copy_async16(s_S + x / (D / P) * SS + x % (D / P) * P, src + (size_t)x * P);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      // needed a few phases on (any earlier, and L2 drops it again)
      if (tid == 0) ask_bulk(src, sizeof(ST) * D * D);
    }

    // ---- the sequence's tree ---------------------------------------------------------------------
    for (int i = tid; i < W; i += NT) {
      int p = a.parent[row0 + i];
      if (p < -1 || p >= i) {  // not an earlier node: flagged, taken as a root
        if (h == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
        p = -1;
      }
      s_par[i] = p;
      s_beta[i] = a.beta[(size_t)(row0 + i) * H + h];
    }
    __syncthreads();
    for (int i = tid; i < W; i += NT) {
      int u = i, tap[4];
#pragma unroll
      for (int y = 3; y >= 0; --y) {
        tap[y] = u;
        u = u >= 0 ? s_par[u] : (u > -3 ? u - 1 : -3);
      }
      s_tap[i] = make_int4(tap[0], tap[1], tap[2], tap[3]);
    }
    if (warp == 0)
      for (int i0 = 0, base = 0; i0 < W; i0 += 32) {
        const int i = i0 + lane;
        int cnt = 0;
        if (i < W)
          for (int j = i; j >= 0; j = s_par[j]) ++cnt;
        int x = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        int k = base + x - cnt;
        base += __shfl_sync(0xffffffffu, x, 31);
        if (i < W) {
          s_off[i] = k;
          if (i == W - 1) s_off[W] = base;
          for (int j = i; j >= 0; j = s_par[j]) s_pair[k++] = (uint16_t)(i << 6 | j);
        }
      }
    asm volatile("cp.async.wait_group %0;" ::"n"(RESIDENT ? 1 : 0) : "memory");
    __syncthreads();

    // ---- q, k, v of every node after the convolution along its path (a thread four channels of a
    //      stream), beside them the retentions summed along the paths (the other threads, four
    //      channels each), as powers of two
    uint32_t past = 0;
    if (tid < CT) {
      const int c4 = tid % (D / 4), st = tid / (D / 4);
      const size_t ch = (size_t)st * H * D + (size_t)h * D + 4 * c4;
      Conv4 cw;
      cw.load(reinterpret_cast<const IO *>(a.conv_w), ch);
      float *dst = (st == 2 ? s_v : s_x + (st == 0 ? W * XS : 0)) + 4 * c4;
      const int ld = st == 2 ? D : XS;
      const IO *raw = s_raw + 9 * D + st * D + 4 * c4;
      for (int i = 0; i < W; ++i, dst += ld) {
        const int4 tap = s_tap[i];
        auto at = [&](int j) { return EXACT ? load4(tap_row<IO>(a, row0, slot, j, C) + ch) : load4(raw + j * 3 * D); };
        *reinterpret_cast<float4 *>(dst) = cw(at(tap.x), at(tap.y), at(tap.z), at(tap.w));
      }
    } else if (tid - CT < D / 4) {
      const int c = 4 * (tid - CT);
      for (int i = 0; i < W; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(s_g + i * D + c);
        const int p = s_par[i];
        float4 y = make_float4(fmaxf(x.x, a.g_min) * LOG2E, fmaxf(x.y, a.g_min) * LOG2E, fmaxf(x.z, a.g_min) * LOG2E,
                               fmaxf(x.w, a.g_min) * LOG2E);
        float4 z = make_float4(F_TOP, F_TOP, F_TOP, F_TOP);
        uint32_t n = 0;
        if (p >= 0) {
          z = *reinterpret_cast<const float4 *>(s_g + p * D + c);
          if (SPLIT) n = s_n[(p * D + c) / 4];
        }
        y.x += z.x, y.y += z.y, y.z += z.z, y.w += z.w;
        if (SPLIT) {
          if (fminf(fminf(y.x, y.y), fminf(y.z, y.w)) < -16.f)
            n += wrap(y.x) | wrap(y.y) << 8 | wrap(y.z) << 16 | wrap(y.w) << 24;  // no byte passes 255
          s_n[(i * D + c) / 4] = n;
          past |= n;
        }
        *reinterpret_cast<float4 *>(s_g + i * D + c) = y;
      }
    }
    if (unit + gridDim.x < units) {  // the next unit's inputs
      const uint32_t nu = unit + gridDim.x;
      const int nn = (int)(nu / H), ns = a.slot_idx ? a.slot_idx[nn] : nn;
      int nrow0;
      const int nw = tree_nodes(a, nn, WM, nrow0, false);
      if (ns >= 0 && ns < a.n_slots && nw > 0) ask_inputs<D, IO, 1, 0>(a, nrow0, nw, ns, (int)(nu % H), tid, NT);
    }
    bool deep = false;  // is there an N that is not 0
    if (SPLIT) deep = __syncthreads_or(past);
    else __syncthreads();
    // ---- the norms of k and q (eight lanes a row), kept as factors
    for (int x = tid >> 3; x < 2 * W; x += NT / 8) {
      float ss = 0.f;
      for (int c = 4 * (tid & 7); c < D; c += 32) {
        const float4 y = *reinterpret_cast<const float4 *>(s_x + x * XS + c);
        ss = fmaf(y.x, y.x, fmaf(y.y, y.y, fmaf(y.z, y.z, fmaf(y.w, y.w, ss))));
      }
      const unsigned eight = 0xffu << (lane & 24);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(eight, ss, o);
      if ((tid & 7) == 0) s_rn[x] = a.qk_l2norm ? rsqrtf(ss + a.l2_eps) : 1.f;
    }
    __syncthreads();
    // ---- A and B over the (node, ancestor or itself) pairs: eight lanes a pair
    auto pair_products = [&](auto DEEP) {
      const int sub = 4 * (tid & 7), pairs = s_off[W];
      const unsigned eight = 0xffu << (lane & 24);
      for (int k = tid >> 3; k < pairs; k += NT / 8) {
        const int i = s_pair[k] >> 6, j = s_pair[k] & 63;
        float pa = 0.f, pb = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 32) {
          const int c = c0 + sub;
          if (c < D) {
            const float4 gi = *reinterpret_cast<const float4 *>(s_g + i * D + c),
                         gj = *reinterpret_cast<const float4 *>(s_g + j * D + c);
            const float4 kj = *reinterpret_cast<const float4 *>(s_x + j * XS + c),
                         ki = *reinterpret_cast<const float4 *>(s_x + i * XS + c),
                         qi = *reinterpret_cast<const float4 *>(s_x + (W + i) * XS + c);
            float4 d = make_float4(gi.x - gj.x, gi.y - gj.y, gi.z - gj.z, gi.w - gj.w);
            if (CAPPED ? deep : decltype(DEEP)::value) {
              const uint32_t n = s_n[(i * D + c) / 4] - s_n[(j * D + c) / 4];  // N rises along a path: no borrow
              if (!CAPPED || n) d = unwrap(d, n);
            }
            const float e0 = ex2_(d.x) * kj.x, e1 = ex2_(d.y) * kj.y, e2 = ex2_(d.z) * kj.z, e3 = ex2_(d.w) * kj.w;
            pa = fmaf(ki.x, e0, fmaf(ki.y, e1, fmaf(ki.z, e2, fmaf(ki.w, e3, pa))));
            pb = fmaf(qi.x, e0, fmaf(qi.y, e1, fmaf(qi.z, e2, fmaf(qi.w, e3, pb))));
          }
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          pa += __shfl_xor_sync(eight, pa, o);
          pb += __shfl_xor_sync(eight, pb, o);
        }
        if (sub == 0) {
          s_A[k] = pa * s_rn[i] * s_rn[j];
          s_B[k] = pb * s_rn[W + i] * s_rn[j];
        }
      }
    };
    if (!CAPPED && deep) pair_products(std::true_type{});
    else pair_products(std::false_type{});
    __syncthreads();
    if (RESIDENT) asm volatile("cp.async.wait_group 0;" ::: "memory");
    // ---- X = k e^G over q e^G, a warp a row; with bf16 I/O as [D] high parts, then [D] low parts
    for (int x = warp; x < 2 * W; x += NW) {
      float *row = s_x + x * XS;
      const int node = x < W ? x : x - W;
      const float rn = s_rn[x];
      const int c = 4 * lane;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (c < D) {
        float4 e = *reinterpret_cast<const float4 *>(s_g + node * D + c);
        if (deep) e = unwrap(e, s_n[(node * D + c) / 4]);
        y = *reinterpret_cast<const float4 *>(row + c);
        y.x *= ex2_(e.x - F_TOP) * rn, y.y *= ex2_(e.y - F_TOP) * rn, y.z *= ex2_(e.z - F_TOP) * rn,
            y.w *= ex2_(e.w - F_TOP) * rn;
      }
      if (EXACT) {
        if (c < D) *reinterpret_cast<float4 *>(row + c) = y;
      } else {
        uint2 hi, lo;
        split2(y.x, y.y, hi.x, lo.x);
        split2(y.z, y.w, hi.y, lo.y);
        __syncwarp();  // the row has been read
        if (c < D) {
          *reinterpret_cast<uint2 *>(row + c / 2) = hi;
          *reinterpret_cast<uint2 *>(row + D / 2 + c / 2) = lo;
        }
      }
    }
    __syncthreads();
    // ---- X S: k's rows over G's place, q's into s_o
    for (int m0 = 0; m0 < 2 * W; m0 += 16) {
      float acc[NJ][4] = {};
      const ST *mine = (RESIDENT ? s_S : src) + CW * warp + NJ * g;
      constexpr int LD = RESIDENT ? SS : D;
      auto rows_of = [&](Cols<NJ> &x, int r) {
        if (RESIDENT) load_cols_shared(x, mine + r * LD);
        else load_cols(x, mine + (size_t)r * LD);
      };
      // lane l of ldmatrix names row l % 8 of block l / 8: rows 0-7 | 8-15, then 16 bytes on; behind the
      // last row that row is read again (its products are dropped)
      const float *rows = s_x + min(m0 + (lane & 15), 2 * W - 1) * XS + (lane >> 4) * 4;
      if (EXACT) {
#pragma unroll 4
        for (int s = 0; s < D / 8; ++s) {  // rows 8 s + t and 8 s + 4 + t
          Cols<NJ> b0, b1;
          rows_of(b0, 8 * s + t);
          rows_of(b1, 8 * s + 4 + t);
          uint32_t x[4], hi[4], lo[4];
          ldmatrix4(x, rows + 8 * s);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            hi[y] = tf32_(__uint_as_float(x[y]));
            lo[y] = tf32_(__uint_as_float(x[y]) - __uint_as_float(hi[y]));
          }
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const uint32_t p1 = tf32_(b0.v[j]), q1 = tf32_(b1.v[j]);
            mma_16x8x8(acc[j], lo, p1, q1);
            mma_16x8x8(acc[j], hi, tf32_(b0.v[j] - __uint_as_float(p1)), tf32_(b1.v[j] - __uint_as_float(q1)));
            mma_16x8x8(acc[j], hi, p1, q1);
          }
        }
      } else {
        constexpr int STEPS = D / 16;
        Cols<NJ> b0[4];  // rows 16 s + 2 t, + 1, + 8, + 9 of this step and the next
        auto fetch = [&](Cols<NJ> (&x)[4], int s) {
#pragma unroll
          for (int y = 0; y < 4; ++y) rows_of(x[y], 16 * s + 2 * t + (y & 1) + (y >> 1) * 8);
        };
        auto multiply = [&](const Cols<NJ> (&x)[4], int s) {
          uint32_t hi[4], lo[4];
          ldmatrix4(hi, rows + 8 * s);
          ldmatrix4(lo, rows + D / 2 + 8 * s);
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            uint32_t p1, q1, p2, q2;
            split2(x[0].v[j], x[1].v[j], p1, p2);
            split2(x[2].v[j], x[3].v[j], q1, q2);
            mma_16x8x16(acc[j], lo, p1, q1);
            mma_16x8x16(acc[j], hi, p2, q2);
            mma_16x8x16(acc[j], hi, p1, q1);
          }
        };
#pragma unroll 1
        for (int s = 0; s < STEPS; ++s) {
          fetch(b0, s);
          multiply(b0, s);
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = m0 + g + 8 * y;
        if (r < 2 * W) {
          float *dst = (r < W ? s_g + r * D : s_o + (r - W) * D) + CW * warp + 2 * NJ * t;
#pragma unroll
          for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int j = 0; j < NJ; ++j) dst[NJ * z + j] = acc[j][2 * y + z];
        }
      }
    }
    __syncthreads();
    // ---- the corrected writes, by substitution down the tree (u over v's place): a thread a column
    for (int c = tid; c < D; c += NT)
      for (int i = 0; i < W; ++i) {
        float u = s_v[i * D + c] - s_g[i * D + c];
        for (int k = s_off[i] + 1; k < s_off[i + 1]; ++k) u = fmaf(-s_A[k], s_v[(s_pair[k] & 63) * D + c], u);
        s_v[i * D + c] = s_beta[i] * u;
      }
    __syncthreads();
    // ---- the reads, norm and gate: a warp a node, a lane four neighbouring columns
    for (int i = warp; i < W; i += NW) {
      const int c = 4 * lane;
      const size_t row = ((size_t)(row0 + i) * H + h) * D + c;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f), z = o, w = make_float4(1.f, 1.f, 1.f, 1.f);
      if (c < D) {
        if (a.gate) z = load4(reinterpret_cast<const IO *>(a.gate) + row);
        if (a.gate && a.norm_w) w = load4(a.norm_w + c);
        o = *reinterpret_cast<const float4 *>(s_o + i * D + c);
        for (int k = s_off[i]; k < s_off[i + 1]; ++k) {
          const float b = s_B[k];
          const float4 u = *reinterpret_cast<const float4 *>(s_v + (s_pair[k] & 63) * D + c);
          o.x = fmaf(b, u.x, o.x), o.y = fmaf(b, u.y, o.y), o.z = fmaf(b, u.z, o.z), o.w = fmaf(b, u.w, o.w);
        }
        o.x *= a.scale, o.y *= a.scale, o.z *= a.scale, o.w *= a.scale;
      }
      if (a.gate) {
        const float rn = rsqrtf(warp_sum(o.x * o.x + o.y * o.y + o.z * o.z + o.w * o.w) / D + a.norm_eps);
        o.x *= rn * w.x * sigmoid_(z.x), o.y *= rn * w.y * sigmoid_(z.y), o.z *= rn * w.z * sigmoid_(z.z),
            o.w *= rn * w.w * sigmoid_(z.w);
      }
      if (c < D) store4(reinterpret_cast<IO *>(a.out) + row, o);
    }
  }
}

// The accepted path replayed: state read once, every path token's decay and corrected write in
// registers, state written once; then the conv tail.  Lane 4 rg + cq of warp w holds rows (D/8) rg ..
// of columns 16 w + 4 cq .. + 3, so a column's sum over the key rows closes inside its warp, and once
// the tokens are staged in shared memory (k normalised, v, retention, strength) the warps need
// nothing from each other.  A CTA takes `group` heads of a sequence at a time and stages all their
// tokens together: the path is worked out once.  The next head's state comes into shared memory by bulk
// copies from when this one's is in registers.  Bound by the state's bytes, read and written: 409 us for
// 256 sequences x 64 heads x 3.2 tokens, 5.5 TB/s (443 with the next state only asked of L2; without the
// next group's inputs asked of L2 457; two CTAs of eight warps an SM are what the registers hold, and they
// do not hide all of the staging).
constexpr int AT = 8;  // path tokens staged at a time; a longer path goes head by head
// its shared memory: the staged tokens, then the next head's state, in eight parts (a lane group's rows each)
// 64 bytes apart, so that a quarter of a warp reads 128 bytes of different banks
template <int D>
__host__ __device__ constexpr size_t accept_tokens(int group) {
  return ((size_t)group * AT * (3 * D + 1) * sizeof(float) + 127) / 128 * 128;
}
template <int D, typename ST>
__host__ __device__ constexpr size_t accept_part() {
  return (size_t)D / 8 * D * sizeof(ST) + 64;
}
template <int D, typename ST>
constexpr size_t accept_smem(int group) {
  return accept_tokens<D>(group) + 8 * accept_part<D, ST>();
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
template <int D, typename IO, typename ST>
__global__ void __launch_bounds__(2 * D, 2) tree_accept_kernel(const TreeArgs a, int group) {
  constexpr int NT = 2 * D, R = D / 8;
  extern __shared__ __align__(16) float smem[];
  __shared__ int s_par[64], s_path[64], s_m;
  __shared__ __align__(8) uint64_t s_bar;
  // [head of the group][token][k | v | retention][D], then the strengths
  float *s_beta = smem + (size_t)group * AT * 3 * D;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cq = lane & 3, rg = lane >> 2, col = 16 * warp + 4 * cq;
  const uint32_t bar = tc::smem_u32(&s_bar);
  uint8_t *s_state = reinterpret_cast<uint8_t *>(smem) + accept_tokens<D>(group);
  if (tid == 0) {
    tc::mbar_init(bar, 1);
    tc::mbar_fence_init();
  }
  __syncthreads();
  after_previous();
  const int H = a.H;
  const uint32_t groups = (uint32_t)a.n_seqs * (uint32_t)H / group;  // at most 65535 x 21845
  const size_t C = (size_t)3 * H * D;

  // the state of head h of slot `slot` on its way into shared memory (by one thread)
  auto load_state = [&](int slot, int h) {
    constexpr uint32_t bytes = D / 8 * D * sizeof(ST);
    const uint8_t *src = reinterpret_cast<const uint8_t *>(a.state) + ((size_t)slot * H + h) * (8 * (size_t)bytes);
    tc::mbar_expect_tx(bar, 8 * bytes);
    for (int y = 0; y < 8; ++y)
      bulk_load(tc::smem_u32(s_state) + y * (uint32_t)accept_part<D, ST>(), src + y * bytes, bytes, bar);
  };
  // the same of the first group from `unit` on that has something to accept
  auto load_from = [&](uint32_t unit) {
    for (; unit < groups; unit += gridDim.x) {
      const int h = (int)(unit * group % H), n = (int)(unit * group / H), slot = a.slot_idx ? a.slot_idx[n] : n;
      int row0;
      const int W = tree_nodes(a, n, 64, row0, false), last = a.accept[n];
      if (slot >= 0 && slot < a.n_slots && last >= 0 && last < W) {
        load_state(slot, h);
        return;
      }
    }
  };
  if (tid == 0) load_from(blockIdx.x);
  uint32_t loads = 0;

  for (uint32_t unit = blockIdx.x; unit < groups; unit += gridDim.x) {
    const int h0 = (int)(unit * group % H), n = (int)(unit * group / H);
    const int slot = a.slot_idx ? a.slot_idx[n] : n;
    int row0;
    const int W = tree_nodes(a, n, 64, row0, tid == 0 && h0 == 0);
    const int last = a.accept[n];
    if (slot < 0 || slot >= a.n_slots || last < -1 || last >= W) {
      if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
      continue;
    }
    if (last < 0) continue;  // nothing accepted: state and tail stay
    ST *state = reinterpret_cast<ST *>(a.state) + ((size_t)slot * H + h0) * (size_t)D * D;
    __syncthreads();  // the previous group's shared memory has been read
    for (int i = tid; i <= last; i += NT) {
      int p = a.parent[row0 + i];
      if (p < -1 || p >= i) {
        if (h0 == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
        p = -1;
      }
      s_par[i] = p;
    }
    __syncthreads();
    if (tid == 0) {
      int x = 0;
      for (int j = last; j >= 0; j = s_par[j]) ++x;
      s_m = x;
      for (int j = last; j >= 0; j = s_par[j]) s_path[--x] = j;
    }
    __syncthreads();
    const int m = s_m;
    auto at = [&](int d) { return d >= 0 ? s_path[d] : d; };  // path position -> node or tail
    // tokens d0 .. d0 + nt - 1 of heads h .. h + heads - 1
    auto stage = [&](int h, int heads, int d0, int nt) {
      const int total = heads * nt * 2 * (D / 4);
      for (int x = tid; x - lane < total; x += NT) {  // D / 4 neighbouring lanes a row
        const int c4 = x % (D / 4), s = x / (D / 4) % 2, i = x / (D / 2) % nt, y = x / (D / 2 * nt), d = d0 + i;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (x < total) {
          const size_t ch = (size_t)(1 + s) * H * D + (size_t)(h + y) * D + 4 * c4;
          Conv4 cw;
          cw.load(reinterpret_cast<const IO *>(a.conv_w), ch);
          v = cw(load4(tap_row<IO>(a, row0, slot, at(d - 3), C) + ch), load4(tap_row<IO>(a, row0, slot, at(d - 2), C) + ch),
                 load4(tap_row<IO>(a, row0, slot, at(d - 1), C) + ch), load4(tap_row<IO>(a, row0, slot, at(d), C) + ch));
        }
        if (a.qk_l2norm) {
          float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
          for (int o = 1; o < D / 4; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (s == 0) {
            const float rk = rsqrtf(ss + a.l2_eps);
            v.x *= rk, v.y *= rk, v.z *= rk, v.w *= rk;
          }
        }
        if (x < total) *reinterpret_cast<float4 *>(smem + ((size_t)(y * AT + i) * 3 + s) * D + 4 * c4) = v;
      }
      for (int x = tid; x < heads * nt * (D / 4); x += NT) {
        const int c4 = x % (D / 4), i = x / (D / 4) % nt, y = x / (D / 4 * nt);
        const float4 g = load4(a.g + ((size_t)(row0 + s_path[d0 + i]) * H + h + y) * D + 4 * c4);
        *reinterpret_cast<float4 *>(smem + ((size_t)(y * AT + i) * 3 + 2) * D + 4 * c4) = make_float4(
            expf(fmaxf(g.x, a.g_min)), expf(fmaxf(g.y, a.g_min)), expf(fmaxf(g.z, a.g_min)), expf(fmaxf(g.w, a.g_min)));
      }
      for (int x = tid; x < heads * nt; x += NT)
        s_beta[x / nt * AT + x % nt] = a.beta[(size_t)(row0 + s_path[d0 + x % nt]) * H + h + x / nt];
    };
    const bool together = m <= AT;
    if (together) {
      stage(h0, group, 0, m);
      __syncthreads();
    }
    for (int y = 0; y < group; ++y) {
      ST *st = state + (size_t)y * D * D + col;
      float S[R][4];
      const bool here = tc::mbar_wait(bar, loads++ & 1);
      const ST *from = reinterpret_cast<const ST *>(s_state + rg * accept_part<D, ST>()) + col;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 x = load4(from + r * D);
        S[r][0] = x.x, S[r][1] = x.y, S[r][2] = x.z, S[r][3] = x.w;
      }
      if (!__syncthreads_and(here)) {  // did not come: nothing is written
        if (tid == 0 && a.err) atomicOr(a.err, ERR_MBAR_TIMEOUT);
        for (int w = 0; w < 100; ++w) __nanosleep(10000);  // let the copies in flight land
        return;
      }
      if (y + 1 < group) {
        if (tid == 0) load_state(slot, h0 + y + 1);
      } else if (unit + gridDim.x < groups) {  // the next group's first head
        if (tid == 0) load_from(unit + gridDim.x);
        const uint32_t nu = (unit + gridDim.x) * group;
        const int nn = (int)(nu / H), ns = a.slot_idx ? a.slot_idx[nn] : nn;
        int nrow0;
        const int nw = tree_nodes(a, nn, 64, nrow0, false), nl = a.accept[nn];
        if (ns >= 0 && ns < a.n_slots && nl >= 0 && nl < nw) {
          if (group == 2) ask_inputs<D, IO, 2, 1>(a, nrow0, nl + 1, ns, (int)(nu % H), tid, NT);
          else ask_inputs<D, IO, 1, 1>(a, nrow0, nl + 1, ns, (int)(nu % H), tid, NT);
        }
      }
      for (int d0 = 0; d0 < m; d0 += AT) {
        const int nt = m - d0 < AT ? m - d0 : AT, at0 = together ? y * AT : 0;
        if (!together) {
          __syncthreads();  // the tokens of before have been read
          stage(h0 + y, 1, d0, nt);
          __syncthreads();
        }
        for (int i = 0; i < nt; ++i) {
          const float *tok = smem + (size_t)(at0 + i) * 3 * D, *kr = tok + R * rg, *ar = tok + 2 * D + R * rg;
          float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int r2 = 0; r2 < R; r2 += 2) {
            const float2 k2 = *reinterpret_cast<const float2 *>(kr + r2), a2 = *reinterpret_cast<const float2 *>(ar + r2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              S[r2][c] *= a2.x;
              p[c] = fmaf(S[r2][c], k2.x, p[c]);
              S[r2 + 1][c] *= a2.y;
              p[c] = fmaf(S[r2 + 1][c], k2.y, p[c]);
            }
          }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
#pragma unroll
            for (int c = 0; c < 4; ++c) p[c] += __shfl_xor_sync(0xffffffffu, p[c], off);
          const float4 v = *reinterpret_cast<const float4 *>(tok + D + col);
          const float b = s_beta[at0 + i];
          const float u[4] = {b * (v.x - p[0]), b * (v.y - p[1]), b * (v.z - p[2]), b * (v.w - p[3])};
#pragma unroll
          for (int r2 = 0; r2 < R; r2 += 2) {
            const float2 k2 = *reinterpret_cast<const float2 *>(kr + r2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              S[r2][c] = fmaf(k2.x, u[c], S[r2][c]);
              S[r2 + 1][c] = fmaf(k2.y, u[c], S[r2 + 1][c]);
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        store4_stream(st + (size_t)(R * rg + r) * D, make_float4(S[r][0], S[r][1], S[r][2], S[r][3]));
    }
    // the last three raw inputs of the path (bit-exact copies; every convolution has read the old
    // tail: the staging barriers are behind)
    for (int x = tid; x < 3 * group * D; x += NT) {
      const size_t ch = (size_t)(x / (group * D)) * H * D + (size_t)h0 * D + x % (group * D);
      const IO x0 = tap_row<IO>(a, row0, slot, at(m - 3), C)[ch], x1 = tap_row<IO>(a, row0, slot, at(m - 2), C)[ch],
               x2 = tap_row<IO>(a, row0, slot, at(m - 1), C)[ch];
      IO *tail = reinterpret_cast<IO *>(a.conv_state) + (size_t)slot * 3 * C + ch;
      tail[0] = x0;
      tail[C] = x1;
      tail[2 * C] = x2;
    }
  }
}

// CTAs of `kernel` that fit on the current device, kept per kernel and device for the last shared
// memory size asked (a query costs the host more than a launch).
template <auto kernel>
cudaError_t fitting(int threads, size_t smem, size_t smem_most, int64_t *ctas) {
  static std::atomic<int64_t> known[64];  // size and count + 1 in one word
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int64_t have = dev < 64 ? known[dev].load() : 0;
  if (have && (size_t)(have >> 32) == smem) {
    *ctas = (have & 0xffffffff) - 1;
    return cudaSuccess;
  }
  int nsm = 0, per_sm = 0;
  // always the largest tree's size: a smaller one set by another host thread could come
  // between this call's opt-in and its launch
  if (smem_most > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *ctas = (int64_t)nsm * (per_sm > 0 ? per_sm : 1);
  if (dev < 64) known[dev].store((int64_t)smem << 32 | (*ctas + 1));
  return cudaSuccess;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t ctas, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &early, cfg.numAttrs = 1, cfg.stream = s;
  cfg.gridDim = dim3((unsigned)ctas), cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

constexpr size_t SMEM_MOST = 220 * 1024;  // of a CTA, beside the kernels' static part
template <int D, typename IO, typename ST>
cudaError_t launch_typed(const TreeArgs &a, bool accept, cudaStream_t s) {
  const int64_t units = (int64_t)a.n_seqs * a.H;
  int64_t fit = 0;
  if (accept) {
    constexpr auto kernel = tree_accept_kernel<D, IO, ST>;
    cudaError_t e = fitting<kernel>(2 * D, accept_smem<D, ST>(2), accept_smem<D, ST>(2), &fit);
    if (e != cudaSuccess) return e;
    // two heads staged together where that leaves every CTA several groups (measured at 256 sequences
    // x 64 heads: 470 us one head at a time, 409 two, 453 four)
    const int group = a.H % 2 == 0 && units / 2 >= 4 * fit ? 2 : 1;
    const int64_t groups = units / group;
    return launch(kernel, groups < fit ? groups : fit, 2 * D, accept_smem<D, ST>(group), s, a, group);
  } else {
    constexpr bool staged = sizeof(IO) == 2;
    constexpr int NT = VerifyShape<D>::NT;
    const size_t smem = verify_smem_floats(a.max_nodes, D, staged, true) * sizeof(float), extra = resident_floats<D, ST>() * sizeof(float);
    if (smem + extra <= SMEM_MOST) {
      constexpr auto kernel = tree_verify_kernel<D, IO, ST, RESIDENT_FORM>;
      cudaError_t e = fitting<kernel>(NT, smem + extra, SMEM_MOST, &fit);
      if (e != cudaSuccess) return e;
      if (units <= fit) {
        return launch(kernel, units, NT, smem + extra, s, a);
      }
    }
    auto go = [&](auto FORM) {
      constexpr bool split = decltype(FORM)::value != SHALLOW_FORM;
      constexpr size_t most = verify_smem_floats(64, D, staged, split) * sizeof(float);
      constexpr auto kernel = tree_verify_kernel<D, IO, ST, decltype(FORM)::value>;
      const size_t mine = verify_smem_floats(a.max_nodes, D, staged, split) * sizeof(float);
      cudaError_t e = fitting<kernel>(NT, mine, most, &fit);
      if (e != cudaSuccess) return e;
      return launch(kernel, units < fit ? units : fit, NT, mine, s, a);
    };
    // see the kernel's comment; 1 KB of an SM's shared memory goes to each CTA beside its own
    if (D == 128 && 6 * (smem + 1024) > 228 * 1024) return go(std::integral_constant<int, LARGE_FORM>{});
    if (a.max_nodes * -a.g_min * LOG2E <= 64.f) return go(std::integral_constant<int, SHALLOW_FORM>{});
    return go(std::integral_constant<int, MANY_FORM>{});
  }
}

template <int D>
cudaError_t launch_dim(const TreeArgs &a, bool accept, bool io_bf16, bool st_bf16, cudaStream_t s) {
  if (io_bf16)
    return st_bf16 ? launch_typed<D, bf16, bf16>(a, accept, s) : launch_typed<D, bf16, float>(a, accept, s);
  return st_bf16 ? launch_typed<D, float, bf16>(a, accept, s) : launch_typed<D, float, float>(a, accept, s);
}

}  // namespace

cudaError_t launch_tree(const TreeArgs &a, bool accept, int D, bool io_bf16, bool st_bf16, cudaStream_t s) {
  if (a.n_seqs == 0) return cudaSuccess;
  return D == 128 ? launch_dim<128>(a, accept, io_bf16, st_bf16, s) : launch_dim<16>(a, accept, io_bf16, st_bf16, s);
}

}  // namespace kda
