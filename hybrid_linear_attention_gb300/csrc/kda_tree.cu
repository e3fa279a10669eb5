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
// is ever stored; every exponent is a sum of log-retentions, at most 0.  The accepted path is
// replayed afterwards (tree_accept_kernel), which reads and writes the state once.
#include "kda_common.cuh"
#include "kda_internal.h"

#include <atomic>

namespace kda {
namespace {

__device__ __forceinline__ void l2_prefetch(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, a.w * b.w)));
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

// SiLU of the width-4 causal convolution for four neighbouring channels, taps oldest first.
template <typename IO>
__device__ __forceinline__ float4 conv4(const IO *t0, const IO *t1, const IO *t2, const IO *t3,
                                        const IO *w, size_t ch) {
  const float4 x0 = load4(t0 + ch), x1 = load4(t1 + ch), x2 = load4(t2 + ch), x3 = load4(t3 + ch);
  const float4 wa = load4(w + 4 * ch), wb = load4(w + 4 * ch + 4), wc = load4(w + 4 * ch + 8),
               wd = load4(w + 4 * ch + 12);
  float4 y;
  y.x = siluf_(wa.x * x0.x + wa.y * x1.x + wa.z * x2.x + wa.w * x3.x);
  y.y = siluf_(wb.x * x0.y + wb.y * x1.y + wb.z * x2.y + wb.w * x3.y);
  y.z = siluf_(wc.x * x0.z + wc.y * x1.z + wc.z * x2.z + wc.w * x3.z);
  y.w = siluf_(wd.x * x0.w + wd.y * x1.w + wd.z * x2.w + wd.w * x3.w);
  return y;
}

// shared memory of the verify kernel for at most W nodes (floats): q, k, v, G / accK [W][D]
// each, accQ [W][D], A and B [W][W]
__host__ __device__ constexpr size_t verify_smem_floats(int W, int D) {
  return (size_t)5 * W * D + (size_t)2 * W * W;
}

// One CTA per (sequence, head) at a time; lane 4 rg + cq of warp w holds rows
// (D/8) rg .. of columns 16 w + 4 cq .. + 3 of the state, so a column's sum over the key rows
// closes inside its warp.
template <int D, typename IO, typename ST>
__global__ void __launch_bounds__(2 * D) tree_verify_kernel(const TreeArgs a) {
  constexpr int NT = 2 * D, R = D / 8, NW = NT / 32;
  extern __shared__ __align__(16) float smem[];
  __shared__ int s_par[64], s_up[64][3];
  __shared__ unsigned long long s_anc[64];
  __shared__ float s_beta[64];
  const int WM = a.max_nodes;
  float *s_q = smem, *s_k = s_q + WM * D, *s_v = s_k + WM * D, *s_g = s_v + WM * D;
  float *s_o = s_g + WM * D, *s_A = s_o + WM * D, *s_B = s_A + WM * WM;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cq = lane & 3, rg = lane >> 2, col = 16 * warp + 4 * cq;
  const int H = a.H;
  const int64_t units = (int64_t)a.n_seqs * H;
  const size_t C = (size_t)3 * H * D;

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int h = (int)(unit % H), n = (int)(unit / H);
    const int slot = a.slot_idx ? a.slot_idx[n] : n;
    {  // the next unit's state into L2
      const int64_t nx = unit + gridDim.x;
      if (nx < units) {
        const int nn = (int)(nx / H), sn = a.slot_idx ? a.slot_idx[nn] : nn;
        if (sn >= 0 && sn < a.n_slots) {
          const char *p = reinterpret_cast<const char *>(a.state) +
                          ((size_t)sn * H + (int)(nx % H)) * D * D * sizeof(ST);
          for (size_t off = (size_t)tid * 128; off < (size_t)D * D * sizeof(ST); off += (size_t)NT * 128)
            l2_prefetch(p + off);
        }
      }
    }
    int row0;
    const int W = tree_nodes(a, n, WM, row0, tid == 0 && h == 0);
    if (slot < 0 || slot >= a.n_slots) {
      if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
      continue;
    }
    if (W == 0) continue;

    float S[R][4];
    {
      const ST *src = reinterpret_cast<const ST *>(a.state) + ((size_t)slot * H + h) * (size_t)D * D + col;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float4 x = load4_stream(src + (size_t)(R * rg + r) * D);
        S[r][0] = x.x, S[r][1] = x.y, S[r][2] = x.z, S[r][3] = x.w;
      }
    }
    __syncthreads();  // the previous unit's shared memory has been read
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
      unsigned long long m = 0;
      int up[3], u = i;
#pragma unroll
      for (int y = 0; y < 3; ++y) {
        u = u >= 0 ? s_par[u] : (u > -3 ? u - 1 : -3);
        up[y] = u;
      }
      for (int j = s_par[i]; j >= 0; j = s_par[j]) m |= 1ull << j;
      s_anc[i] = m;
      s_up[i][0] = up[0], s_up[i][1] = up[1], s_up[i][2] = up[2];
    }
    // G: the log-retention summed along each node's path
    for (int c = tid; c < D; c += NT)
      for (int i = 0; i < W; ++i) {
        const float g = fmaxf(a.g[((size_t)(row0 + i) * H + h) * D + c], a.g_min);
        const int p = s_par[i];
        s_g[i * D + c] = p >= 0 ? s_g[p * D + c] + g : g;
      }
    __syncthreads();
    // q, k, v of every node after the convolution along its path
    for (int t = tid; t < W * 3 * (D / 4); t += NT) {
      const int c4 = t % (D / 4), st = t / (D / 4) % 3, i = t / (3 * (D / 4));
      const size_t ch = (size_t)st * H * D + (size_t)h * D + 4 * c4;
      const float4 y = conv4(tap_row<IO>(a, row0, slot, s_up[i][2], C), tap_row<IO>(a, row0, slot, s_up[i][1], C),
                             tap_row<IO>(a, row0, slot, s_up[i][0], C), tap_row<IO>(a, row0, slot, i, C),
                             reinterpret_cast<const IO *>(a.conv_w), ch);
      float *dst = (st == 0 ? s_q : st == 1 ? s_k : s_v) + i * D + 4 * c4;
      *reinterpret_cast<float4 *>(dst) = y;
    }
    __syncthreads();
    if (a.qk_l2norm) {
      for (int t = warp; t < 2 * W; t += NW) {
        float *x = (t & 1 ? s_k : s_q) + (t >> 1) * D;
        float ss = 0.f;
        for (int c = lane; c < D; c += 32) ss = fmaf(x[c], x[c], ss);
        const float r = rsqrtf(warp_sum(ss) + a.l2_eps);
        for (int c = lane; c < D; c += 32) x[c] *= r;
      }
      __syncthreads();
    }
    // A and B over the (node, ancestor or itself) pairs: a warp per pair
    for (int t = warp; t < W * W; t += NW) {
      const int i = t / W, j = t % W;
      if (j > i || !(j == i || ((s_anc[i] >> j) & 1))) continue;
      float pa = 0.f, pb = 0.f;
      for (int c = lane; c < D; c += 32) {
        const float e = expf(s_g[i * D + c] - s_g[j * D + c]) * s_k[j * D + c];
        pa = fmaf(s_k[i * D + c], e, pa);
        pb = fmaf(s_q[i * D + c], e, pb);
      }
      pa = warp_sum(pa);
      pb = warp_sum(pb);
      if (lane == 0) s_A[i * WM + j] = pa, s_B[i * WM + j] = pb;
    }
    __syncthreads();
    for (int t = tid; t < W * D; t += NT) {
      const float e = expf(s_g[t]);
      s_q[t] *= e;
      s_k[t] *= e;
    }
    __syncthreads();
    // S^T (k e^G) over G's place, S^T (q e^G) into s_o
    for (int x = 0; x < 2 * W; ++x) {
      const float *vec = (x < W ? s_k + x * D : s_q + (x - W) * D) + R * rg;
      float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[c] = fmaf(S[r][c], vec[r], p[c]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int c = 0; c < 4; ++c) p[c] += __shfl_xor_sync(0xffffffffu, p[c], off);
      float *dst = (x < W ? s_g + x * D : s_o + (x - W) * D) + col;
      if (rg == 0) *reinterpret_cast<float4 *>(dst) = make_float4(p[0], p[1], p[2], p[3]);
    }
    __syncthreads();
    // the corrected writes, by substitution down the tree (u over v's place), then the reads
    if (tid < D)
      for (int i = 0; i < W; ++i) {
        float u = s_v[i * D + tid] - s_g[i * D + tid];
        for (unsigned long long m = s_anc[i]; m; m &= m - 1) {
          const int j = __ffsll((long long)m) - 1;
          u = fmaf(-s_A[i * WM + j], s_v[j * D + tid], u);
        }
        s_v[i * D + tid] = s_beta[i] * u;
      }
    __syncthreads();
    for (int t = tid; t < W * D; t += NT) {
      const int i = t / D, c = t % D;
      float o = s_o[t];
      for (unsigned long long m = s_anc[i] | (1ull << i); m; m &= m - 1) {
        const int j = __ffsll((long long)m) - 1;
        o = fmaf(s_B[i * WM + j], s_v[j * D + c], o);
      }
      s_o[t] = a.scale * o;
    }
    __syncthreads();
    for (int i = warp; i < W; i += NW) {
      const size_t row = ((size_t)(row0 + i) * H + h) * D;
      float rn = 1.f;
      if (a.gate) {
        float ss = 0.f;
        for (int c = lane; c < D; c += 32) ss = fmaf(s_o[i * D + c], s_o[i * D + c], ss);
        rn = rsqrtf(warp_sum(ss) / D + a.norm_eps);
      }
      for (int c = lane; c < D; c += 32) {
        float o = s_o[i * D + c];
        if (a.gate)
          o = o * rn * (a.norm_w ? a.norm_w[c] : 1.f) *
              sigmoidf_(to_f(reinterpret_cast<const IO *>(a.gate)[row + c]));
        reinterpret_cast<IO *>(a.out)[row + c] = from_f<IO>(o);
      }
    }
  }
}

// The accepted path replayed: state read once, every path token's decay and corrected write in
// registers, state written once; then the conv tail of the unit's channels.
constexpr int AT = 8;  // path tokens staged at a time
template <int D, typename IO, typename ST>
__global__ void __launch_bounds__(2 * D) tree_accept_kernel(const TreeArgs a) {
  constexpr int NT = 2 * D, R = D / 8, NW = NT / 32;
  __shared__ __align__(16) float s_k[AT][D], s_v[AT][D], s_a[AT][D];
  __shared__ float s_beta[AT];
  __shared__ int s_par[64], s_path[64], s_m;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cq = lane & 3, rg = lane >> 2, col = 16 * warp + 4 * cq;
  const int H = a.H;
  const int64_t units = (int64_t)a.n_seqs * H;
  const size_t C = (size_t)3 * H * D;

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int h = (int)(unit % H), n = (int)(unit / H);
    const int slot = a.slot_idx ? a.slot_idx[n] : n;
    {
      const int64_t nx = unit + gridDim.x;
      if (nx < units) {
        const int nn = (int)(nx / H), sn = a.slot_idx ? a.slot_idx[nn] : nn;
        if (sn >= 0 && sn < a.n_slots && a.accept[nn] >= 0) {
          const char *p = reinterpret_cast<const char *>(a.state) +
                          ((size_t)sn * H + (int)(nx % H)) * D * D * sizeof(ST);
          for (size_t off = (size_t)tid * 128; off < (size_t)D * D * sizeof(ST); off += (size_t)NT * 128)
            l2_prefetch(p + off);
        }
      }
    }
    int row0;
    const int W = tree_nodes(a, n, 64, row0, tid == 0 && h == 0);
    const int last = a.accept[n];
    if (slot < 0 || slot >= a.n_slots || last < -1 || last >= W) {
      if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
      continue;
    }
    if (last < 0) continue;  // nothing accepted: state and tail stay

    float S[R][4];
    ST *st = reinterpret_cast<ST *>(a.state) + ((size_t)slot * H + h) * (size_t)D * D + col;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 x = load4_stream(st + (size_t)(R * rg + r) * D);
      S[r][0] = x.x, S[r][1] = x.y, S[r][2] = x.z, S[r][3] = x.w;
    }
    __syncthreads();  // the previous unit's shared memory has been read
    for (int i = tid; i <= last; i += NT) {
      int p = a.parent[row0 + i];
      if (p < -1 || p >= i) {
        if (h == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
        p = -1;
      }
      s_par[i] = p;
    }
    __syncthreads();
    if (tid == 0) {
      int m = 0;
      for (int j = last; j >= 0; j = s_par[j]) ++m;
      s_m = m;
      for (int j = last; j >= 0; j = s_par[j]) s_path[--m] = j;
    }
    __syncthreads();
    const int m = s_m;
    auto at = [&](int d) { return d >= 0 ? s_path[d] : d; };  // path position -> node or tail
    for (int d0 = 0; d0 < m; d0 += AT) {
      const int nt = m - d0 < AT ? m - d0 : AT;
      if (d0) __syncthreads();
      for (int t = tid; t < nt * 2 * (D / 4); t += NT) {
        const int c4 = t % (D / 4), s = 1 + t / (D / 4) % 2, i = t / (2 * (D / 4)), d = d0 + i;
        const size_t ch = (size_t)s * H * D + (size_t)h * D + 4 * c4;
        const float4 y = conv4(tap_row<IO>(a, row0, slot, at(d - 3), C), tap_row<IO>(a, row0, slot, at(d - 2), C),
                               tap_row<IO>(a, row0, slot, at(d - 1), C), tap_row<IO>(a, row0, slot, at(d), C),
                               reinterpret_cast<const IO *>(a.conv_w), ch);
        *reinterpret_cast<float4 *>((s == 1 ? s_k[i] : s_v[i]) + 4 * c4) = y;
      }
      for (int t = tid; t < nt * D; t += NT) {
        const int i = t / D, c = t % D;
        s_a[i][c] = expf(fmaxf(a.g[((size_t)(row0 + s_path[d0 + i]) * H + h) * D + c], a.g_min));
      }
      if (tid < nt) s_beta[tid] = a.beta[(size_t)(row0 + s_path[d0 + tid]) * H + h];
      __syncthreads();
      if (a.qk_l2norm) {
        for (int t = warp; t < nt; t += NW) {
          float ss = 0.f;
          for (int c = lane; c < D; c += 32) ss = fmaf(s_k[t][c], s_k[t][c], ss);
          const float r = rsqrtf(warp_sum(ss) + a.l2_eps);
          for (int c = lane; c < D; c += 32) s_k[t][c] *= r;
        }
        __syncthreads();
      }
      for (int i = 0; i < nt; ++i) {
        float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float al = s_a[i][R * rg + r], k = s_k[i][R * rg + r];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            S[r][c] *= al;
            p[c] = fmaf(S[r][c], k, p[c]);
          }
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
#pragma unroll
          for (int c = 0; c < 4; ++c) p[c] += __shfl_xor_sync(0xffffffffu, p[c], off);
        const float4 v = *reinterpret_cast<const float4 *>(&s_v[i][col]);
        const float b = s_beta[i];
        const float u[4] = {b * (v.x - p[0]), b * (v.y - p[1]), b * (v.z - p[2]), b * (v.w - p[3])};
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float k = s_k[i][R * rg + r];
#pragma unroll
          for (int c = 0; c < 4; ++c) S[r][c] = fmaf(k, u[c], S[r][c]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      store4_stream(st + (size_t)(R * rg + r) * D, make_float4(S[r][0], S[r][1], S[r][2], S[r][3]));
    // the last three raw inputs of the path (bit-exact copies; every convolution has read the
    // old tail: the last staging barrier is behind)
    for (int t = tid; t < 3 * D; t += NT) {
      const size_t ch = (size_t)(t / D) * H * D + (size_t)h * D + t % D;
      const IO x0 = tap_row<IO>(a, row0, slot, at(m - 3), C)[ch], x1 = tap_row<IO>(a, row0, slot, at(m - 2), C)[ch],
               x2 = tap_row<IO>(a, row0, slot, at(m - 1), C)[ch];
      IO *tail = reinterpret_cast<IO *>(a.conv_state) + (size_t)slot * 3 * C + ch;
      tail[0] = x0;
      tail[C] = x1;
      tail[2 * C] = x2;
    }
  }
}

template <typename K>
cudaError_t launch_units(K kernel, const TreeArgs &a, int threads, size_t smem, size_t smem_most,
                         cudaStream_t s) {
  int dev = 0, nsm = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  // always the largest tree's size: a smaller one set by another host thread could come
  // between this call's opt-in and its launch
  if (e == cudaSuccess && smem_most > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_most);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.n_seqs * a.H;
  const int64_t fit = (int64_t)nsm * (per_sm > 0 ? per_sm : 1);
  kernel<<<(unsigned)(units < fit ? units : fit), threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int D, typename IO, typename ST>
cudaError_t launch_typed(const TreeArgs &a, bool accept, cudaStream_t s) {
  if (accept) return launch_units(tree_accept_kernel<D, IO, ST>, a, 2 * D, 0, 0, s);
  return launch_units(tree_verify_kernel<D, IO, ST>, a, 2 * D, verify_smem_floats(a.max_nodes, D) * sizeof(float),
                      verify_smem_floats(64, D) * sizeof(float), s);
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
