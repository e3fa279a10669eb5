// mla_tree.cu -- latent attention of a tree of drafted tokens over the paged cache.
//
// The absorbed form's function ("Ling-3.1-flash: Grouped Routing and Two Different MLA Caches",
// section "Why weight absorption keeps the same attention function") for several query nodes of
// a sequence at once: node i, head h has the 576-wide query [q~ ; q^R], every cached position t
// < len the key [c_t ; r_t] and the value c_t, and drafted node j, whose row is at position
// len + j, is a key of node i where bit j of i's mask is set:
//     s_t = scale q . [c_t ; r_t],  z = sum_t softmax(s)_t c_t  over the visible positions
// (z = 0 where none is).
#include "kda_common.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int TL = 512, TK = 576;

__global__ void __launch_bounds__(128) tree_attn_kernel(const TreeAttnArgs a) {
  __shared__ float s_q[TK], s_p[128], s_red[4];
  __shared__ int64_t s_at[128];
  const int64_t t = blockIdx.x;
  const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = seq_of_token(a.cu_nodes, a.n_seqs, t);
  const int64_t lo = a.cu_nodes[n], hi = a.cu_nodes[n + 1];
  if (t < lo || t >= hi) return;  // a row of no sequence
  if (lo < 0 || hi > a.total || hi - lo > 64) {
    if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_SEQLEN);
    return;
  }
  const int W = (int)(hi - lo), i = (int)(t - lo);
  int64_t len = a.c.lengths[n], end = len + W;
  if (len < 0 || end > (int64_t)a.c.max_pages * a.c.page_size) {
    if (tid == 0 && a.err) atomicOr(a.err, ERR_BAD_INDEX);
    len = end = 0;
  }
  const unsigned long long mask = a.mask ? (unsigned long long)a.mask[t] : (2ull << i) - 1;
  const bf16 *q = reinterpret_cast<const bf16 *>(a.q) + (t * a.H + h) * TK;
  for (int c = tid; c < TK; c += 128) s_q[c] = to_f(q[c]);
  const bf16 *pool = reinterpret_cast<const bf16 *>(a.c.pool);
  float m = -INFINITY, l = 0.f, z[4] = {0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  for (int64_t p0 = 0; p0 < end; p0 += 128) {
    const int64_t pos = p0 + tid;
    float s = -INFINITY;
    s_at[tid] = -1;
    if (pos < end && (pos < len || ((mask >> (pos - len)) & 1))) {
      const int page = a.c.table[(int64_t)n * a.c.max_pages + pos / a.c.page_size];
      if (page >= 0 && page < a.c.n_pages) {
        const int64_t row = ((int64_t)page * a.c.page_size + pos % a.c.page_size) * TK;
        s_at[tid] = row;
        s = 0.f;
        for (int c = 0; c < TK; c += 4) {
          const float4 x = load4(pool + row + c);
          s = fmaf(x.x, s_q[c], fmaf(x.y, s_q[c + 1], fmaf(x.z, s_q[c + 2], fmaf(x.w, s_q[c + 3], s))));
        }
        s *= a.scale_log2;
      } else if (a.err) {
        atomicOr(a.err, ERR_BAD_INDEX);
      }
    }
    const float wm = warp_max(s);
    if (lane == 0) s_red[warp] = wm;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float base = mn == -INFINITY ? 0.f : mn, al = exp2f(m - base);
    s_p[tid] = exp2f(s - base);
    __syncthreads();
    float ls = 0.f;
#pragma unroll
    for (int y = 0; y < 4; ++y) z[y] *= al;
    for (int j = 0; j < 128; ++j) {
      if (s_at[j] < 0) continue;
      const float p = s_p[j];
      const float4 x = load4(pool + s_at[j] + 4 * tid);
      z[0] = fmaf(p, x.x, z[0]), z[1] = fmaf(p, x.y, z[1]), z[2] = fmaf(p, x.z, z[2]), z[3] = fmaf(p, x.w, z[3]);
      ls += p;
    }
    l = l * al + ls;
    m = mn;
    __syncthreads();
  }
  const float r = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (t * a.H + h) * TL + 4 * tid;
  const float4 v = make_float4(z[0] * r, z[1] * r, z[2] * r, z[3] * r);
  if (a.z_bf16) store4(reinterpret_cast<bf16 *>(a.z) + at, v);
  else store4(reinterpret_cast<float *>(a.z) + at, v);
}

}  // namespace

size_t mla_tree_ws_bytes(int, int64_t, int) { return 256; }

cudaError_t launch_mla_tree(const TreeAttnArgs &a, int *launches, cudaStream_t s) {
  *launches = 1;
  tree_attn_kernel<<<dim3((unsigned)a.total, a.H), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
