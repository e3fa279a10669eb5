// batch_sums.h -- running sums over a batch's sequences by the threads of a CTA, as many sequences a
// pass as there are threads.  Host code compiles it too: its barriers are tested with slow warps on the CPU.
#pragma once

#ifdef __CUDACC__
#define KDA_BOTH __host__ __device__ __forceinline__
#else
#define KDA_BOTH inline
#endif

namespace kda {

// The warps' sums of a pass.  There are two places, taken in turn, so that the one barrier of each pass is
// enough: a pass writes where the one before the last was read, and every warp has come to the barrier between.
template <int WARPS>
struct PassSums {
  long long slot[2][WARPS];
};

// One pass, by the whole CTA: the sum of x over the threads before this one, on top of `before`, which grows by the
// sum over all.  `pass` counts the CTA's passes over `s`, from 0 on.  Cta: warp(), last_lane(), barrier() and
// inclusive(x), the sum over the lanes up to this one.
template <int WARPS, typename Cta>
KDA_BOTH long long sum_pass(const Cta &cta, PassSums<WARPS> &s, int &pass, long long x, long long &before) {
  long long *slot = s.slot[pass++ & 1];
  const long long up_to = cta.inclusive(x);
  if (cta.last_lane()) slot[cta.warp()] = up_to;
  cta.barrier();
  long long at = before + up_to - x;
#ifdef __CUDACC__
#pragma unroll
#endif
  for (int w = 0; w < WARPS; ++w) {
    const long long v = slot[w];
    if (w < cta.warp()) at += v;
    before += v;
  }
  return at;
}

}  // namespace kda
