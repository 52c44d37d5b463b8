// Shared pieces of the attention-mass kernels: how much attention each cached position receives.
//
//   mass[u, g] = decay * mass[u, g] + sum over new tokens t and q-heads h of g of exp(scale q[t,h].K[u,g] - lse[t,h]),
//   lse[t,h] = log sum over u <= p_t of exp(scale q[t,h].K[u,g])
//
// Many rows per question: two passes over the scores, which are not kept -- the rows' log sums first (a row tile against
// its key tiles, the work line of kev_span.cuh, pieces of a row joined by a small kernel), then the positions' sums (a key
// tile against the row tiles that see it).  A position's sum belongs to one CTA, in the order of the rows, so the result
// does not depend on the order in which the GPU works.
#pragma once

#include "kev_span.cuh"

namespace kev {

struct MassArgs {
  SpanArgs s;
  float* mass;
  float decay;
  size_t lse;     // workspace: float[T][h_q] log2 sums
  size_t ticket;  // workspace: next unit of the second pass (CUDA cores)
  size_t cuts;    // workspace: parts of the second pass (tensor cores)
};

cudaError_t launch_mass_simt(const MassArgs& m, int num_sms, cudaStream_t s);
cudaError_t launch_mass_rows(const MassArgs& m, int num_sms, cudaStream_t s);  // bf16 q, at most 16 rows a question
cudaError_t launch_mass_tc(const MassArgs& m, int num_sms, cudaStream_t s);    // bf16 q
size_t mass_cuts_bytes();

// Key tiles (units of the second pass, per kv head) before each question that brings tokens, and all of them: the
// calling CTA's threads, into shared memory [n + 1].  Ends with a barrier.
__device__ __forceinline__ void mass_tiles_before(const SpanArgs& a, int32_t* before) {
  __shared__ int s_sum[33];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x / 32;
  const int per = (a.n + blockDim.x - 1) / blockDim.x;
  auto tiles = [&](int i) {
    const kev_interval v = a.intervals[i];
    return v.end > v.begin ? (a.prefix[i] + v.end - v.begin - 1) / kSpanKeys + 1 : 0;
  };
  int mine = 0;
  for (int e = 0; e < per; ++e)
    if (t * per + e < a.n) mine += tiles(t * per + e);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int x = lane < warps ? s_sum[lane] : 0, y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_sum[lane] = y - x;
    if (lane == 31) s_sum[32] = y;
  }
  __syncthreads();
  int at = s_sum[warp] + incl - mine;
  for (int e = 0; e < per; ++e)
    if (t * per + e < a.n) {
      before[t * per + e] = at;
      at += tiles(t * per + e);
    }
  if (t == 0) before[a.n] = s_sum[32];
  __syncthreads();
}
// the last question i with before[i] <= x: it has tile x (questions without tiles share their successor's value)
__device__ __forceinline__ int mass_question(const int32_t* before, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (before[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace kev
