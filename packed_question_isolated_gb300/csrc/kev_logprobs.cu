// Log probabilities of given tokens, entropy and the likeliest tokens of rows of logits.
//
// With m the largest logit of a row, y_k = (x_k - m) / T and S = sum_k e^{y_k}:
//   log p_k = y_k - log S,     H = log S - (sum_k e^{y_k} y_k) / S     (no cancellation: y <= 0 and S >= 1).
// One pass over the row.  Every thread keeps a maximum of its own with S and W = sum e^y y relative to it, in log2 units
// (moved when a tile brings a larger logit); joined at the end.  Terms with e^y = 0 add 0 to W, so masked logits
// (-infinity) and logits far below the maximum are harmless.  A NaN, or +infinity less itself, makes S a NaN: such a row,
// and one without anything above -infinity, has no distribution.
//
// Likeliest tokens in the same pass.  Candidates are collected in shared memory: after the first tile a threshold is
// known that at least n logits of the tile reach (the n-th largest of the threads' own maxima), and every later logit has
// to be larger (an equal one loses to those by its index), which a thread tests once per tile on its maximum.  Of random
// rows some hundred candidates are left; the n largest of them, ties to the lowest index, are picked at the end.  While
// the threshold is -infinity (a masked run of tokens at the row's beginning) the next tile makes a new one.  A row whose
// logits rise so steadily that the candidates overflow is read a second time, tile by tile, with the best n kept exactly.
//
// A cluster of up to 8 CTAs takes a row when there are few rows, each a contiguous part of it; with many rows a CTA takes
// whole rows, one after the other.  Every CTA first checks every live row's temperature and token, so an invalid call
// writes nothing.  Bound by memory: V elements a row, once.
#include <algorithm>

#include "kev_internal.cuh"

namespace kev {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kLoads = 4;  // 16-byte loads of a thread and tile
constexpr int kMaxCluster = 8;
constexpr int kCap = 4096;  // candidates: a tile that sets a threshold leaves 31 * 32 + 1024 of them at most
constexpr int kTop = KEV_MAX_TOP;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t ld_peer_u32(const void* p, uint32_t rank) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whole numbers in the order of the floats (-0 and 0 the same); -infinity is above 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
// The float of such a number; of E = 2 bytes: of its upper half (a bf16 value's lower bits are 0)
template <int E>
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float((o & 0x80000000u ? o & 0x7fffffffu : ~o) & (E == 2 ? 0xffff0000u : 0xffffffffu));
}
// a candidate: larger logits first, of equal ones the lowest index
__device__ __forceinline__ unsigned long long key_of(float x, int k) {
  return (unsigned long long)order_of(x) << 32 | (0xffffffffu - (uint32_t)k);
}

struct Stats {  // of logits, relative to the largest, log2 units
  float m, s, w;
};
__device__ __forceinline__ void join(Stats& a, const Stats& b, float c) {
  if (b.m == -INFINITY && b.s == 0.f) return;
  if (a.m == -INFINITY && a.s == 0.f) {
    a = b;
    return;
  }
  const float m = nan_max(a.m, b.m);
  const float da = (a.m - m) * c, db = (b.m - m) * c;  // one of them 0 (or both NaN)
  const float fa = ex2(da), fb = ex2(db);
  // where a factor is 0 the sum is out of reach of fp32, however large its w
  a.w = (fa == 0.f ? 0.f : fa * fmaf(da, a.s, a.w)) + (fb == 0.f ? 0.f : fb * fmaf(db, b.s, b.w));
  a.s = fmaf(a.s, fa, b.s * fb);
  a.m = m;
}

struct Shared {
  unsigned long long cand[kCap];
  unsigned long long best[kTop];
  unsigned long long merged[kMaxCluster * kTop];
  float warp_m[kWarps], warp_s[kWarps], warp_w[kWarps];
  float part[3];  // this CTA's stats, for the peers
  int scan[kWarps];
  int count, n_best;
  float row_lse2, row_m;
  int bad;
};

// A row, or a cluster's part of it: chunks of 16 bytes [c0, c1) from an aligned address; element e of chunk i is logit
// i * EV + e - head.
template <int E>
struct Part {
  static constexpr int EV = 16 / E;
  const uint4* base;
  int head, c0, c1, vocab;
  // chunk i; what lies outside the row is -infinity
  __device__ __forceinline__ uint4 load(int i) const {
    const int k0 = i * EV - head;
    if (i < c1 && k0 >= 0 && k0 + EV <= vocab) return __ldcs(base + i);
    uint32_t u[4];
    if constexpr (E == 2) {
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(base) + head;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t v = 0xff80ff80u;
        if (i < c1) {
          const int k = k0 + 2 * e;
          if (k >= 0 && k < vocab) v = (v & 0xffff0000u) | __bfloat16_as_ushort(row[k]);
          if (k + 1 >= 0 && k + 1 < vocab) v = (v & 0xffffu) | (uint32_t)__bfloat16_as_ushort(row[k + 1]) << 16;
        }
        u[e] = v;
      }
    } else {
      const float* row = reinterpret_cast<const float*>(base) + head;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = k0 + e;
        u[e] = i < c1 && k >= 0 && k < vocab ? __float_as_uint(row[k]) : 0xff800000u;
      }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <int E>
__device__ __forceinline__ void unpack(uint4 w, float (&f)[16 / E]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E == 2) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    } else {
      f[i] = __uint_as_float(u[i]);
    }
  }
}

// A tile: kLoads chunks a thread, chunk first + l * kThreads + thread.
template <int E>
struct Tile {
  static constexpr int EV = 16 / E;
  uint4 w[kLoads];
  int first;
  __device__ __forceinline__ void load(const Part<E>& p, int at) {
    first = at + threadIdx.x;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) w[l] = p.load(first + l * kThreads);
  }
  __device__ __forceinline__ float top() const {
    float m = -INFINITY;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      float f[EV];
      unpack<E>(w[l], f);
#pragma unroll
      for (int e = 0; e < EV; ++e) m = nan_max(m, f[e]);
    }
    return m;
  }
  // f(logit, index) for every logit of the row
  template <typename F>
  __device__ __forceinline__ void each(const Part<E>& p, F f) const {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      float x[EV];
      unpack<E>(w[l], x);
      const int i = first + l * kThreads, k0 = i * EV - p.head;
      if (i >= p.c1) continue;
#pragma unroll
      for (int e = 0; e < EV; ++e)
        if (k0 + e >= 0 && k0 + e < p.vocab) f(x[e], k0 + e);
    }
  }
};

__device__ __forceinline__ void push(Shared& sm, float x, int k) {
  const int at = atomicAdd(&sm.count, 1);
  if (at < kCap) sm.cand[at] = key_of(x, k);
}

// The largest u of which at least n of the threads' numbers are not below it (0: there is none above 0); the whole CTA.
template <int kBits>
__device__ uint32_t nth_largest(uint32_t mine, int n) {
  uint32_t u = 0;
#pragma unroll 1
  for (int b = 31; b >= 32 - kBits; --b) {
    const uint32_t t = u | 1u << b;
    if (__syncthreads_count(mine >= t) >= n) u = t;
  }
  return u;
}

// A tile that sets the threshold: candidates above `thr` (any, if `open`: nothing came before) of the n largest of the
// tile, or a few more.  Returns the new threshold; later logits have to be larger.  At most 31 * EV * kLoads + 1024
// candidates are pushed.  The whole CTA.
template <int E>
__device__ float threshold(Shared& sm, const Part<E>& p, const Tile<E>& t, float top, float thr, bool open, int n) {
  // a thread without a logit of the row (or without one above the threshold) counts for nothing
  const bool any = open ? t.first < p.c1 : top > thr;
  const uint32_t u = nth_largest<8 * E>(any ? order_of(top) : 0u, n);
  if (u == 0) {  // fewer than n threads have one: all that they have
    t.each(p, [&](float x, int k) {
      if (open || x > thr) push(sm, x, k);
    });
    return thr;
  }
  const float at = value_of<E>(u);
  int ties = 0;
  t.each(p, [&](float x, int k) {
    if (x > at) push(sm, x, k);
    ties += x == at;
  });
  if (__syncthreads_count(ties > 0) <= 1024 / (kLoads * Tile<E>::EV)) {
    t.each(p, [&](float x, int k) {
      if (x == at) push(sm, x, k);
    });
    return at;
  }
  // many equal ones: the n of the lowest indices, in the tile's order of chunks
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
#pragma unroll 1
  for (int l = 0; l < kLoads && before < n; ++l) {
    const int i = t.first + l * kThreads, k0 = i * Tile<E>::EV - p.head;
    float x[Tile<E>::EV];
    unpack<E>(l == 0 ? t.w[0] : l == 1 ? t.w[1] : l == 2 ? t.w[2] : t.w[3], x);
    auto tie = [&](int e) { return i < p.c1 && k0 + e >= 0 && k0 + e < p.vocab && x[e] == at; };
    int c = 0;
#pragma unroll
    for (int e = 0; e < Tile<E>::EV; ++e) c += tie(e);
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int rank = before + incl - c, total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) rank += sm.scan[w];
      total += sm.scan[w];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < Tile<E>::EV; ++e)
      if (tie(e)) {
        if (rank < n) push(sm, x[e], k0 + e);
        ++rank;
      }
    before += total;
  }
  return at;
}

// The n largest candidates (fewer if there are fewer) in order, into sm.best; the whole CTA.
template <int E>
__device__ void pick(Shared& sm, int n) {
  __syncthreads();
  const int count = min(sm.count, kCap), t = threadIdx.x;
  const int slots = (count + kThreads - 1) / kThreads;
  uint32_t u = 0;  // the n-th largest value
  if (count > n) {
#pragma unroll 1
    for (int b = 31; b >= 32 - 8 * E; --b) {
      const uint32_t v = u | 1u << b;
      int c = 0;
      for (int s = 0; s < slots; ++s) {
        const int x = s * kThreads + t;
        c += __syncthreads_count(x < count && (uint32_t)(sm.cand[x] >> 32) >= v);
      }
      if (c >= n) u = v;
    }
  }
  // those from it on, n and the ties of the last, ranked against each other
  for (int s = 0; s < slots; ++s) {
    const int x = s * kThreads + t;
    if (x >= count) continue;
    const unsigned long long mine = sm.cand[x];
    if ((uint32_t)(mine >> 32) < u) continue;
    int rank = 0;
    for (int y = 0; y < count && rank < n; ++y) rank += sm.cand[y] > mine;
    if (rank < n) sm.best[rank] = mine;
  }
  __syncthreads();
  if (t == 0) sm.n_best = min(count, n);
  __syncthreads();
}

template <int E>
__global__ void __launch_bounds__(kThreads, 2) logprobs_kernel(const __grid_constant__ LogprobsArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = (int)cluster_size(), rank = (int)cluster_rank();
  constexpr int EV = 16 / E, kTile = kThreads * kLoads;
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  for (int r = tid; r < a.n; r += kThreads) {
    if (a.active && !a.active[r]) continue;
    if (a.temperature) {
      const float t = a.temperature[r];
      bad |= !(t >= 0.f) || isinf(t);
    }
    if (a.tokens) bad |= a.tokens[r] < 0 || a.tokens[r] >= a.vocab;
  }
  // the same answer in every CTA: whole clusters leave together
  const bool invalid = __syncthreads_or(bad);
  if (blockIdx.x == 0 && tid == 0 && a.dev_status) *a.dev_status = invalid ? ST_SAMPLING : ST_OK;
  if (invalid) return;

  for (int r = (int)blockIdx.x / S; r < a.n; r += (int)gridDim.x / S) {
    if (a.active && !a.active[r]) continue;  // the whole cluster
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = T == 0.f;
    const int need = greedy ? max(a.top_n, 1) : a.top_n;
    const float c = greedy ? kLog2e : fminf(kLog2e / T, 1e30f);
    const char* row = static_cast<const char*>(a.logits) + (int64_t)r * a.vocab * E;
    Part<E> p;
    p.head = (int)((uintptr_t)row & 15) / E;
    p.base = reinterpret_cast<const uint4*>(row - p.head * E);
    p.vocab = a.vocab;
    const int chunks = (p.head + a.vocab + EV - 1) / EV, per = (chunks + S - 1) / S;
    p.c0 = min(chunks, rank * per);
    p.c1 = min(chunks, p.c0 + per);
    float token_logit = 0.f;
    if (a.tokens && tid == 0) {
      const int64_t at = (int64_t)r * a.vocab + a.tokens[r];
      token_logit = E == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
    }
    __syncthreads();  // the row before has been read out of shared memory
    if (tid == 0) sm.count = 0;
    __syncthreads();

    Stats st = {-INFINITY, 0.f, 0.f};
    float thr = -INFINITY;
    bool open = true;
    Tile<E> next;
    next.load(p, p.c0);
    for (int at = p.c0; at < p.c1; at += kTile) {
      const Tile<E> t = next;
      if (at + kTile < p.c1) next.load(p, at + kTile);
      const float top = t.top();
      if (top != -INFINITY) {  // (a NaN goes on)
        if (top > st.m) {
          const float d = (st.m - top) * c, f = ex2(d);
          st.w = f == 0.f ? 0.f : f * fmaf(d, st.s, st.w);
          st.s *= f;
          st.m = top;
        }
        float s = 0.f, w = 0.f;
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          float x[EV];
          unpack<E>(t.w[l], x);
#pragma unroll
          for (int e = 0; e < EV; ++e) {
            const float y = (x[e] - st.m) * c, z = ex2(y);
            s += z;
            w = fmaf(z, nan_max(y, -1000.f), w);
          }
        }
        st.s += s;
        st.w += w;
      }
      if (need > 0) {
        if (thr == -INFINITY) {
          thr = threshold<E>(sm, p, t, top, thr, open, need);
          open = false;
        } else if (top > thr) {
          t.each(p, [&](float x, int k) {
            if (x > thr) push(sm, x, k);
          });
        }
      }
    }
    if (need > 0) {
      __syncthreads();
      if (sm.count > kCap) {  // read again, the best n so far kept after every tile
        __syncthreads();
        if (tid == 0) sm.count = 0;
        thr = -INFINITY;
        open = true;
        for (int at = p.c0; at < p.c1; at += kTile) {
          __syncthreads();
          Tile<E> t;
          t.load(p, at);
          threshold<E>(sm, p, t, t.top(), thr, open, need);
          open = false;
          pick<E>(sm, need);
          if (tid < sm.n_best) sm.cand[tid] = sm.best[tid];
          if (tid == 0) sm.count = sm.n_best;
          thr = sm.n_best == need ? value_of<E>((uint32_t)(sm.best[need - 1] >> 32)) : -INFINITY;
        }
      }
      pick<E>(sm, need);
    }
    // the CTA's sums, then the cluster's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Stats b = {__shfl_xor_sync(0xffffffffu, st.m, o), __shfl_xor_sync(0xffffffffu, st.s, o), __shfl_xor_sync(0xffffffffu, st.w, o)};
      join(st, b, c);
    }
    if (lane == 0) {
      sm.warp_m[warp] = st.m;
      sm.warp_s[warp] = st.s;
      sm.warp_w[warp] = st.w;
    }
    __syncthreads();
    if (warp == 0) {
      Stats b = lane < kWarps ? Stats{sm.warp_m[lane], sm.warp_s[lane], sm.warp_w[lane]} : Stats{-INFINITY, 0.f, 0.f};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        join(b, {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.w, o)}, c);
      st = b;
      if (lane == 0) {
        sm.part[0] = b.m;
        sm.part[1] = b.s;
        sm.part[2] = b.w;
      }
    }
    if (S > 1) {
      cluster_sync_all();
      if (rank == 0) {
        if (warp == 0) {
          Stats b = {-INFINITY, 0.f, 0.f};
          if (lane < S)
            b = {__uint_as_float(ld_peer_u32(&sm.part[0], lane)), __uint_as_float(ld_peer_u32(&sm.part[1], lane)),
                 __uint_as_float(ld_peer_u32(&sm.part[2], lane))};
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            join(b, {__shfl_xor_sync(0xffffffffu, b.m, o), __shfl_xor_sync(0xffffffffu, b.s, o), __shfl_xor_sync(0xffffffffu, b.w, o)}, c);
          st = b;
        }
        if (need > 0) {  // the parts' best, ranked against each other
          unsigned long long mine = 0;
          if (tid < S * kTop) {
            const int from = tid / kTop, j = tid % kTop;
            if (j < need && j < (int)ld_peer_u32(&sm.n_best, from))
              mine = (unsigned long long)ld_peer_u32(reinterpret_cast<const uint32_t*>(&sm.best[j]) + 1, from) << 32 |
                     ld_peer_u32(&sm.best[j], from);
            sm.merged[tid] = mine;
          }
          __syncthreads();
          int place = kTop;
          if (mine) {
            place = 0;
            for (int y = 0; y < S * kTop; ++y) place += sm.merged[y] > mine;
          }
          const bool write = place < need;
          cluster_sync_all();  // nobody reads this CTA's own list any more
          if (write) sm.best[place] = mine;
        } else {
          cluster_sync_all();
        }
      } else {
        cluster_sync_all();
      }
    }
    if (rank == 0) {
      if (tid == 0) {
        sm.bad = !(st.s > 0.f) || isinf(st.m);
        sm.row_m = st.m;
        sm.row_lse2 = log2f(st.s);
      }
      __syncthreads();
      const bool none = sm.bad;
      const float lse2 = sm.row_lse2;
      auto lp = [&](float x) { return ((x - sm.row_m) * c - lse2) * kLn2; };
      if (tid == 0) {
        const int first = greedy && !none ? (int)(0xffffffffu - (uint32_t)sm.best[0]) : 0;
        if (a.tokens) a.logprobs[r] = none ? NAN : greedy ? (a.tokens[r] == first ? 0.f : -INFINITY) : lp(token_logit);
        if (a.entropy) a.entropy[r] = none ? NAN : greedy ? 0.f : (lse2 - st.w / st.s) * kLn2;
      }
      if (tid < a.top_n) {
        const unsigned long long key = none ? 0ull : sm.best[tid];
        a.top_tokens[(int64_t)r * a.top_n + tid] = none ? -1 : (int32_t)(0xffffffffu - (uint32_t)key);
        a.top_logprobs[(int64_t)r * a.top_n + tid] =
            none ? NAN : greedy ? (tid == 0 ? 0.f : -INFINITY) : lp(value_of<E>((uint32_t)(key >> 32)));
      }
    }
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& a, int num_sms, cudaStream_t s) {
  auto kern = a.elem == 2 ? logprobs_kernel<2> : logprobs_kernel<4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared));
  if (e != cudaSuccess) return e;
  // two CTAs on every SM: as many rows, or fewer rows in parts of 4096 logits or more
  const int slots = 2 * num_sms;
  int S = 1;
  while (S < kMaxCluster && (int64_t)a.n * 2 * S <= slots && a.vocab / (2 * S) >= 4096) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min(a.n, std::max(slots / S, 1)) * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace kev
