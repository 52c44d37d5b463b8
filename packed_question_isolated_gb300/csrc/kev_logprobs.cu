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
// whole rows, one after the other.  A thread brings the parts in by bulk copies, tiles of 32 KB, on into the next row while
// this one is finished; what of a row is no whole 16 bytes is read by itself.  Every CTA first checks every live row's
// temperature and token, so an invalid call writes nothing.
//
// Bound by no single unit: 4096 rows of 151,936 bf16 logits with the 5 likeliest tokens take 280 us (4.4 TB/s, 65 % of the
// measured copy rate), without 233, with 20 of them 329; 2048 rows of fp32 230.  An instruction issues in 62 % of the cycles
// (11.7 a logit), the exponentials' pipe is 25 % busy, and the largest stall, with the wait for a result, is the one at block
// barriers: 16 of them where a threshold is made, and those of the ranking.  32 rows with 20 tokens take 15 us, one row 12,
// mostly the chain of loads, thresholds and cluster barriers.
// Rows with a mask: a thread's tile that holds -infinity beside other logits is summed a second time, one by one.  4096 rows
// whose mask leaves one logit in fifty, scattered, take 441 us, where it leaves a run of the first ones 232; 2048 rows of
// fp32 303 and 208.
// Measured and left: tiles in registers one ahead instead of in shared memory (370 us for the first, the compiler spills
// them); candidates read again from global memory (760); tiles of 16 KB (410).
#include <algorithm>

#include "kev_internal.cuh"
#include "kev_sm100.cuh"

namespace kev {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCtas = 2;  // on an SM
constexpr int kLoads = 4;  // 16-byte chunks of a thread and tile
constexpr int kTile = kThreads * kLoads;  // chunks of a tile
constexpr int kMaxCluster = 8;
constexpr int kCap = 2048;  // candidates: a tile that sets a threshold leaves 31 * 32 + 1024 of them at most, beside 32 before
constexpr int kChunks = 512;  // chunks with a candidate
constexpr int kStages = 2;     // tiles on their way
constexpr size_t kStageBytes = (size_t)kStages * kTile * 16;
constexpr int kRanked = 512;  // candidates that are ranked at once, without thinning them out
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

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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
  uint64_t full[kStages], empty[kStages], stall;
  volatile int abort;
  unsigned long long cand[kCap];
  unsigned long long best[kTop];
  unsigned long long merged[kMaxCluster * kTop];
  float warp_m[kWarps], warp_s[kWarps], warp_w[kWarps];
  float part[3];  // this CTA's stats, for the peers
  uint32_t came;  // and whether its tiles came, all of them
  int scan[kWarps];
  int count, n_best;
  uint4 chunk[kChunks];  // chunks with a candidate, and which they are
  int chunk_at[kChunks];
  int chunks;
  float row_lse2, row_m;
  int bad;
};

// A row, or a cluster's part of it: chunks of 16 bytes [c0, c1) from an aligned address; element e of chunk i is logit
// i * EV + e - head.
template <int E>
struct Part {
  static constexpr int EV = 16 / E;
  __device__ __forceinline__ Part(const LogprobsArgs& a, int r, int rank, int S) {
    const char* row = static_cast<const char*>(a.logits) + (int64_t)r * a.vocab * E;
    head = (int)((uintptr_t)row & 15) / E;
    base = reinterpret_cast<const uint4*>(row - head * E);
    vocab = a.vocab;
    const int chunks = (head + vocab + EV - 1) / EV, per = (chunks + S - 1) / S;
    c0 = min(chunks, rank * per);
    c1 = min(chunks, c0 + per);
    i0 = c0 + (c0 == 0 && head > 0);
    i1 = max(i0, c1 - (c1 == chunks && c1 > c0 && (head + vocab) % EV != 0));
  }
  const uint4* base;
  int head, c0, c1, vocab;
  int i0, i1;  // its whole chunks
};
// Chunk i; what lies outside the row is -infinity.
template <int E>
__device__ __forceinline__ uint4 edge(const Part<E>& p, int i) {
  constexpr int EV = 16 / E;
  const int k0 = i * EV - p.head;
  if (i >= p.i0 && i < p.i1) return __ldg(p.base + i);
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = E == 2 ? 0xff80ff80u : 0xff800000u;
  if (i < p.c1) {
    if constexpr (E == 2) {
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(p.base) + p.head;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k0 + e >= 0 && k0 + e < p.vocab)
          u[e / 2] = (u[e / 2] & (e % 2 ? 0xffffu : 0xffff0000u)) | (uint32_t)__bfloat16_as_ushort(row[k0 + e]) << (e % 2 * 16);
    } else {
      const float* row = reinterpret_cast<const float*>(p.base) + p.head;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k0 + e >= 0 && k0 + e < p.vocab) u[e] = __float_as_uint(row[k0 + e]);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
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
  int first, valid;  // its first chunk; how many it has
  static constexpr uint32_t kNone = E == 2 ? 0xff80ff80u : 0xff800000u;  // -infinity
  // whole chunks [at, end) out of a stage
  __device__ __forceinline__ void load(const uint4* stage, int at, int end) {
    first = at + threadIdx.x;
    valid = min(kLoads, (end - first + kThreads - 1) / kThreads);
#pragma unroll
    for (int l = 0; l < kLoads; ++l)
      w[l] = first + l * kThreads < end ? stage[threadIdx.x + l * kThreads] : make_uint4(kNone, kNone, kNone, kNone);
  }
  // chunk i alone, which may lie across an end of the row (i < 0: none)
  __device__ __forceinline__ void load_edge(const Part<E>& p, int i) {
    first = i;
    valid = i >= 0;
    w[0] = i >= 0 ? edge<E>(p, i) : make_uint4(kNone, kNone, kNone, kNone);
#pragma unroll
    for (int l = 1; l < kLoads; ++l) w[l] = make_uint4(kNone, kNone, kNone, kNone);
  }
  // any chunks from `at` on, from global memory
  __device__ __forceinline__ void load_again(const Part<E>& p, int at) {
    first = at + threadIdx.x;
    valid = kLoads;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) w[l] = edge<E>(p, first + l * kThreads);
  }
  // the largest logit, or NaN: two bf16 values at a time
  __device__ __forceinline__ float top() const {
    if constexpr (E == 2) {
      uint32_t m = 0xff80ff80u;
#pragma unroll
      for (int l = 0; l < kLoads; ++l) m = max2(max2(max2(w[l].x, w[l].y), max2(w[l].z, w[l].w)), m);
      return nan_max(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    } else {
      float m = -INFINITY;
#pragma unroll
      for (int l = 0; l < kLoads; ++l)
        m = nan_max(m, nan_max(nan_max(__uint_as_float(w[l].x), __uint_as_float(w[l].y)),
                               nan_max(__uint_as_float(w[l].z), __uint_as_float(w[l].w))));
      return m;
    }
  }
  // the chunks with a logit that reaches thr, into the list
  __device__ __forceinline__ void put(Shared& sm, float thr) const {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      float m;
      if constexpr (E == 2) {
        const uint32_t u = max2(max2(w[l].x, w[l].y), max2(w[l].z, w[l].w));
        m = nan_max(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
      } else {
        m = nan_max(nan_max(__uint_as_float(w[l].x), __uint_as_float(w[l].y)), nan_max(__uint_as_float(w[l].z), __uint_as_float(w[l].w)));
      }
      if (m >= thr && m > -INFINITY) {
        const int at = atomicAdd(&sm.chunks, 1);
        if (at < kChunks) {
          sm.chunk[at] = w[l];
          sm.chunk_at[at] = first + l * kThreads;
        }
      }
    }
  }
  // s = sum of 2^y and w = sum of 2^y y over the tile, y = (x - m) c; where 2^y is 0 nothing is added.  One fused
  // operation gives x c - R with R = m c rounded; what the rounding left, rho = m c - R, is taken out of the sums.  (Where
  // R is so large that rho is too, and where a masked logit makes 0 times -infinity of its term, one by one.)
  __device__ __forceinline__ void sums(float m, float c, float& s, float& w_sum) const {
    const float R = m * c, rho = fmaf(m, c, -R);
    const unsigned long long rx2 = sm100::f2pack(-R, -R), cx2 = sm100::f2pack(c, c);
    unsigned long long s2 = 0, w2 = 0;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      if (l >= valid) break;
      float x[EV];
      unpack<E>(w[l], x);
#pragma unroll
      for (int e = 0; e < EV; e += 2) {
        const unsigned long long y2 = sm100::fma2(sm100::f2pack(x[e], x[e + 1]), cx2, rx2);
        const float2 y = sm100::unpack2(y2);
        const unsigned long long z2 = sm100::f2pack(ex2(y.x), ex2(y.y));
        s2 = sm100::add2(s2, z2);
        w2 = sm100::fma2(z2, y2, w2);
      }
    }
    const float2 sa = sm100::unpack2(s2), wa = sm100::unpack2(w2);
    const float f = ex2(-rho);
    s = sa.x + sa.y;
    w_sum = f * fmaf(-rho, s, wa.x + wa.y);
    s *= f;
    if (!(fabsf(R) < 16777216.f) || w_sum != w_sum) {
      s = w_sum = 0.f;
#pragma unroll 1
      for (int l = 0; l < valid; ++l) {
        float x[EV];
        unpack<E>(l == 0 ? w[0] : l == 1 ? w[1] : l == 2 ? w[2] : w[3], x);
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float y = (x[e] - m) * c, z = ex2(y);
          s += z;
          w_sum = fmaf(z, fmaxf(y, -1000.f), w_sum);
        }
      }
    }
  }
};

// f(logit, index) for every logit of chunk i that belongs to the part.  The chunk is read again: few are looked at.
template <int E, typename F>
__device__ __forceinline__ void each_of(const Part<E>& p, int i, F f) {
  constexpr int EV = 16 / E;
  if (i >= p.c1) return;
  float x[EV];
  unpack<E>(edge<E>(p, i), x);
  const int k0 = i * EV - p.head;
#pragma unroll
  for (int e = 0; e < EV; ++e)
    if (k0 + e >= 0 && k0 + e < p.vocab) f(x[e], k0 + e);
}

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

// Of a tile's logits equal to `at`, the n of the lowest indices as candidates: the tile's chunks are in order.  The whole CTA.
template <int E>
__device__ __noinline__ void first_equal(Shared& sm, const Part<E>& p, int first, float at, int n) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
#pragma unroll 1
  for (int l = 0; l < kLoads && before < n; ++l) {
    int c = 0;
    each_of<E>(p, first + l * kThreads, [&](float x, int k) { c += x == at; });
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
    each_of<E>(p, first + l * kThreads, [&](float x, int k) {
      if (x != at) return;
      if (rank < n) push(sm, x, k);
      ++rank;
    });
    before += total;
  }
}

// A tile (chunks first + l * kThreads, its largest logit of this thread `top`) that sets the threshold: candidates above
// `thr` (any, if `open`: nothing came before) of the n largest of the tile, or a few more.  Returns the new threshold; later
// logits have to be larger.  At most 31 * EV * kLoads + 1024 candidates are pushed.  The whole CTA.
template <int E>
__device__ __noinline__ float threshold(Shared& sm, const Part<E>& p, int first, float top, float thr, bool open, int n) {
  constexpr int EV = 16 / E;
  // a thread without a logit of the row (or without one above the threshold) counts for nothing
  const bool any = open ? first < p.c1 : top > thr;
  const uint32_t u = nth_largest<8 * E>(any ? order_of(top) : 0u, n);
  if (u == 0) {  // fewer than n threads have one: all that they have
    if (any)
#pragma unroll 1
      for (int l = 0; l < kLoads; ++l)
        each_of<E>(p, first + l * kThreads, [&](float x, int k) {
          if (open || x > thr) push(sm, x, k);
        });
    return thr;
  }
  const float at = value_of<E>(u);
  int ties = 0;
  if (any && top >= at)
#pragma unroll 1
    for (int l = 0; l < kLoads; ++l)
      each_of<E>(p, first + l * kThreads, [&](float x, int k) {
        if (x > at) push(sm, x, k);
        ties += x == at;
      });
  if (__syncthreads_count(ties > 0) <= 1024 / (kLoads * EV)) {
    if (ties)
#pragma unroll 1
      for (int l = 0; l < kLoads; ++l)
        each_of<E>(p, first + l * kThreads, [&](float x, int k) {
          if (x == at) push(sm, x, k);
        });
    return at;
  }
  first_equal<E>(sm, p, first, at, n);  // many
  return at;
}

// The n largest candidates (fewer if there are fewer) in order, into sm.best; the whole CTA.
template <int E>
__device__ __noinline__ void pick(Shared& sm, int n) {
  __syncthreads();
  const int count = min(sm.count, kCap), t = threadIdx.x;
  int left = count;               // candidates that may be among them, in front of the list
  if (count > kRanked) {          // so many that they are thinned out first: the n-th largest value, bit by bit
    const int slots = (count + kThreads - 1) / kThreads;
    uint32_t u = 0;
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
    // those from it on move to the front: n, and the ties of the last
    if (t == 0) sm.count = 0;
    unsigned long long mine[kCap / kThreads];
#pragma unroll
    for (int s = 0; s < kCap / kThreads; ++s) mine[s] = s * kThreads + t < count ? sm.cand[s * kThreads + t] : 0ull;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kCap / kThreads; ++s)
      if (mine[s] && (uint32_t)(mine[s] >> 32) >= u) sm.cand[atomicAdd(&sm.count, 1)] = mine[s];
    __syncthreads();
    left = sm.count;
  }
  for (int x = t; x < left; x += kThreads) {  // ranked against each other
    const unsigned long long mine = sm.cand[x];
    int rank = 0;
#pragma unroll 8
    for (int y = 0; y < left; ++y) rank += sm.cand[y] > mine;
    if (rank < n) sm.best[rank] = mine;
  }
  if (t == 0) sm.n_best = min(count, n);
  __syncthreads();
}

template <int E>
__global__ void __launch_bounds__(kThreads, kCtas) logprobs_kernel(const __grid_constant__ LogprobsArgs a) {
  extern __shared__ __align__(128) unsigned char raw[];
  uint4* stages = reinterpret_cast<uint4*>(raw);  // [kStages][kTile]
  Shared& sm = *reinterpret_cast<Shared*>(raw + kStageBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = (int)cluster_size(), rank = (int)cluster_rank();
  constexpr int EV = 16 / E;
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

  // tiles come by bulk copies, kStages of them ahead, across the rows of this CTA
  bool ok = true;
  uint32_t seq = 0, issued = 0;
  auto give_up = [&] {
    ok = false;
    sm.abort = 1;
    set_status(a.dev_status, ST_TIMEOUT);
  };
  auto next_row = [&](int r) {  // the first live row from r on
    while (r < a.n && a.active && !a.active[r]) r += (int)gridDim.x / S;
    return r;
  };
  int ahead = next_row((int)blockIdx.x / S), ahead_at = 0, ahead_end = -1;
  const uint4* ahead_base = nullptr;
  auto issue = [&] {  // by thread 0
    while (ahead < a.n) {
      if (ahead_end < 0) {
        const Part<E> p(a, ahead, rank, S);
        ahead_at = p.i0;
        ahead_end = p.i1;
        ahead_base = p.base;
      }
      if (ahead_at < ahead_end) {
        const uint32_t bytes = (uint32_t)min(kTile, ahead_end - ahead_at) * 16;
        uint64_t* bar = &sm.full[issued % kStages];
        sm100::mbar_arrive_expect_tx(bar, bytes);
        sm100::bulk_load(stages + issued % kStages * kTile, ahead_base + ahead_at, bytes, bar);
        ++issued;
        ahead_at += kTile;
        return;
      }
      ahead = next_row(ahead + (int)gridDim.x / S);
      ahead_end = -1;
    }
  };
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      sm100::mbar_init(&sm.full[s], 1);
      sm100::mbar_init(&sm.empty[s], kWarps);
    }
    sm100::mbar_init(&sm.stall, 1);
    sm.abort = 0;
    sm100::fence_mbar_init();
    for (int s = 0; s < kStages; ++s) issue();
    // (the last CTA of the first cluster: the row is written by another)
    if (a.test_stall && (int)blockIdx.x == S - 1 && !sm100::mbar_wait(&sm.stall, 0, &sm.abort, a.wait_budget)) give_up();
  }
  __syncthreads();

  for (int r = (int)blockIdx.x / S; r < a.n; r += (int)gridDim.x / S) {
    if (a.active && !a.active[r]) continue;  // the whole cluster
    const float T = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = T == 0.f;
    const int need = greedy ? max(a.top_n, 1) : a.top_n;
    const float c = greedy ? kLog2e : fminf(kLog2e / T, 3.4028235e38f);  // finite: 0 times it is 0
    const Part<E> p(a, r, rank, S);
    float token_logit = 0.f;
    if (a.tokens && tid == 0) {
      const int64_t at = (int64_t)r * a.vocab + a.tokens[r];
      token_logit = E == 2 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
    }
    __syncthreads();  // the row before has been read out of shared memory
    if (tid == 0) sm.count = sm.chunks = 0;
    __syncthreads();

    Stats st = {-INFINITY, 0.f, 0.f};
    float thr = -INFINITY;
    auto take = [&](const Tile<E>& t, bool later) {  // later: the tile's logits have higher indices than all before
      const float top = t.top();
      if (top != -INFINITY) {  // (a NaN goes on)
        if (top > st.m) {
          const float d = (st.m - top) * c, f = ex2(d);
          st.w = f == 0.f ? 0.f : f * fmaf(d, st.s, st.w);
          st.s *= f;
          st.m = top;
        }
        float s, w;
        t.sums(st.m, c, s, w);
        st.s += s;
        st.w += w;
      }
      if (need > 0) {
        bool holds = later ? top > thr : top >= thr && top > -INFINITY;
        if (thr == -INFINITY) {
          const uint32_t u = nth_largest<8 * E>(holds ? order_of(top) : 0u, need);
          if (u) thr = value_of<E>(u);
          holds = u ? top >= thr : holds;
        }
        if (holds) t.put(sm, thr);
      }
    };
    for (int at = p.i0; at < p.i1; at += kTile, ++seq) {
      if (tid == 0 && seq > 0) {  // the stage of the tile before is free again
        const uint32_t old = seq - 1;
        if (ok && !sm100::mbar_wait(&sm.empty[old % kStages], (old / kStages) & 1, &sm.abort, a.wait_budget)) give_up();
        if (ok) issue();
      }
      // (after a wait that gave up the rows are walked on, for the barriers that the threads share; a row of which any
      // thread of the cluster missed a tile is not written)
      if (ok && !sm100::mbar_wait(&sm.full[seq % kStages], (seq / kStages) & 1, &sm.abort, a.wait_budget)) give_up();
      Tile<E> t;
      t.load(stages + seq % kStages * kTile, at, p.i1);
      sm100::mbar_arrive_warp(&sm.empty[seq % kStages]);
      take(t, true);
    }
    if (p.i0 > p.c0 || p.i1 < p.c1) {  // chunks across the row's ends
      const int e0 = p.i0 > p.c0 ? p.c0 : -1, e1 = p.i1 < p.c1 && p.c1 - 1 != e0 ? p.c1 - 1 : -1;
      Tile<E> t;
      t.load_edge(p, tid == 0 ? e0 : tid == 1 ? e1 : -1);
      take(t, false);
    }
    if (need > 0) {
      __syncthreads();
      const int chunks_put = sm.chunks;
      if (chunks_put <= kChunks) {
        for (int x = tid; x < chunks_put; x += kThreads) {
          float y[EV];
          unpack<E>(sm.chunk[x], y);
          const int k0 = sm.chunk_at[x] * EV - p.head;
#pragma unroll
          for (int e = 0; e < EV; ++e)
            if (y[e] >= thr && y[e] > -INFINITY) push(sm, y[e], k0 + e);
        }
        __syncthreads();
      }
      const int found = sm.count;
      __syncthreads();
      if (chunks_put > kChunks || found > kCap) {  // read again, the best n so far kept after every tile
        if (tid == 0) sm.count = 0;
        thr = -INFINITY;
        bool open = true;
        for (int at = p.c0; at < p.c1; at += kTile) {
          __syncthreads();
          Tile<E> t;
          t.load_again(p, at);
          threshold<E>(sm, p, t.first, t.top(), thr, open, need);
          open = false;
          pick<E>(sm, need);
          if (tid < sm.n_best) sm.cand[tid] = sm.best[tid];
          if (tid == 0) sm.count = sm.n_best;
          thr = sm.n_best == need ? value_of<E>((uint32_t)(sm.best[need - 1] >> 32)) : -INFINITY;
        }
      } else if (found < need) {  // fewer than n above -infinity: the first of those at it are all in the first tile
        first_equal<E>(sm, p, p.c0 + tid, -INFINITY, need);
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
    bool came = __syncthreads_and(ok);
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
        sm.came = came;
      }
    }
    if (S > 1) {
      cluster_sync_all();
      if (rank == 0) {
        if (warp == 0) {
          Stats b = {-INFINITY, 0.f, 0.f};
          came = __all_sync(0xffffffffu, lane >= S || ld_peer_u32(&sm.came, lane) != 0u);
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
      // (came: the whole CTA's, or in the first warp the cluster's; the first warp writes)
      static_assert(kTop <= 32, "top tokens are written by one warp");
      if (tid == 0 && came) {
        const int first = greedy && !none ? (int)(0xffffffffu - (uint32_t)sm.best[0]) : 0;
        if (a.tokens) a.logprobs[r] = none ? NAN : greedy ? (a.tokens[r] == first ? 0.f : -INFINITY) : lp(token_logit);
        if (a.entropy) a.entropy[r] = none ? NAN : greedy ? 0.f : (lse2 - st.w / st.s) * kLn2;
      }
      if (tid < a.top_n && came) {
        const unsigned long long key = none ? 0ull : sm.best[tid];
        a.top_tokens[(int64_t)r * a.top_n + tid] = none ? -1 : (int32_t)(0xffffffffu - (uint32_t)key);
        a.top_logprobs[(int64_t)r * a.top_n + tid] =
            none ? NAN : greedy ? (tid == 0 ? 0.f : -INFINITY) : lp(value_of<E>((uint32_t)(key >> 32)));
      }
    }
  }
  if (tid == 0 && sm.abort)  // every copy issued lands before the CTA leaves
    for (uint32_t x = issued < kStages ? 0 : issued - kStages; x < issued; ++x) {
      volatile int never = 0;
      sm100::mbar_wait(&sm.full[x % kStages], (x / kStages) & 1, &never, 4000000000ll);
    }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs& call, int num_sms, cudaStream_t s) {
  LogprobsArgs a = call;
  a.wait_budget = wait_budget_cycles();
  a.test_stall = test_stall_requested();
  auto kern = a.elem == 2 ? logprobs_kernel<2> : logprobs_kernel<4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(kStageBytes + sizeof(Shared)));
  if (e != cudaSuccess) return e;
  // kCtas CTAs on every SM: as many rows, or fewer rows in parts of 4096 logits or more.  Shorter parts cost more than they
  // share out: 32 rows of 32,000 logits take 10.1 us so, in parts of 2048 13.7, of 8192 9.7; 8 rows of 8000 8.0, 9.3 and 7.8
  const int slots = kCtas * num_sms;
  int S = 1;
  while (S < kMaxCluster && (int64_t)a.n * 2 * S <= slots && a.vocab / (2 * S) >= 4096) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(std::min(a.n, std::max(slots / S, 1)) * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kStageBytes + sizeof(Shared);
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
