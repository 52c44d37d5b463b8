// The plan of a span call: every check of device data, then the work line and its cuts.
//
// Checked before anything is written: intervals inside [0, T) and disjoint, no question longer
// than max_chunk (KEV_ERR_INTERVALS); prefixes not negative (KEV_ERR_PREFIX); the block table's
// rows long enough (KEV_ERR_SLOT_OVERFLOW); and every page that is written or seen in range and
// used once (KEV_ERR_SLOT; two questions on one block is the shared-state bug of the KV-cache
// isolation article, hnwysp.cn, §2.3).  Pages that lie wholly outside every new token's window and
// sinks are neither checked nor read: a serving program may have given them back.
//
// One CTA.  Latency bound: a handful of dependent passes over n questions, their pages and their
// items.  Disjointness is one prefix maximum of the interval ends when the intervals come in
// order, and a sort first when they do not.
#include "kev_span.cuh"

namespace kev {
namespace {

constexpr int kThreads = 1024;
constexpr int kPer = kMaxQuestions / kThreads;  // questions per thread in the scans

template <typename T, typename Op>
__device__ T block_scan(T v, Op op, T zero, T* tmp, T* total) {  // exclusive, in thread order
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = op(x, y);
  }
  T before = __shfl_up_sync(0xffffffffu, x, 1);
  if (lane == 0) before = zero;
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = tmp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = op(w, y);
    }
    tmp[lane] = w;
  }
  __syncthreads();
  if (warp > 0) before = op(tmp[warp - 1], before);
  *total = tmp[kThreads / 32 - 1];
  __syncthreads();
  return before;
}

struct AddI { __device__ int operator()(int a, int b) const { return a + b; } };
struct AddL { __device__ long long operator()(long long a, long long b) const { return a + b; } };
struct MaxI { __device__ int operator()(int a, int b) const { return a > b ? a : b; } };

// Ends before each interval (prefix maximum over `get`, in its order); returns whether every
// interval begins at or after it, and writes the gaps between them.
template <typename Get>
__device__ bool in_order(int n, int T, Get get, int* tmp, int2* gaps, int* n_gaps, int* flag) {
  const int t = threadIdx.x;
  int mine = 0;
  for (int e = 0; e < kPer; ++e) {
    const int i = t * kPer + e;
    if (i < n) {
      const kev_interval v = get(i);
      if (v.end > v.begin) mine = max(mine, v.end);
    }
  }
  int last;
  int before = block_scan(mine, MaxI(), 0, tmp, &last);
  bool ok = true;
  int b = before, count = 0;
  for (int e = 0; e < kPer; ++e) {
    const int i = t * kPer + e;
    if (i < n) {
      const kev_interval v = get(i);
      if (v.end > v.begin) {
        ok = ok && v.begin >= b;
        count += v.begin > b;
        b = max(b, v.end);
      }
    }
  }
  if (t == 0) *flag = 0;
  __syncthreads();
  if (!ok) *flag = 1;
  __syncthreads();
  if (*flag) {
    __syncthreads();  // everyone has read the flag
    return false;
  }
  int total;
  int at = block_scan(count, AddI(), 0, tmp, &total);
  b = before;
  for (int e = 0; e < kPer; ++e) {
    const int i = t * kPer + e;
    if (i < n) {
      const kev_interval v = get(i);
      if (v.end > v.begin) {
        if (v.begin > b) gaps[at++] = make_int2(b, v.begin);
        b = max(b, v.end);
      }
    }
  }
  if (t == 0) {
    if (last < T) gaps[total] = make_int2(last, T);
    *n_gaps = total + (last < T);
  }
  return true;
}

__global__ void __launch_bounds__(kThreads, 1) span_plan_kernel(SpanArgs a) {
  extern __shared__ unsigned long long dyn[];  // sort keys, then the bit map of used blocks
  __shared__ int s_base[kMaxQuestions + 1];    // first item of each question
  __shared__ long long s_tmp[32];
  __shared__ int s_itmp[32];
  __shared__ int s_flag, s_err, s_gaps;
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  SpanHeader* hdr = reinterpret_cast<SpanHeader*>(a.ws);
  int32_t* cu = reinterpret_cast<int32_t*>(a.ws + a.layout.cu);
  int2* gaps = reinterpret_cast<int2*>(a.ws + a.layout.gaps);
  if (t == 0) s_err = 0;
  __syncthreads();
  // error ranks: intervals, prefix, overflow, slot -- the first that applies is reported
  auto error = [&](int rank) { atomicMax(&s_err, 8 - rank); };
  auto prefix_of = [&](int i) { return a.prefix ? a.prefix[i] : 0; };

  for (int i = t; i < a.n; i += kThreads) {
    const kev_interval v = a.intervals[i];
    if (v.begin < 0 || v.end < v.begin || v.end > a.T || v.end - v.begin > a.max_chunk) {
      error(0);
    } else if (v.end > v.begin && a.prefix) {
      const int p = a.prefix[i];
      if (p < 0) error(1);
      else if (a.pool_elem && (int64_t)p + (v.end - v.begin) > (int64_t)a.max_blocks * kPage) error(2);
    }
  }
  __syncthreads();
  const bool bad = s_err != 0;
  __syncthreads();
  if (!bad) {
    const kev_interval* iv = a.intervals;
    bool ok = in_order(a.n, a.T, [&](int i) { return iv[i]; }, s_itmp, gaps, &s_gaps, &s_flag);
    if (!ok) {  // sort by begin, then once more
      int n2 = 1;
      while (n2 < a.n) n2 <<= 1;
      for (int i = t; i < n2; i += kThreads) {
        kev_interval v = {0x7fffffff, 0x7fffffff};
        if (i < a.n && iv[i].end > iv[i].begin) v = iv[i];
        dyn[i] = (unsigned long long)(unsigned)v.begin << 32 | (unsigned)v.end;
      }
      __syncthreads();
      for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
          for (int i = t; i < n2; i += kThreads) {
            const int p = i ^ j;
            if (p > i) {
              const unsigned long long x = dyn[i], y = dyn[p];
              if ((x > y) == ((i & k) == 0)) {
                dyn[i] = y;
                dyn[p] = x;
              }
            }
          }
          __syncthreads();
        }
      ok = in_order(a.n, a.T,
                    [&](int i) {
                      return kev_interval{(int)(dyn[i] >> 32), (int)(dyn[i] & 0xffffffffu)};
                    },
                    s_itmp, gaps, &s_gaps, &s_flag);
      if (!ok && t == 0) error(0);
    }
  }
  __syncthreads();

  if (s_err == 0 && a.pool_elem) {
    // pages: one warp per question, a lane per page; a block's bit may be set once
    unsigned* used = reinterpret_cast<unsigned*>(dyn);
    const int words = (a.n_blocks + 31) / 32;
    for (int i = t; i < words; i += kThreads) used[i] = 0u;
    __syncthreads();
    for (int i = warp; i < a.n; i += kThreads / 32) {
      const kev_interval v = a.intervals[i];
      const int L = v.end - v.begin;
      if (L <= 0) continue;
      const int p0 = prefix_of(i), p1 = p0 + L - 1;
      int ns = 0, lo = p0 / kPage;
      if (a.attend) {
        const SpanTiles s(p0, p1, a.window, a.sinks);
        ns = s.ns;
        lo = s.lo;
      }
      const int pages = ns + p1 / kPage - lo + 1;
      for (int e = lane; e < pages; e += 32) {
        const int b = a.table[(int64_t)i * a.max_blocks + (e < ns ? e : lo + e - ns)];
        if (b < 0 || b >= a.n_blocks) {
          error(3);
        } else {
          const unsigned bit = 1u << (b & 31);
          if (atomicOr(&used[b >> 5], bit) & bit) error(3);
        }
      }
    }
    __syncthreads();
  }
  if (s_err) {
    if (t == 0) {
      const int rank = 8 - s_err;
      const int code = rank == 0 ? ST_INTERVALS : rank == 1 ? ST_PREFIX : rank == 2 ? ST_OVERFLOW : ST_SLOT;
      hdr->status = code;
      if (a.dev_status) *a.dev_status = code;
    }
    return;
  }

  // prefix sums of the lengths, and of the items
  int len = 0, items = 0;
  const int item_tokens = a.tile_tokens * a.item_tiles;
  for (int e = 0; e < kPer; ++e) {
    const int i = t * kPer + e;
    if (i < a.n) {
      const int L = a.intervals[i].end - a.intervals[i].begin;
      len += L;
      if (a.attend) items += (L + item_tokens - 1) / item_tokens;
    }
  }
  int n_new, n_items;
  int at = block_scan(len, AddI(), 0, s_itmp, &n_new);
  int ib = block_scan(items, AddI(), 0, s_itmp, &n_items);
  for (int e = 0; e < kPer; ++e) {
    const int i = t * kPer + e;
    if (i < a.n) {
      const int L = a.intervals[i].end - a.intervals[i].begin;
      cu[i] = at;
      s_base[i] = ib;
      at += L;
      if (a.attend) ib += (L + item_tokens - 1) / item_tokens;
    }
  }
  if (t == 0) {
    cu[a.n] = n_new;
    s_base[a.n] = n_items;
    hdr->n_items = n_items;
    hdr->n_gaps = s_gaps;
    hdr->n_new = n_new;
    hdr->status = ST_OK;
    if (a.dev_status) *a.dev_status = ST_OK;
  }
  __syncthreads();
  if (!a.attend) return;

  // items and the key tiles before each
  SpanItem* out = reinterpret_cast<SpanItem*>(a.ws + a.layout.items);
  long long* cum = reinterpret_cast<long long*>(a.ws + a.layout.cum);
  long long run = 0;
  for (int base = 0; base < n_items; base += kThreads) {
    const int x = base + t;
    long long tiles = 0;
    if (x < n_items) {
      int lo = 0, hi = a.n - 1;  // the last question whose first item is at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_base[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      SpanItem w;
      const kev_interval v = a.intervals[lo];
      const int token0 = (x - s_base[lo]) * item_tokens;
      w.question = lo;
      w.row0 = v.begin + token0;
      w.tokens = min(item_tokens, v.end - w.row0);
      w.p0 = prefix_of(lo) + token0;
      w.tiles = SpanTiles(w.p0, w.p0 + w.tokens - 1, a.window, a.sinks).n;
      out[x] = w;
      tiles = (long long)w.tiles * a.h_kv;
    }
    long long sum;
    const long long before = block_scan(tiles, AddL(), 0ll, s_tmp, &sum);
    if (x < n_items) cum[x] = run + before;
    run += sum;
  }
  if (t == 0) cum[n_items] = run;
  __syncthreads();

  // cuts: part c begins at tile floor(c * total / parts) of the line; with at most one part per
  // tile, no part is empty
  SpanCut* cuts = reinterpret_cast<SpanCut*>(a.ws + a.layout.cuts);
  int32_t* arrived = reinterpret_cast<int32_t*>(a.ws + a.layout.arrived);
  const long long total = run;
  const int parts = total < a.ctas ? (int)total : a.ctas;
  for (int c = t; c <= a.ctas; c += kThreads) {
    if (c < a.ctas) arrived[c] = 0;
    const long long g = parts ? total / parts : 0, r = parts ? total % parts : 0;
    auto place = [&](int x) { return (long long)x * g + (long long)x * r / parts; };
    const long long w = c < parts ? place(c) : total;
    SpanCut cut = {n_items, 0, 0, 0, 0};
    if (w < total) {
      int lo = 0, hi = n_items - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cum[mid] <= w) lo = mid;
        else hi = mid - 1;
      }
      const int tiles = out[lo].tiles;
      const long long in = w - cum[lo];
      cut.item = lo;
      cut.head = (int)(in / tiles);
      cut.tile = (int)(in - (long long)cut.head * tiles);
      if (cut.tile > 0) {
        const long long begin = w - cut.tile, end = begin + tiles;
        int first = c - 1, last = c;  // parts that hold a piece of the unit
        while (first > 0 && place(first) > begin) --first;
        while (last + 1 < parts && place(last + 1) < end) ++last;
        cut.first = first;
        cut.parts = last - first + 1;
      }
    }
    cuts[c] = cut;
  }
}

}  // namespace

cudaError_t launch_span_plan(const SpanArgs& a, cudaStream_t s) {
  size_t sort = 8;
  while (sort < sizeof(unsigned long long) * (size_t)a.n) sort <<= 1;
  const size_t map = a.pool_elem ? ((size_t)a.n_blocks + 63) / 64 * 8 : 0;
  const size_t smem = sort > map ? sort : map;
  if (smem > 24 * 1024) {  // always the same limit: calls from several threads do not lower each other's
    const cudaError_t e =
        cudaFuncSetAttribute(span_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpanMaxBlocks / 8);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(span_plan_kernel, dim3(1), dim3(kThreads), smem, s, a);
}

}  // namespace kev
