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
// items -- 5 us for a batch without a cache, 6 to 8 with 500 to 2000 pages to look at.  Disjointness is one
// prefix maximum of the interval ends when the intervals come in order, and a sort first when they do
// not.  Equal parts by key tiles (and a fixed cost per unit) rather than whole units, longest first: a
// decode step has fewer units than SMs or a few more, of lengths that differ by 30.
#include "kev_span.cuh"

namespace kev {
namespace {

constexpr int kCumSmem = 4096;  // items whose tile counts are searched in shared memory

// What of a work line the plan needs.
struct PlanLine {
  SpanLine at;
  int32_t item_tokens, min_tokens, max_tokens, ctas, unit_cost, join_from;
};
struct PlanArgs {
  SpanArgs a;
  int32_t lines;
  int32_t seen;  // look at every page that a new token sees, not only at those that are written
  PlanLine line[2];
};

// What the checks and the work lines scan over the questions: end of the intervals so far, new
// tokens, items of both lines, gaps.
struct Scan {
  int end, tokens, items[2], gaps;
};
__device__ __forceinline__ Scan join(const Scan& a, const Scan& b) {
  return {max(a.end, b.end), a.tokens + b.tokens, {a.items[0] + b.items[0], a.items[1] + b.items[1]}, a.gaps + b.gaps};
}
__device__ __forceinline__ Scan up(const Scan& x, int o) {
  return {__shfl_up_sync(0xffffffffu, x.end, o),
          __shfl_up_sync(0xffffffffu, x.tokens, o),
          {__shfl_up_sync(0xffffffffu, x.items[0], o), __shfl_up_sync(0xffffffffu, x.items[1], o)},
          __shfl_up_sync(0xffffffffu, x.gaps, o)};
}
__device__ __forceinline__ long long join(long long a, long long b) { return a + b; }
__device__ __forceinline__ long long up(long long x, int o) { return __shfl_up_sync(0xffffffffu, x, o); }

// Exclusive scan in thread order; two barriers.
template <int kThreads, typename T>
__device__ T block_scan(T v, T zero, T* tmp /* [33] */, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const T y = up(x, o);
    if (lane >= o) x = join(y, x);
  }
  T before = up(x, 1);
  if (lane == 0) before = zero;
  if (lane == 31) tmp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = lane < kThreads / 32 ? tmp[lane] : zero;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const T y = up(w, o);
      if (lane >= o) w = join(y, w);
    }
    T ex = up(w, 1);
    tmp[lane] = lane == 0 ? zero : ex;
    if (lane == 31) tmp[32] = w;
  }
  __syncthreads();
  *total = tmp[32];
  return join(tmp[warp], before);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1) span_plan_kernel(const __grid_constant__ PlanArgs p) {
  const SpanArgs& a = p.a;
  extern __shared__ unsigned long long dyn[];  // intervals, prefixes; sort keys, bit map of used blocks or tile counts
  __shared__ Scan s_scan[33];
  __shared__ long long s_sum[33];
  __shared__ int s_err, s_joins;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = a.n;
  kev_interval* iv = reinterpret_cast<kev_interval*>(dyn);
  int* pre = reinterpret_cast<int*>(iv + n);
  int* base0 = pre + n;  // first item of each question, in each line
  int* base1 = base0 + n + 1;
  unsigned long long* area = dyn + (20 * (size_t)n + 8 + 7) / 8;  // 8 + 4 + 4 + 4 bytes a question, and the two ends
  unsigned* used = reinterpret_cast<unsigned*>(area);
  const int words = a.pool_elem ? (a.n_blocks + 31) / 32 : 0;
  if (t == 0) s_err = s_joins = 0;
  for (int i = t; i < words; i += kThreads) used[i] = 0u;
  pdl_wait();
  pdl_trigger();
#pragma unroll 1
  for (int l = 0; l < p.lines; ++l) {
    uint4* arrived = reinterpret_cast<uint4*>(a.ws + p.line[l].at.arrived);
    for (int x = t; x < p.line[l].ctas * (kSpanRows / 4); x += kThreads) arrived[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  SpanHeader* hdr = reinterpret_cast<SpanHeader*>(a.ws);
  int32_t* cu = reinterpret_cast<int32_t*>(a.ws + a.layout.cu);
  int2* gaps = reinterpret_cast<int2*>(a.ws + a.layout.gaps);
  // ranks as for span_code
  auto error = [&](int rank) { atomicMax(&s_err, 8 - rank); };
  auto items_of = [&](int l, int L) {
    return l < p.lines && L >= p.line[l].min_tokens && L <= p.line[l].max_tokens ? (L + p.line[l].item_tokens - 1) / p.line[l].item_tokens : 0;
  };

  // A thread's questions: `per` consecutive ones.
  const int per = (n + kThreads - 1) / kThreads;
  Scan mine = {};
#pragma unroll 1
  for (int e = 0; e < per; ++e) {
    const int i = t * per + e;
    if (i >= n) break;
    const kev_interval v = a.intervals[i];
    const int first = a.prefix ? a.prefix[i] : 0;
    iv[i] = v;
    pre[i] = first;
    if (v.begin < 0 || v.end < v.begin || v.end > a.T || v.end - v.begin > a.max_chunk) {
      error(0);
    } else if (v.end > v.begin) {
      const int L = v.end - v.begin;
      if (first < 0) error(1);
      else if (a.pool_elem && (int64_t)first + L > (int64_t)a.max_blocks * kPage) error(2);
      if (!span_positions(a, i, first, L)) error(4);
      mine.end = max(mine.end, v.end);
      mine.tokens += L;
      mine.items[0] += items_of(0, L);
      mine.items[1] += items_of(1, L);
    }
  }
  Scan all;
  const Scan before = block_scan<kThreads>(mine, Scan{}, s_scan, &all);

  const bool clean = s_err <= 4;   // the checks of single questions passed (but for positions: the pages come first)
  const bool inside = s_err != 8;  // at least those of their intervals
  __syncthreads();

  // Disjoint, if every interval begins at or after the end of all before it; otherwise sorted by
  // beginning and looked at again.
  bool ok = true;
  if (inside) {
    int end = before.end, tokens = before.tokens, items0 = before.items[0], items1 = before.items[1];
#pragma unroll 1
    for (int e = 0; e < per; ++e) {
      const int i = t * per + e;
      if (i >= n) break;
      const int L = iv[i].end - iv[i].begin;
      cu[i] = tokens;
      base0[i] = items0;
      base1[i] = items1;
      if (L > 0) {
        ok = ok && iv[i].begin >= end;
        mine.gaps += iv[i].begin > end;
        end = max(end, iv[i].end);
        tokens += L;
        items0 += items_of(0, L);
        items1 += items_of(1, L);
      }
    }
    if (t == 0) {
      cu[n] = all.tokens;
      base0[n] = all.items[0];
      base1[n] = all.items[1];
    }
    if (words && clean) {  // pages: one or more warps per question, a lane per page; a block's bit may be set once
      const int slices = n < kThreads / 32 ? kThreads / 32 / n : 1;
#pragma unroll 1
      for (int x = warp; x < n * slices; x += kThreads / 32) {
        const int i = x / slices;
        const int L = iv[i].end - iv[i].begin;
        if (L <= 0) continue;
        const int p0 = pre[i], p1 = p0 + L - 1;
        int ns = 0, lo = p0 / kPage;
        if (p.seen) {
          const SpanTiles s(p0, p1, a.window, a.sinks);
          ns = s.ns;
          lo = s.lo;
        }
        const int pages = ns + p1 / kPage - lo + 1;
        const int32_t* row = a.table + (int64_t)i * a.max_blocks;
#pragma unroll 4
        for (int e = x % slices * 32 + lane; e < pages; e += 32 * slices) {
          const int b = row[e < ns ? e : lo + e - ns];
          const unsigned bit = 1u << (b & 31);
          if (b < 0 || b >= a.n_blocks || atomicOr(&used[b >> 5], bit) & bit) error(3);
        }
      }
    }
  }
  bool sorted = __syncthreads_and(ok);
  auto interval = [&](int i) { return iv[i]; };
  auto ordered = [&](int i) { return kev_interval{(int)(area[i] >> 32), (int)(area[i] & 0xffffffffu)}; };
  if (inside && !sorted) {
    int n2 = 1;
    while (n2 < n) n2 <<= 1;
    for (int i = t; i < n2; i += kThreads)  // empty intervals last
      area[i] = i < n && iv[i].end > iv[i].begin ? (unsigned long long)iv[i].begin << 32 | (unsigned)iv[i].end
                                                 : 0x7fffffff7fffffffull;
    __syncthreads();
#pragma unroll 1
    for (int k = 2; k <= n2; k <<= 1)
#pragma unroll 1
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = t; i < n2; i += kThreads) {
          const int other = i ^ j;
          if (other > i) {
            const unsigned long long x = area[i], y = area[other];
            if ((x > y) == ((i & k) == 0)) {
              area[i] = y;
              area[other] = x;
            }
          }
        }
        __syncthreads();
      }
  }
  // gaps between the intervals in order
  auto find_gaps = [&](auto get, bool check) {
    Scan v = {}, total;
    for (int e = 0; e < per; ++e) {
      const int i = t * per + e;
      if (i < n && get(i).end > get(i).begin) v.end = max(v.end, get(i).end);
    }
    const int first = block_scan<kThreads>(v, Scan{}, s_scan, &total).end;
    int end = first;
    for (int e = 0; e < per; ++e) {
      const int i = t * per + e;
      if (i < n && get(i).end > get(i).begin) {
        if (check && get(i).begin < end) error(0);
        v.gaps += get(i).begin > end;
        end = max(end, get(i).end);
      }
    }
    __syncthreads();  // the scan's scratch is free
    int at = block_scan<kThreads>(v, Scan{}, s_scan, &total).gaps;
    end = first;
    for (int e = 0; e < per; ++e) {
      const int i = t * per + e;
      if (i < n && get(i).end > get(i).begin) {
        if (get(i).begin > end) gaps[at++] = make_int2(end, get(i).begin);
        end = max(end, get(i).end);
      }
    }
    if (t == 0) {
      if (total.end < a.T) gaps[total.gaps] = make_int2(total.end, a.T);
      hdr->n_gaps = total.gaps + (total.end < a.T);
    }
  };
  if (inside) {
    if (!sorted) find_gaps(ordered, true);
    else if (p.lines && all.tokens < a.T) find_gaps(interval, false);
    else if (t == 0) hdr->n_gaps = 0;
    __syncthreads();
  }
  if (s_err) {
    if (t == 0) {
      const int code = span_code(s_err);
      hdr->status = code;
      if (a.dev_status) *a.dev_status = code;
    }
    return;
  }
  if (t == 0) {
    hdr->n_new = all.tokens;
    hdr->status = ST_OK;
    if (a.dev_status) *a.dev_status = ST_OK;
  }

#pragma unroll 1
  for (int l = 0; l < p.lines; ++l) {
    const PlanLine& line = p.line[l];
    const int* base = l ? base1 : base0;
    // items and the key tiles before each
    SpanItem* out = reinterpret_cast<SpanItem*>(a.ws + line.at.items);
    const int n_items = base[n];
    long long* cum = n_items <= kCumSmem ? reinterpret_cast<long long*>(area)
                                         : reinterpret_cast<long long*>(a.ws + line.at.cum);
    auto record = [&](int x) {
      int lo = 0, hi = n - 1;  // the last question whose first item is at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      SpanItem w = {};
      const int token0 = (x - base[lo]) * line.item_tokens;
      w.question = lo;
      w.row0 = iv[lo].begin + token0;
      w.tokens = min(line.item_tokens, iv[lo].end - w.row0);
      w.p0 = pre[lo] + token0;
      w.tiles = SpanTiles(w.p0, w.p0 + w.tokens - 1, a.window, a.sinks).n;
      return w;
    };
    long long run = 0;
#pragma unroll 1
    for (int first = 0; first < n_items; first += kThreads) {
      const int x = first + t;
      long long tiles = 0;
      if (x < n_items) {
        const SpanItem w = record(x);
        out[x] = w;
        tiles = (long long)(w.tiles + line.unit_cost) * a.h_kv;
      }
      long long sum;
      const long long at = block_scan<kThreads>(tiles, 0ll, s_sum, &sum);
      if (x < n_items) cum[x] = run + at;
      run += sum;
      __syncthreads();
    }

    // cuts: part c begins at place floor(c * total / parts) of the line, where a unit is its fixed cost
    // and then its tiles; a cut in the fixed cost moves to the unit's beginning
    SpanCut* cuts = reinterpret_cast<SpanCut*>(a.ws + line.at.cuts);
    int32_t* joins = reinterpret_cast<int32_t*>(a.ws + line.at.joins);
    const long long total = run;
    const int parts = total < line.ctas ? (int)total : line.ctas;
    // place(c) without 64-bit divisions per thread; the part that holds a place by an estimate and steps
    const long long q = parts ? total / parts : 0;
    const unsigned r = parts ? (unsigned)(total - q * parts) : 0u;
    // x / parts for x < 2^17 and parts < 2^9, by a rounded-up reciprocal (its error times x stays below 2^32)
    const unsigned per_part = parts ? 0xffffffffu / (unsigned)parts + 1u : 0u;
    auto place = [&](int c) { return c * q + (parts == 1 ? 0u : __umulhi((unsigned)c * r, per_part)); };
    const float per_place = total ? (float)parts / (float)total : 0.f;
    auto part_of = [&](long long x) {
      int c = min(parts - 1, (int)((float)x * per_place));
      while (c > 0 && place(c) > x) --c;
      while (c + 1 < parts && place(c + 1) <= x) ++c;
      return c;
    };
    for (int c = t; c <= line.ctas; c += kThreads) {
      const long long w = c < parts ? place(c) : total;
      SpanCut cut = {};
      cut.item = n_items;
      if (w < total) {
        int lo = 0, hi = n_items - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cum[mid] <= w) lo = mid;
          else hi = mid - 1;
        }
        cut.item = lo;
        cut.record = record(lo);
        const int size = cut.record.tiles + line.unit_cost;
        const long long in = w - cum[lo];
        cut.head = in < 0x7fffffffll ? (int)in / size : (int)(in / size);
        const int at = (int)(in - (long long)cut.head * size);
        cut.tile = max(0, at - line.unit_cost);
        if (cut.tile > 0) {
          const long long begin = w - cut.tile, end = w - at + size;  // its tiles
          cut.first = part_of(begin);
          cut.parts = part_of(end - 1) - cut.first + 1;
          if (cut.first == c - 1 && cut.parts >= line.join_from) joins[atomicAdd(&s_joins, 1)] = c;
        }
      }
      cuts[c] = cut;
    }
    __syncthreads();
  }
  if (t == 0) hdr->n_joins = s_joins;
}

}  // namespace

cudaError_t launch_span_plan(const SpanArgs& a, int lines, const SpanArgs* line0, const SpanArgs* line1, cudaStream_t s, bool seen) {
  PlanArgs p = {};
  p.a = a;
  // No questions, no pages: the kernel divides by n where there are pages (a test in the kernel costs 0.4 us a call)
  if (a.n == 0) p.a.pool_elem = 0;
  p.lines = lines;
  p.seen = lines > 0 || seen;
  // intervals, prefixes and first items of the questions, and beside them the largest of: the sort
  // keys, the bit map of the blocks, the tile counts of the items
  size_t area = 8;
  while (area < 8 * (size_t)a.n) area <<= 1;
  const size_t map = a.pool_elem ? ((size_t)a.n_blocks + 63) / 64 * 8 : 0;
  area = area > map ? area : map;
  for (int l = 0; l < lines; ++l) {
    const SpanArgs& x = l ? *line1 : *line0;
    const int item_tokens = x.tile_tokens * x.item_tiles;
    p.line[l] = {x.line, item_tokens, x.min_tokens, x.max_tokens, x.ctas, x.unit_cost, x.join_from};
    const int64_t items = (int64_t)a.T / item_tokens + a.n;
    const size_t cum = items < kCumSmem ? 8 * (size_t)items : 8 * kCumSmem;
    area = area > cum ? area : cum;
  }
  const size_t smem = 20 * (size_t)a.n + 24 + area;
  constexpr int kMost = 20 * kMaxQuestions + 24 + kSpanMaxBlocks / 8;
  static_assert(kMost <= 220 * 1024, "shared memory of the plan");
  // Few threads scan faster, many look at more pages at once.  Measured with 256 and 1024: 64 packed questions
  // 59.0 and 60.1 us, one question after 100 positions 10.5 and 11.7; 64 windowed decode steps over tables of 136
  // pages 40.0 and 36.4, 32 short ones 29.9 and 29.0
  const bool wide = a.n > 512 || (a.pool_elem && (int64_t)a.n * a.max_blocks > 512);
  auto kern = wide ? span_plan_kernel<1024> : span_plan_kernel<256>;
  if (smem > 40 * 1024) {  // always the same limit: calls from several threads do not lower each other's
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(1), dim3(wide ? 1024 : 256), smem, s, p);
}

}  // namespace kev
