// Shared pieces of the "span" operators: attention of each question's new tokens over the span of
// positions they see -- all earlier ones, or a sliding window and the first few (sinks) -- with
// keys and values in a paged cache or in the packed rows themselves, and the writes and reads of
// that cache (bf16, fp32 or e4m3 with one scale per row).
//
// Work.  Question i's L_i tokens sit at positions P_i .. P_i + L_i - 1.  A kv head's G q-heads
// read the same keys, so rows are (token, q-head of the group) pairs: a row tile holds
// floor(M / G) tokens of one question and one kv head, row = token * G + head.  An item is one or
// two row tiles of consecutive tokens; a unit is an item and a kv head; its keys are 128-position
// tiles: the tiles that hold sinks, then the tiles from the first token's window to the last
// token.  The plan kernel (kev_span_plan.cu) lays all units' key tiles end to end and cuts that
// line into equal parts, one per CTA, so every CTA does the same number of key tiles whatever the
// lengths; the units that a cut goes through are joined from partial results.
#pragma once

#include <cuda.h>

#include "kev_internal.cuh"

namespace kev {

constexpr int kSpanKeys = 128;     // positions per key tile: one page
constexpr int kSpanMaxCtas = 304;  // parts of the work line (2 CTAs on each of 152 SMs)
constexpr int kSpanRows = 16;      // rows of a unit in the kernel for few rows
constexpr int kSpanMaxBlocks = 1 << 20;  // pool blocks: the plan marks used blocks in a bit map in shared memory

struct SpanHeader {
  int32_t status;
  int32_t n_gaps;
  int32_t n_new;  // tokens in questions
  int32_t n_joins;
};

struct alignas(16) SpanItem {
  int32_t row0;      // packed row of its first token
  int32_t p0;        // that token's position
  int32_t tokens;    // its tokens
  int32_t tiles;     // key tiles they see
  int32_t question;
  int32_t pad[3];
};

// Cut c of the work line: the unit (item, kv head) and the key tile of it where part c begins, with
// the item's record beside them (a part begins with one load).  Where tile > 0 the cut is inside the
// unit: first = the part the unit begins in, parts = how many parts it has.
struct alignas(16) SpanCut {
  SpanItem record;
  int32_t item, head, tile, first, parts;
  int32_t pad[3];
};

// A work line in the workspace.
struct SpanLine {
  size_t items;    // SpanItem[max_items]
  size_t cum;      // int64[max_items + 1] key tiles (over all kv heads) before each item
  size_t cuts;     // SpanCut[kSpanMaxCtas + 1]
  size_t arrived;  // int32[kSpanMaxCtas][kSpanRows] finished pieces of the unit that begins in part c and goes on
  size_t joins;    // int32[kSpanMaxCtas] cuts of the units that the merge kernel joins
};

struct SpanLayout {
  size_t cu;       // int32[n + 1] prefix sums of the lengths, in question order
  size_t gaps;     // int2[n + 1] token ranges of no question
  SpanLine line[2];
  size_t part_ml;  // float2[2 * kSpanMaxCtas][rows] running maximum (log2 units) and sum
  size_t part_o;   // float[2 * kSpanMaxCtas][d / 8][rows][8] (few rows: [rows][d])
  size_t total;
  int32_t rows;    // rows of a partial result
  int64_t max_items;
};

// Rows of a unit in the kernels: 256 on the tensor cores (two 128-row tiles), 64 on the CUDA
// cores, 16 for a few rows.
inline SpanLayout span_layout(int32_t n, int32_t T, int32_t group, int32_t d) {
  SpanLayout L;
  const int64_t rows = (int64_t)T * group;
  L.rows = (int32_t)(rows > 224 ? 256 : (rows + 31) / 16 * 16);  // up to 11 rows lie unused between two tiles
  L.max_items = (int64_t)T / 4 + n + 1;  // an item holds at least 4 tokens or a question's last ones
  size_t off = align_up(sizeof(SpanHeader), 256);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.cu = take(sizeof(int32_t) * ((size_t)n + 1));
  L.gaps = take(sizeof(int2) * ((size_t)n + 1));
  for (SpanLine& l : L.line) {
    l.items = take(sizeof(SpanItem) * (size_t)L.max_items);
    l.cum = take(sizeof(int64_t) * ((size_t)L.max_items + 1));
    l.cuts = take(sizeof(SpanCut) * (kSpanMaxCtas + 1));
    l.arrived = take(sizeof(int32_t) * kSpanRows * kSpanMaxCtas);
    l.joins = take(sizeof(int32_t) * kSpanMaxCtas);
  }
  L.part_ml = take(sizeof(float2) * 2 * kSpanMaxCtas * (size_t)L.rows);
  L.part_o = take(sizeof(float) * 2 * kSpanMaxCtas * (size_t)L.rows * d);
  L.total = off;
  return L;
}

// Everything the span kernels take.
struct SpanArgs {
  const void* q;
  const void* k;  // packed new rows (the keys themselves without a cache)
  const void* v;
  void* out;
  const kev_interval* intervals;
  const int32_t* prefix;  // null: 0
  int32_t n, T;
  int32_t h_q, h_kv, group, d;
  int32_t elem;       // bytes of a q/k/v/out element: 2 bf16, 4 fp32
  int32_t pool_elem;  // bytes of a cached element: 0 no cache, 1 e4m3, 2 bf16, 4 fp32
  float scale;
  void* pool_k;
  void* pool_v;
  float* scale_k;
  float* scale_v;
  const int32_t* table;
  int32_t max_blocks, n_blocks;
  int32_t window, sinks;  // window 0: every earlier position
  int32_t max_chunk;      // no question has more tokens
  const int32_t* positions;  // rotation: each question's first position (null: its prefix)
  int32_t max_pos;           // and how many the angle table has (0: no rotation)
  // The work line of this launch: the questions of min_tokens .. max_tokens tokens
  SpanLine line;
  int32_t min_tokens, max_tokens;
  int32_t tile_rows;      // M: rows of a row tile (128, 64 or 16)
  int32_t tile_tokens;    // floor(M / group)
  int32_t item_tiles;     // row tiles of an item
  int32_t ctas;           // parts of the work line
  int32_t join_from;      // units of so many pieces or more are joined by the merge kernel
  int32_t unit_cost;      // what a unit costs beside its key tiles, in key tiles
  char* ws;
  SpanLayout layout;
  int32_t* dev_status;
};

// Norms, rotation and cache write in one pass (kev_norm_rope.cu): a.q, a.k, a.v with rows of any stride
struct NormRopeArgs {
  SpanArgs s;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  void* q_out;
  void* k_out;  // null: not wanted
  const void* q_weight;  // null: not normalised
  const void* k_weight;
  float eps;
  const float2* table;
};
cudaError_t launch_norm_rope(const NormRopeArgs& p, bool checked, int num_sms, cudaStream_t s);

// tensor maps (kev_span_tc.cu): `rank` dimensions, innermost first and contiguous, of `elem`-byte elements
bool span_tensor_map(CUtensorMap* m, const void* base, int elem, int rank, const cuuint64_t* dims, const cuuint32_t* box,
                     CUtensorMapSwizzle swizzle);
// The checks of a call, and the work lines of its attention launches: none for a cache write or read,
// or one or two (same call, other line) whose questions between them are all that have tokens.  seen: a call without
// lines reads every page that its tokens see (else only those that they are written to are looked at)
cudaError_t launch_span_plan(const SpanArgs& a, int lines, const SpanArgs* line0, const SpanArgs* line1, cudaStream_t s,
                             bool seen = false);
// checked: behind a plan; else a small call (span_small_copy), which checks for itself
bool span_small_copy(const SpanArgs& a);
cudaError_t launch_span_write(const SpanArgs& a, bool checked, int num_sms, cudaStream_t s);
cudaError_t launch_span_read(const SpanArgs& a, void* k_out, void* v_out, bool checked, int num_sms, cudaStream_t s);
cudaError_t launch_span_simt(const SpanArgs& a, cudaStream_t s);  // fp32
cudaError_t launch_span_tc(const SpanArgs& a, cudaStream_t s);    // bf16
cudaError_t launch_span_rows(const SpanArgs& a, bool write, cudaStream_t s);  // bf16, at most 16 rows a question
int span_rows_ctas(int d, int rows);  // CTAs per SM of that kernel for 8 or 16 rows
cudaError_t launch_span_merge(const SpanArgs& a, int num_sms, cudaStream_t s);

// Key tiles of tokens at positions p0 .. p1: tile j holds positions 128 * at(j) ...
struct SpanTiles {
  int ns, lo, n;  // sink tiles 0 .. ns - 1, then tiles lo .. lo + n - ns - 1
  __host__ __device__ SpanTiles(int p0, int p1, int window, int sinks) {
    lo = window > 0 && p0 >= window ? (p0 - window + 1) / kSpanKeys : 0;
    const int s = (int)(((int64_t)sinks + kSpanKeys - 1) / kSpanKeys);
    ns = s < lo ? s : lo;
    n = ns + p1 / kSpanKeys - lo + 1;
  }
  __host__ __device__ int at(int j) const { return j < ns ? j : lo + (j - ns); }
};

// The units of part `part` of the work line, one after the other: unit (item, head) and its key
// tiles [j0, j1).  The next item's record is loaded while the current one is worked on.
struct SpanWalk {
  const SpanItem* items;
  SpanItem item, ahead;
  SpanCut to;
  int from_first, from_parts, it, head, h_kv, j0, j1;
  __device__ __forceinline__ SpanWalk(const SpanArgs& a, int part) {
    items = reinterpret_cast<const SpanItem*>(a.ws + a.line.items);
    const SpanCut* cuts = reinterpret_cast<const SpanCut*>(a.ws + a.line.cuts);
    const SpanCut from = cuts[part];
    to = cuts[part + 1];
    from_first = from.first;
    from_parts = from.parts;
    it = from.item;
    head = from.head;
    h_kv = a.h_kv;
    j0 = from.tile;
    if (live()) {
      item = from.record;
      if (it < to.item) ahead = items[it + 1];  // one record past the last item is laid out
      j1 = last();
    }
  }
  __device__ __forceinline__ int last() const { return it == to.item && head == to.head ? to.tile : item.tiles; }
  __device__ __forceinline__ bool live() const {
    return it < to.item || (it == to.item && (head < to.head || (head == to.head && j0 < to.tile)));
  }
  __device__ __forceinline__ bool ends() const {  // the part's last unit
    return it == to.item ? head == to.head || (to.tile == 0 && head + 1 == to.head)
                         : to.tile == 0 && to.head == 0 && it + 1 == to.item && head + 1 == h_kv;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == item.tiles; }
  // slot of this unit's partial result: the unit began in an earlier part, or ends in a later one
  __device__ __forceinline__ int64_t slot(int part) const { return 2 * (int64_t)part + (j0 == 0); }
  // the unit's pieces: the part it begins in, and how many
  __device__ __forceinline__ int first() const { return j0 ? from_first : to.first; }
  __device__ __forceinline__ int parts() const { return j0 ? from_parts : to.parts; }
  __device__ __forceinline__ void next() {
    j0 = 0;
    if (++head == h_kv) {
      head = 0;
      ++it;
      item = ahead;
      if (it < to.item) ahead = items[it + 1];
    }
    j1 = last();
  }
};

// Place of elements 8 c .. 8 c + 7 of a row in the partial results (neighbouring rows side by side).
__device__ __forceinline__ int64_t span_part(const SpanArgs& a, int64_t slot, int c, int row) {
  return ((slot * (a.d / 8) + c) * a.layout.rows + row) * 8;
}

// A row's quantisation: scale = top / 448 (a NaN for a row that holds a NaN or an infinity), and its
// elements' quotients x / scale, both the correctly rounded ones.  The quotients take the residual
// correction of Markstein (1990): with r the correctly rounded reciprocal and q = x r, the fused
// q + (x - q scale) r is the correctly rounded quotient -- as long as the residual is exact, so far
// from the subnormals; smaller scales divide.  (The divisions were three quarters of the write's
// instructions.)
__device__ __forceinline__ float span_scale(float top) {
  if (top >= 7.8886091e-31f && top < INFINITY) {  // 2^-100
    const float r = 1.f / 448.f, q = top * r;
    return fmaf(fmaf(-q, 448.f, top), r, q);
  }
  return top < INFINITY ? __fdiv_rn(top, 448.f) : __int_as_float(0x7fffffff);
}
template <int N>
__device__ __forceinline__ void span_quotients(float (&f)[N], float scale) {
  if (scale >= 8.2718061e-25f) {  // 2^-80
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float q = f[e] * r;
      f[e] = fmaf(fmaf(-q, scale, f[e]), r, q);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = scale == 0.f ? 0.f : __fdiv_rn(f[e], scale);
  }
}

// Errors of device data by rank -- intervals, prefix, overflow, slot, position: the first that applies is
// reported -- as 8 - rank in a word that starts at 0, and the status of that word.
__device__ __forceinline__ int span_code(int err) {
  const int rank = 8 - err;
  return err == 0 ? ST_OK : rank == 0 ? ST_INTERVALS : rank == 1 ? ST_PREFIX : rank == 2 ? ST_OVERFLOW : rank == 3 ? ST_SLOT : ST_POSITION;
}
// Are the positions of question i's L new tokens, cached from `prefix` on, rows of the angle table?
__device__ __forceinline__ bool span_positions(const SpanArgs& a, int i, int prefix, int L) {
  if (a.max_pos == 0) return true;
  const int first = a.positions ? a.positions[i] : prefix;
  return first >= 0 && (int64_t)first + L <= a.max_pos;
}

// Small calls: every CTA makes the plan's checks (kev_span_plan.cu) for itself and comes to the same verdict,
// so none has to wait for another.  Overlapping intervals show as a token that is marked twice; the mark is
// also the token's question.
constexpr int kSpanSmall = 512;  // tokens and questions of a small call at most, and threads of its kernels
struct SpanSmall {
  int2 iv[kSpanSmall];
  int prefix[kSpanSmall], owner[kSpanSmall], err;
};
// Before the launch's inputs are ready: shared memory cleared (`used`: a bit per block of the pool).
__device__ __forceinline__ void span_small_clear(const SpanArgs& a, SpanSmall& sm, unsigned* used) {
  const int words = a.pool_elem ? (a.n_blocks + 31) / 32 : 0, t = threadIdx.x;
  if (t == 0) sm.err = 0;
  for (int i = t; i < words; i += kSpanSmall) used[i] = 0u;
  for (int i = t; i < a.T; i += kSpanSmall) sm.owner[i] = -1;
}
// The checks, by kSpanSmall threads that have passed a barrier since the clearing; true: the call is valid.
__device__ __forceinline__ bool span_small_check(const SpanArgs& a, SpanSmall& sm, unsigned* used) {
  const int t = threadIdx.x, warp = t / 32, lane = t & 31;
  auto error = [&](int rank) { atomicMax(&sm.err, 8 - rank); };
  for (int i = t; i < a.n; i += kSpanSmall) {
    const kev_interval v = a.intervals[i];
    const int first = a.prefix ? a.prefix[i] : 0;
    sm.iv[i] = make_int2(v.begin, v.end);
    sm.prefix[i] = first;
    if (v.begin < 0 || v.end < v.begin || v.end > a.T) {
      error(0);
    } else if (v.end > v.begin) {
      if (first < 0) error(1);
      else if (a.pool_elem && (int64_t)first + (v.end - v.begin) > (int64_t)a.max_blocks * kPage) error(2);
      if (!span_positions(a, i, first, v.end - v.begin)) error(4);
    }
  }
  __syncthreads();
  // clean: the checks of single questions passed (positions are no one's address yet); inside: every interval at least
  const bool clean = sm.err <= 4, inside = sm.err != 8;
  __syncthreads();
  if (clean && a.pool_elem) {
    for (int i = t; i < a.n; i += kSpanSmall) {  // pages; a block's bit may be set once
      const int L = sm.iv[i].y - sm.iv[i].x;
      if (L <= 0) continue;
      for (int e = sm.prefix[i] / kPage; e <= (sm.prefix[i] + L - 1) / kPage; ++e) {
        const int b = a.table[(int64_t)i * a.max_blocks + e];
        const unsigned bit = 1u << (b & 31);
        if (b < 0 || b >= a.n_blocks || atomicOr(&used[b >> 5], bit) & bit) error(3);
      }
    }
  }
  if (inside) {
    for (int i = warp; i < a.n; i += kSpanSmall / 32)
      for (int x = sm.iv[i].x + lane; x < sm.iv[i].y; x += 32)
        if (atomicExch(&sm.owner[x], i) >= 0) error(0);
  }
  __syncthreads();
  if (blockIdx.x == 0 && t == 0 && a.dev_status) *a.dev_status = span_code(sm.err);
  return sm.err == 0;
}

// Is position u visible to the token at position p?
__device__ __forceinline__ bool span_sees(int p, int u, int window, int sinks) {
  return u <= p && (window == 0 || p - u < window || u < sinks);
}

// Rows of tokens in no question are zero: the calling CTA's share, by its first `threads` threads.
__device__ __forceinline__ void span_zero_gaps(const SpanArgs& a, int threads) {
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  const int2* gaps = reinterpret_cast<const int2*>(a.ws + a.layout.gaps);
  const int64_t vec = (int64_t)a.h_q * a.d * a.elem / 16;
  uint4* out = static_cast<uint4*>(a.out);
  for (int i = 0; i < h->n_gaps; ++i) {
    const int2 g = gaps[i];
    for (int64_t x = g.x * vec + (int64_t)blockIdx.x * threads + threadIdx.x; x < g.y * vec; x += (int64_t)gridDim.x * threads)
      out[x] = make_uint4(0u, 0u, 0u, 0u);
  }
}

}  // namespace kev
