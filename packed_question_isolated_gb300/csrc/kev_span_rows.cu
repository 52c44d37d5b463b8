// Span attention for a few rows per question -- above all decode steps: bf16 q and out, paged cache
// bf16 or e4m3, at most 16 (token, q-head of the group) rows per question and kv head.
//
// Every cached row is read once and meets only those rows, so the bound is HBM (the cache, once)
// and below it the instructions per element that unpack it: e4m3 codes become fp16 (one conversion
// per two; as bf16 it takes four integer operations), and q and the weights fp16 with scales of
// their own.  Here the matrix instruction takes the
// cache as its A operand straight from registers (mma.sync m16n8k16): S^T[16 keys x 8 rows] = K q^T,
// O^T[dims x 8 rows] += V^T P^T.  With 8 rows nothing is padded, where tcgen05 would spend a 128-row
// tile (or an extra trip of the unpacked codes through shared memory, which at HBM speed is more than
// shared memory carries); the matrix pipe stays below half its time.
//
// One or two persistent CTAs per SM walk their equal parts of the work line (kev_span.cuh):
//   warp 8      loads pages into a ring: TMA boxes of 16 positions, only those that some row sees
//   warps 0-7   a warp takes 16 of a page's 128 positions, with a running reference maximum, sum and
//               accumulator of its own, which it leaves in shared memory when the unit ends
//               A warp that comes to positions of the chunk itself puts their K/V rows into the loaded page
//   warp 9      prepares those rows, up to two units ahead: from the inputs, quantised for e4m3, into the
//               cache and into shared memory.  Every (unit, tile) has one owner, so a row is written
//               once, and nobody waits for the write.  Between that it joins the eight warps' results
//               while they work on the next unit, and the pieces of a unit that a cut goes through, if
//               its own piece is the last one done -- in the order of the pieces, so the result does not
//               depend on which CTA that is
//
// Measured on a GB300: decode of 16 bf16 caches of 2 to 32 Ki positions 116 us (5.7 TB/s, 84 % of the
// measured copy rate); 32 e4m3 caches of 64 to 2400 positions 29 us and 64 windowed ones (1024 positions, 4
// sinks) 37 us, of which the plan is 5 to 7, the first page 4 and the last unit's joins 4: with 10 to 17
// pages per SM these are most of it.  16 long e4m3 caches take 84 us (4.0 TB/s, 59 %): there the conversions, one
// per two codes, are the likely bound.  Measured and left: 8 warps with tcgen05-shaped 128-row tiles (the
// tensor-core kernel: 78 us for the 32 caches); codes widened to bf16 by integer operations (94 us against
// 82 for 16 long caches); the joins by the warps that compute (31.9 against 31.2); the new rows written by a
// warp of their own before their pages are loaded (33 against 31).
//
// Registers instead of ldmatrix: the contraction index of an MMA may be permuted freely, so a lane
// takes whole 16-byte chunks of a row (8 bf16 or 16 codes) as its share of several k-steps.  For K,
// lane (g, c) of group g = lane / 4 holds chunks c, c + 4, ... of the row of key slot g; for V, chunk g
// of the rows of slots 2c, 2c + 1, 2c + 8, 2c + 9, byte-permuted into (key, key) pairs.  Slot s is
// position perm(s) of its 8, chosen so that with the 128-byte swizzle a quarter warp's 16-byte loads
// of either kind touch all banks once.
#include "kev_sm100.cuh"
#include "kev_span.cuh"

namespace kev {
namespace {

using namespace sm100;

constexpr int kWarps = 8;  // of 16 positions each: a page
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kLoadWarp = kWarps, kJoinWarp = kWarps + 1;
constexpr float kBig = 1.8446744e19f;  // 2^64: a weight above it moves the reference
constexpr long long kDrainBudget = 4000000000ll;

// CTAs per SM.  Two, so that one's beginnings and ends of units lie beside the other's streaming, where
// registers and pages are small: d = 64 with 8 rows (32 bf16 caches of 2 to 32 Ki positions 146 us against
// 159 with one).  At d = 128 one, with every register and three to five pages in flight: 16 such bf16 caches
// 115 us against 121, e4m3 decode of 32 short ones 29.2 against 31.1 (of 16 long ones 84.7 against 81.8).
constexpr int few_rows_ctas(int d, int tiles) { return tiles == 1 && d == 64 ? 2 : 1; }

template <int D, int E, int NT>
struct Smem {
  static constexpr int kCtas = few_rows_ctas(D, NT);     // per SM
  static constexpr int kRow = D * E;                        // bytes of a cached row
  static constexpr int kPitch = kRow < 128 ? kRow : 128;    // row of a swizzled sub-tile
  static constexpr int kSubs = kRow / kPitch;
  static constexpr int kTile = kPage * kRow;                // K or V of a stage
  static constexpr int kScales = E == 1 ? 2 * kPage * 4 : 0;
  static constexpr int kStageBytes = 2 * kTile + (kScales + 1023) / 1024 * 1024;
  static constexpr int kPad = D + 4;                        // floats of a row in the join buffer
  static constexpr int kJoinBytes = kWarps * 8 * kPad * 4;  // float [8 warps][8 rows][kPad]
  static constexpr int kQPitch = 2 * D + 16;                // bytes of a staged q row
  static constexpr int kQBytes = NT * 8 * kQPitch;          // q rows of a unit
  static constexpr int kNewRows = NT * 8;                   // new tokens of a unit at most
  static constexpr int kNewBytes = kNewRows * (2 * kRow + 16);  // their K and V rows and scales
  static constexpr int kRoom =
      (kCtas == 2 ? 113 * 1024 : 226 * 1024) - 2048 - kJoinBytes - kWarps * 64 - 2 * kQBytes - 2 * kNewBytes;
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static constexpr int kJoin = kStages * kStageBytes;
  static constexpr int kMl = kJoin + kJoinBytes;            // float2 [8 warps][8 rows]
  static constexpr int kQ = kMl + kWarps * 64;              // two units' q rows
  static constexpr int kNew = kQ + 2 * kQBytes;             // two units' new rows
  static constexpr int kBar = kNew + 2 * kNewBytes;
  static constexpr int kBytes = kBar + 256 + 1024;
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_full[2], q_empty[2];
  uint64_t new_full[2], new_empty[2];
  uint64_t join_full, join_empty;
  uint64_t stall;        // timeout test hook: nothing ever arrives on it
  uint64_t join_empty8;  // the last unit's first 8 rows are joined
  int abort;
  int never;
};
static_assert(sizeof(Bars) <= 256, "barriers");

struct RowsArgs {
  SpanArgs s;
  float scale_log2;
  long long wait_budget;
  int32_t write;
  int32_t test_stall;  // timeout test hook
};

__device__ __forceinline__ int perm(int s) {  // position of slot s: 0 5 2 7 4 1 6 3
  return s & 1 ? (s ^ 4) : s;
}

// D += A B, bf16 (E = 2) or fp16 (E = 1) operands
template <int E>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if (E == 2)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
  return x;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at));
  return x;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 x;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at));
  return x;
}

// two e4m3 codes (the low or high half of w) as fp16, which holds every one of them exactly
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Some row of the item (tokens at p0 .. p1) sees one of positions u .. u + 15.
__device__ __forceinline__ bool group_seen(const SpanArgs& a, int u, int p0, int p1) {
  return u <= p1 && (a.window == 0 || p0 - (u + 15) < a.window || u < a.sinks);
}

// A row of the output: D / 32 consecutive dims per lane.
template <int D>
__device__ __forceinline__ void store_row(const SpanArgs& a, const SpanItem& w, int head, int row, const float (&o)[D / 32],
                                          float sum) {
  constexpr int kD = D / 32;
  const float inv = 1.f / sum;
  uint32_t x[kD / 2];
#pragma unroll
  for (int e = 0; e < kD; e += 2) x[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      static_cast<__nv_bfloat16*>(a.out) +
      ((int64_t)(w.row0 + row / a.group) * a.h_q + head * a.group + row % a.group) * D + (threadIdx.x & 31) * kD);
  if (kD == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(x[0], x[kD / 2 - 1]);
  else *dst = x[0];
}

// The pieces of a row of a unit, joined by a warp.
template <int D>
__device__ __forceinline__ void join_pieces(const SpanArgs& a, const SpanItem& w, int head, int row, int first, int parts) {
  constexpr int kD = D / 32;
  const int lane = threadIdx.x & 31;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + a.layout.part_ml);
  const float* po = reinterpret_cast<const float*>(a.ws + a.layout.part_o);
  auto piece = [&](int i) { return (2 * (int64_t)(first + i) + (i == 0)) * a.layout.rows + row; };
  float top = -INFINITY;
  for (int i = lane; i < parts; i += 32) top = fmaxf(top, __ldcg(ml + piece(i)).x);
  top = warp_max(top);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[kD] = {};
#pragma unroll 4
  for (int i = 0; i < parts; ++i) {
    const float2 y = __ldcg(ml + piece(i));
    const float f = ex2_approx(y.x - ref);
    sum = fmaf(y.y, f, sum);
#pragma unroll
    for (int e = 0; e < kD; e += 2) {
      const float2 x = __ldcg(reinterpret_cast<const float2*>(po + piece(i) * D + lane * kD + e));
      acc[e] = fmaf(x.x, f, acc[e]);
      acc[e + 1] = fmaf(x.y, f, acc[e + 1]);
    }
  }
  store_row<D>(a, w, head, row, acc, sum);
}

// Row r of the eight warps' results in the join buffer, by a warp: D / 32 consecutive dims per lane.
template <int D, int E>
__device__ __forceinline__ void join_warps(const float* join, const float2* join_ml, int r, float (&acc)[D / 32], float& top,
                                           float& sum) {
  constexpr int kD = D / 32, kPad = D + 4;
  const int lane = threadIdx.x & 31;
  float2 y[kWarps];
  top = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < kD; ++e) acc[e] = 0.f;
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    y[v] = join_ml[v * 8 + r];
    top = fmaxf(top, y[v].x);
  }
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int v = 0; v < kWarps; ++v) {
    const float f = ex2_approx(y[v].x - ref);
    sum = fmaf(y[v].y, f, sum);
#pragma unroll
    for (int e = 0; e < kD; e += 2) {
      const int dim = lane * kD + e;  // held by group g in its tile mt
      const int g = E == 1 ? dim / (D / 8) : dim / 8 % 8, mt = E == 1 ? dim % (D / 8) / 2 : dim / 64 * 4 + dim % 8 / 2;
      const float2 z = *reinterpret_cast<const float2*>(join + (v * 8 + r) * kPad + mt * 16 + 2 * g);
      acc[e] = fmaf(z.x, f, acc[e]);
      acc[e + 1] = fmaf(z.y, f, acc[e + 1]);
    }
  }
}

template <int D>
__device__ __forceinline__ void store_piece(const SpanArgs& a, int64_t slot, const float (&acc)[D / 32], float top, float sum) {
  const int lane = threadIdx.x & 31;
  float* dst = reinterpret_cast<float*>(a.ws + a.layout.part_o) + slot * D + lane * (D / 32);
#pragma unroll
  for (int e = 0; e < D / 32; e += 2) *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e], acc[e + 1]);
  if (lane == 0) reinterpret_cast<float2*>(a.ws + a.layout.part_ml)[slot] = make_float2(top, sum);
}

template <int D, int E, int NT>
__global__ void __launch_bounds__(kThreads, few_rows_ctas(D, NT))
    span_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ RowsArgs p) {
  using L = Smem<D, E, NT>;
  const SpanArgs& a = p.s;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], kWarps);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&bars->q_full[u], 1);
      mbar_init(&bars->q_empty[u], kWarps);
      mbar_init(&bars->new_full[u], 1);
      mbar_init(&bars->new_empty[u], kWarps);
    }
    mbar_init(&bars->join_full, kWarps);
    mbar_init(&bars->join_empty, 1);
    mbar_init(&bars->join_empty8, kWarps);
    mbar_init(&bars->stall, 1);
    bars->abort = bars->never = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == kLoadWarp * 32) {
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  volatile int* abort_flag = &bars->abort;
  const volatile int* never = &bars->never;
  const long long budget = p.wait_budget;
  pdl_wait();
  pdl_trigger();
  if (reinterpret_cast<const SpanHeader*>(a.ws)->status != ST_OK) return;
  float* join = reinterpret_cast<float*>(smem + L::kJoin);
  float2* join_ml = reinterpret_cast<float2*>(smem + L::kMl);
  auto timeout = [&]() {
    atomicCAS(&reinterpret_cast<SpanHeader*>(a.ws)->status, 0, ST_TIMEOUT);
    set_status(a.dev_status, ST_TIMEOUT);
    *abort_flag = 1;
  };

  if (warp == kLoadWarp) {
    // -------------------------------------------------------------------- page loads
    constexpr int kBoxes = 2 * L::kSubs * kWarps;  // 16-position boxes of a page: one per lane
    const int is_v = lane / (kBoxes / 2), sub = lane / kWarps % L::kSubs, grp = lane % kWarps;
    uint32_t seq = 0, n = 0;
    bool ok = !(p.test_stall && blockIdx.x == 0) ||
              __all_sync(0xffffffffu, mbar_wait(&bars->stall, 0, abort_flag, budget));
    for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next()) {
      const int p0 = w.item.p0, p1 = p0 + w.item.tokens - 1, rows = w.item.tokens * a.group;
      const SpanTiles tiles(p0, p1, a.window, a.sinks);
      const int32_t* row = a.table + (int64_t)w.item.question * a.max_blocks;
      int ids = 0;
      if (n >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_empty[n & 1], (n / 2 - 1) & 1, abort_flag, budget));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&bars->q_full[n & 1], rows * 2 * D);
      __syncwarp();
      if (lane < rows)
        bulk_load(smem + L::kQ + (n & 1) * L::kQBytes + lane * L::kQPitch,
                  static_cast<const __nv_bfloat16*>(a.q) +
                      ((int64_t)(w.item.row0 + lane / a.group) * a.h_q + w.head * a.group + lane % a.group) * D,
                  2 * D, &bars->q_full[n & 1]);
      ++n;
      for (int j = w.j0; ok && j < w.j1; ++j) {
        if ((j - w.j0) % 32 == 0) ids = j + lane < w.j1 ? row[tiles.at(j + lane)] : 0;  // 32 pages ahead
        const int block = __shfl_sync(0xffffffffu, ids, (j - w.j0) % 32);
        const int u0 = tiles.at(j) * kPage;
        const int s = seq % L::kStages;
        if (seq >= L::kStages)
          ok = __all_sync(0xffffffffu, mbar_wait(&bars->empty[s], (seq / L::kStages - 1) & 1, abort_flag, budget));
        if (!ok) break;
        const bool mine = lane < kBoxes && group_seen(a, u0 + grp * 16, p0, p1);
        const int boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const int cell = (block * a.h_kv + w.head) * kPage;
        unsigned char* dst = smem + s * L::kStageBytes;
        if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], boxes * 16 * L::kPitch + L::kScales);
        __syncwarp();
        if (mine)
          tma_load_2d(dst + is_v * L::kTile + (sub * kPage + grp * 16) * L::kPitch, is_v ? &tm_v : &tm_k, sub * L::kPitch / E,
                      cell + grp * 16, &bars->full[s]);
        if (E == 1 && lane < 2)
          bulk_load(dst + 2 * L::kTile + lane * kPage * 4, (lane ? a.scale_v : a.scale_k) + cell, kPage * 4, &bars->full[s]);
        ++seq;
      }
    }
    if (!ok && lane == 0) timeout();
    if (*abort_flag) {  // every copy issued lands before the CTA leaves
      for (uint32_t u = n < 2 ? 0 : n - 2; u < n; ++u) mbar_wait(&bars->q_full[u & 1], (u / 2) & 1, never, kDrainBudget);
      for (uint32_t q = seq < L::kStages ? 0 : seq - L::kStages; q < seq; ++q)
        mbar_wait(&bars->full[q % L::kStages], (q / L::kStages) & 1, never, kDrainBudget);
    }
  } else if (warp == kJoinWarp) {
    // -------------------------------------------------------------------- new rows
    bool ok = true;
    uint32_t made = 0;
    SpanWalk ahead(a, blockIdx.x);
    auto new_rows = [&]() {  // of the next unit
      if (!p.write || !ok || !ahead.live()) return;
      if (made >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&bars->new_empty[made & 1], (made / 2 - 1) & 1, abort_flag, budget));
      if (!ok) return;
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes of a bf16 row
      const int sub = lane % kLanes, p0 = ahead.item.p0, tokens = ahead.item.tokens;
      const SpanTiles tiles(p0, p0 + tokens - 1, a.window, a.sinks);
      const int32_t* row = a.table + (int64_t)ahead.item.question * a.max_blocks;
      unsigned char* base = smem + L::kNew + (made & 1) * L::kNewBytes;
      for (int x0 = 0; x0 < 2 * tokens; x0 += kAtOnce) {
        const int x = x0 + lane / kLanes, token = x >> 1, pos = p0 + token, is_v = x & 1;
        const int j = tiles.ns + pos / kPage - tiles.lo;  // its tile of the unit
        const bool mine = token < tokens && j >= ahead.j0 && j < ahead.j1;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        int64_t cell = 0;
        if (mine) {
          v = reinterpret_cast<const uint4*>(is_v ? a.v : a.k)[((int64_t)(ahead.item.row0 + token) * a.h_kv + ahead.head) * kLanes + sub];
          cell = ((int64_t)row[pos / kPage] * a.h_kv + ahead.head) * kPage + pos % kPage;
        }
        unsigned char* here = base + x * L::kRow;  // [token][K, V][kRow]
        unsigned char* dst = static_cast<unsigned char*>(is_v ? a.pool_v : a.pool_k) + cell * L::kRow;
        if (E == 2) {
          if (mine) {
            reinterpret_cast<uint4*>(here)[sub] = v;
            reinterpret_cast<uint4*>(dst)[sub] = v;
          }
        } else {
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
          float f[8], top = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] = __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
            top = nan_max(top, fabsf(f[e]));
          }
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float scale = span_scale(top);
          span_quotients(f, scale);
          const uint2 code = make_uint2(e4m3x2(f[0], f[1]) | e4m3x2(f[2], f[3]) << 16, e4m3x2(f[4], f[5]) | e4m3x2(f[6], f[7]) << 16);
          if (mine) {
            reinterpret_cast<uint2*>(here)[sub] = code;
            reinterpret_cast<uint2*>(dst)[sub] = code;
            if (sub == 0) {
              reinterpret_cast<float*>(base + 2 * L::kNewRows * L::kRow)[x] = scale;
              (is_v ? a.scale_v : a.scale_k)[cell] = scale;
            }
          }
        }
      }
      mbar_arrive_warp(&bars->new_full[made & 1]);
      ++made;
      ahead.next();
    };
    new_rows();
    new_rows();

    // -------------------------------------------------------------------- joins, of all units but the last
    uint32_t joins = 0;
    for (SpanWalk w(a, blockIdx.x); ok && w.live() && !w.ends(); w.next()) {
      const int rows = w.item.tokens * a.group;
      const bool whole = w.whole();
      const int64_t slot = w.slot(blockIdx.x) * a.layout.rows;
      for (int nt = 0; nt < NT; ++nt, ++joins) {
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->join_full, joins & 1, abort_flag, budget)))) break;
#pragma unroll 2
        for (int r = 0; r < 8; ++r) {
          if (nt * 8 + r >= rows) break;
          float acc[D / 32], top, sum;
          join_warps<D, E>(join, join_ml, r, acc, top, sum);
          if (whole) store_row<D>(a, w.item, w.head, nt * 8 + r, acc, sum);
          else store_piece<D>(a, slot + nt * 8 + r, acc, top, sum);
        }
        mbar_arrive_warp(&bars->join_empty);
      }
      if (ok && !whole) {  // the warp that finishes a row's last piece joins them all, in their order
        const int first = w.first(), parts = w.parts();
        int32_t* arrived = reinterpret_cast<int32_t*>(a.ws + a.line.arrived) + first * kSpanRows;
        __threadfence();
        __syncwarp();
        uint32_t all = __ballot_sync(0xffffffffu, lane < rows && atomicAdd(arrived + min(lane, kSpanRows - 1), lane < rows) == parts - 1);
        __threadfence();
        for (; all; all &= all - 1) join_pieces<D>(a, w.item, w.head, __ffs(all) - 1, first, parts);
      }
      new_rows();
    }
    if (!ok && lane == 0) timeout();
  } else {
    // -------------------------------------------------------------------- attention
    span_zero_gaps(a, kWarps * 32);
    constexpr int kChunks = L::kRow / 64;      // 16-byte chunks of a K row per lane
    constexpr int kSteps = E == 2 ? 2 : 4;     // k-steps of a chunk
    constexpr int kTiles = D / 16;             // 16-dim tiles of O^T
    const int g = lane >> 2, c = lane & 3;
    const uint32_t smem0 = smem_u32(smem);
    // swizzled address of 16-byte chunk ch of row r
    auto at = [&](uint32_t tile, int r, int ch) {
      if (L::kPitch == 128)
        return tile + (ch >> 3) * (kPage * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
      return tile + r * 64 + ((ch ^ (r >> 1 & 3)) << 4);
    };
    uint32_t seq = 0, n = 0, joins = 0;
    bool ok = true;
    for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next()) {
      const int p0 = w.item.p0, p1 = p0 + w.item.tokens - 1, rows = w.item.tokens * a.group;
      const SpanTiles tiles(p0, p1, a.window, a.sinks);
      // q as the B operand: row nt * 8 + g, the dims of this lane's chunks
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->q_full[n & 1], (n / 2) & 1, abort_flag, budget)))) break;
      uint32_t q[NT][kChunks * kSteps][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
        const uint32_t src = smem0 + L::kQ + (n & 1) * L::kQBytes + r * L::kQPitch;
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
          for (int h = 0; h < kSteps; ++h) {
            const int dim = (E == 2 ? 8 : 16) * (c + 4 * i) + 4 * h;
            const uint2 x = r < rows ? lds64(src + 2 * dim) : make_uint2(0u, 0u);
            q[nt][i * kSteps + h][0] = x.x;
            q[nt][i * kSteps + h][1] = x.y;
          }
      }
      mbar_arrive_warp(&bars->q_empty[n & 1]);
      ++n;
      // fp16 has no exponents to spare: a row of q is scaled by a power of two that puts its largest element
      // in [2^14, 2^15) -- exact down to 2^-29 of it, and off by at most 2^-40 of it below -- and the
      // scores by its inverse; or by 2^126, the largest that has an inverse, which is exact for every element of
      // the rows below 2^-112 that it is left to
      float q_inv[NT][2];
      if (E == 1) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < kChunks * kSteps; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              top = max(top, max(q[nt][i][x] & 0x7fffu, q[nt][i][x] >> 16 & 0x7fffu));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int up = min(127 + 14 - (int)(top >> 7), 126);  // 2^up; 14 - (exponent - 127)
          const float mul = __int_as_float((127 + up) << 23);
#pragma unroll
          for (int i = 0; i < kChunks * kSteps; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              q[nt][i][x] = pack_f16x2(__uint_as_float(q[nt][i][x] << 16) * mul, __uint_as_float(q[nt][i][x] & 0xffff0000u) * mul);
          const float inv = __int_as_float((127 - up) << 23);  // of row g: rows 2c, 2c + 1 are other lanes'
          q_inv[nt][0] = __shfl_sync(0xffffffffu, inv, 8 * c) * p.scale_log2;
          q_inv[nt][1] = __shfl_sync(0xffffffffu, inv, 8 * c + 4) * p.scale_log2;
        }
      }
      int pos[NT][2];  // positions of rows nt * 8 + 2c, + 1
      float m[NT][2], l[NT][2], o[kTiles][NT][4];
      float per[NT][2];  // e4m3: O is in units of 1 / per (below); 0: none yet
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pos[nt][x] = min(p0 + (nt * 8 + 2 * c + x) / a.group, p1);  // rows past the last: as its own
          m[nt][x] = -INFINITY;
          l[nt][x] = per[nt][x] = 0.f;
        }
#pragma unroll
      for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[mt][nt][x] = 0.f;

      for (int j = w.j0; j < w.j1; ++j, ++seq) {
        const int s = seq % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->full[s], (seq / L::kStages) & 1, abort_flag, budget));
        if (!ok) break;
        const int k0 = warp * 16, u0 = tiles.at(j) * kPage + k0;  // this warp's 16 positions
        if (group_seen(a, u0, p0, p1)) {
          const uint32_t tk = smem0 + s * L::kStageBytes, tv = tk + L::kTile;
          if (p.write && u0 + 15 >= p0) {  // positions of the chunk among them: their rows, from shared memory
            const uint32_t from = (n - 1) & 1;
            ok = __all_sync(0xffffffffu, mbar_wait(&bars->new_full[from], ((n - 1) / 2) & 1, abort_flag, budget));
            if (!ok) break;
            const uint32_t rows0 = smem0 + L::kNew + from * L::kNewBytes;
            constexpr int kWords = L::kRow / 16;  // 16-byte chunks of a row; lanes beyond K's and V's have none
#pragma unroll 1
            for (int t = max(0, u0 - p0); t < w.item.tokens && p0 + t < u0 + 16; ++t) {
              const int r = k0 + p0 + t - u0;
              if (lane < 2 * kWords) {
                const uint4 x = lds128(rows0 + (2 * t) * L::kRow + lane * 16);
                st_shared_v4(at(lane < kWords ? tk : tv, r, lane % kWords), x.x, x.y, x.z, x.w);
              }
              if (E == 1 && lane < 2) {
                const float x = lds32(rows0 + 2 * L::kNewRows * L::kRow + (2 * t + lane) * 4);
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(tk + 2 * L::kTile + (lane * kPage + r) * 4), "f"(x) : "memory");
              }
            }
            __syncwarp();
            fence_proxy_async_smem();  // before the slot's next load
          }
          const int r0 = k0 + perm(g);  // slots g and g + 8
          float z[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) z[nt][x] = 0.f;
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            const uint4 x = lds128(at(tk, r0, c + 4 * i)), y = lds128(at(tk, r0 + 8, c + 4 * i));
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int h = 0; h < kSteps; ++h) {
              uint32_t a0, a1, a2, a3;
              if (E == 2) {
                a0 = xs[(2 * h) & 3];
                a1 = ys[(2 * h) & 3];
                a2 = xs[(2 * h + 1) & 3];
                a3 = ys[(2 * h + 1) & 3];
              } else {
                a0 = widen_lo(xs[h & 3]);
                a1 = widen_lo(ys[h & 3]);
                a2 = widen_hi(xs[h & 3]);
                a3 = widen_hi(ys[h & 3]);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma<E>(z[nt], a0, a1, a2, a3, q[nt][i * kSteps + h][0], q[nt][i * kSteps + h][1]);
            }
          }
          float kf0 = p.scale_log2, kf1 = kf0, vf0 = 1.f, vf1 = 1.f;
          if (E == 1) {
            const uint32_t sc = tk + 2 * L::kTile + r0 * 4;
            kf0 = lds32(sc);
            kf1 = lds32(sc + 32);
            vf0 = lds32(sc + kPage * 4);
            vf1 = lds32(sc + kPage * 4 + 32);
          }
          // every row sees all 16 positions
          const bool edge = !(u0 + 15 <= p0 && (a.window == 0 || p1 - u0 < a.window || u0 + 15 < a.sinks));
          const int key0 = u0 + perm(g), key1 = key0 + 8;
          bool unset = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              z[nt][x] *= E == 1 ? kf0 * q_inv[nt][x] : kf0;
              z[nt][2 + x] *= E == 1 ? kf1 * q_inv[nt][x] : kf1;
              if (edge) {
                if (!span_sees(pos[nt][x], key0, a.window, a.sinks)) z[nt][x] = -INFINITY;
                if (!span_sees(pos[nt][x], key1, a.window, a.sinks)) z[nt][2 + x] = -INFINITY;
              }
              unset = unset || m[nt][x] == -INFINITY || (E == 1 && per[nt][x] == 0.f);
            }
          }
          // the largest over a row's 16 positions: over the lanes that share c
          auto top_of = [&](float x, float y) {
            float t = fmaxf(x, y);
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
            return fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          };
          // The weights exp2(z - m), and for V the weight times V's scale times `per`.  m and 1 / per are
          // references, not exact maxima: they move only when a weight outgrows them -- 2^64 for bf16
          // weights, 2^14 for fp16 ones (the row's largest stays above 1, so what fp16 rounds below its
          // normal range is off by 2^-25 of it at most) -- so between moves no row maximum is taken.
          float pr[NT][4], wv[NT][4];
          auto weights = [&]() {
            bool big = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const float ref = m[nt][x & 1] == -INFINITY ? 0.f : m[nt][x & 1];
                pr[nt][x] = ex2_approx(z[nt][x] - ref);
                if (E == 1) {
                  wv[nt][x] = pr[nt][x] * ((x < 2 ? vf0 : vf1) * per[nt][x & 1]);
                  if (edge && z[nt][x] == -INFINITY) wv[nt][x] = 0.f;  // a masked row's scale may be anything
                  big = big || !(wv[nt][x] <= 16384.f);
                } else {
                  wv[nt][x] = pr[nt][x];
                }
                big = big || !(pr[nt][x] <= kBig);
              }
            return big;
          };
          bool move = weights();
          if (__any_sync(0xffffffffu, move || unset)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float t = fmaxf(top_of(z[nt][x], z[nt][2 + x]), m[nt][x]);
                const float alpha = m[nt][x] == -INFINITY ? 0.f : ex2_approx(m[nt][x] - t);
                m[nt][x] = t;
                l[nt][x] *= alpha;
                float mul = alpha;
                if (E == 1) {  // O keeps its size when m moves, its unit takes the factor
                  const float ref = t == -INFINITY ? 0.f : t;
                  const float w0 = z[nt][x] == -INFINITY ? 0.f : ex2_approx(z[nt][x] - ref) * vf0;
                  const float w1 = z[nt][2 + x] == -INFINITY ? 0.f : ex2_approx(z[nt][2 + x] - ref) * vf1;
                  const float top = top_of(w0, w1), old = per[nt][x] > 0.f ? alpha / per[nt][x] : 0.f;
                  float unit = top > old * 16384.f ? top : old;
                  // 2^-126 at the least, or 1 / unit is infinite (values below 1e-36, or beside a key far above
                  // them whose own are zero); the smallest scale, 2^-149, is in fp16's range then too
                  if (unit > 0.f) unit = fmaxf(unit, 1.17549435e-38f);
                  mul = unit == old ? 1.f : old / unit;
                  per[nt][x] = unit > 0.f ? 1.f / unit : 0.f;
                }
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt) {
                  o[mt][nt][x] *= mul;
                  o[mt][nt][2 + x] *= mul;
                }
              }
            weights();
          }
          uint32_t b[NT][2];  // rounded to 16 bits here, as the product's operand
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) l[nt][x] += pr[nt][x] + pr[nt][2 + x];
            b[nt][0] = transpose8x8(E == 1 ? pack_f16x2(wv[nt][0], wv[nt][1]) : pack_bf16x2(wv[nt][0], wv[nt][1]));
            b[nt][1] = transpose8x8(E == 1 ? pack_f16x2(wv[nt][2], wv[nt][3]) : pack_bf16x2(wv[nt][2], wv[nt][3]));
          }
          // V: rows of slots 2c, 2c + 1, 2c + 8, 2c + 9
          const int v0 = k0 + perm(2 * c), v1 = k0 + perm(2 * c + 1);
          const int vr[4] = {v0, v1, v0 + 8, v1 + 8};
          if (E == 2) {
#pragma unroll
            for (int i = 0; i < L::kRow / 128; ++i) {
              uint32_t x[4][4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 y = lds128(at(tv, vr[e], g + 8 * i));
                x[e][0] = y.x;
                x[e][1] = y.y;
                x[e][2] = y.z;
                x[e][3] = y.w;
              }
              if (edge) {
                // What masked positions hold must not meet a weight of zero as a NaN or an infinity: those
                // become zeros here, and the rows that do see them get them added below.
                uint32_t any = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int t = 0; t < 4; ++t) {
                    const uint32_t bad = ((x[e][t] & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                    any |= bad;
                    if (bad & 0x8000u) x[e][t] &= 0xffff0000u;
                    if (bad & 0x80000000u) x[e][t] &= 0x0000ffffu;
                  }
                if (__any_sync(0xffffffffu, any != 0)) {
#pragma unroll 1
                  for (int k = 0; k < 16; ++k) {
                    const uint4 y = lds128(at(tv, k0 + k, g + 8 * i));
                    const uint32_t ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                          if (!span_sees(pos[nt][r], u0 + k, a.window, a.sinks)) continue;
                          if ((ys[t] & 0x7f80u) == 0x7f80u) o[4 * i + t][nt][r] += __uint_as_float(ys[t] << 16);
                          if ((ys[t] & 0x7f800000u) == 0x7f800000u) o[4 * i + t][nt][2 + r] += __uint_as_float(ys[t] & 0xffff0000u);
                        }
                  }
                }
              }
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint32_t a0 = __byte_perm(x[0][t], x[1][t], 0x5410), a1 = __byte_perm(x[0][t], x[1][t], 0x7632);
                const uint32_t a2 = __byte_perm(x[2][t], x[3][t], 0x5410), a3 = __byte_perm(x[2][t], x[3][t], 0x7632);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<E>(o[4 * i + t][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
              }
            }
          } else {
            uint32_t x[4][D / 32];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (D == 128) {
                const uint4 y = lds128(at(tv, vr[e], g));
                x[e][0] = y.x;
                x[e][1] = y.y;
                x[e][2 % (D / 32)] = y.z;
                x[e][3 % (D / 32)] = y.w;
              } else {
                const uint2 y = lds64(at(tv, vr[e], g >> 1) + (g & 1) * 8);
                x[e][0] = y.x;
                x[e][1] = y.y;
              }
            }
            if (edge) {  // the NaN codes of masked positions; rows that see one have its NaN scale in their weight
#pragma unroll
              for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int t = 0; t < D / 32; ++t) {
                  const uint32_t bad = ((x[e][t] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                  x[e][t] &= ~((bad >> 7) * 0xffu);
                }
            }
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // (key, key) pairs of dims 4t + 2h, + 1
                const uint32_t u = __byte_perm(x[0][t], x[1][t], h ? 0x7362 : 0x5140);
                const uint32_t v = __byte_perm(x[2][t], x[3][t], h ? 0x7362 : 0x5140);
                const uint32_t a0 = widen_lo(u), a1 = widen_hi(u), a2 = widen_lo(v), a3 = widen_hi(v);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma<E>(o[2 * t + h][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
              }
          }
        }
        mbar_arrive_warp(&bars->empty[s]);
      }

      if (!ok) break;
      if (p.write) {  // every warp sees every phase, or a later one could pass for it
        ok = __all_sync(0xffffffffu, mbar_wait(&bars->new_full[(n - 1) & 1], ((n - 1) / 2) & 1, abort_flag, budget));
        if (!ok) break;
        mbar_arrive_warp(&bars->new_empty[(n - 1) & 1]);
      }
      // leave the results to the joining warp, 8 rows at a time
      const bool ends = w.ends();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt, ++joins) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = l[nt][x];
          t += __shfl_xor_sync(0xffffffffu, t, 4);
          t += __shfl_xor_sync(0xffffffffu, t, 8);
          t += __shfl_xor_sync(0xffffffffu, t, 16);
          l[nt][x] = t;
        }
        if (ok && ends && nt > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->join_empty8, 0, abort_flag, budget));
        else if (ok && joins > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->join_empty, (joins - 1) & 1, abort_flag, budget));
        if (!ok) break;
        float* mine = join + warp * 8 * L::kPad;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float unit = per[nt][x] > 0.f ? 1.f / per[nt][x] : 0.f;
          if (g == 0) join_ml[warp * 8 + 2 * c + x] = make_float2(m[nt][x], l[nt][x]);
#pragma unroll
          for (int mt = 0; mt < kTiles; ++mt)  // [row][tile][g][2]: no two lanes of a half warp share a bank
            *reinterpret_cast<float2*>(mine + (2 * c + x) * L::kPad + mt * 16 + 2 * g) =
                E == 1 ? make_float2(o[mt][nt][x] * unit, o[mt][nt][2 + x] * unit)
                       : make_float2(o[mt][nt][x], o[mt][nt][2 + x]);
        }
        mbar_arrive_warp(&bars->join_full);
        if (!ends) continue;
        // The part's last unit: nothing else to do here, so a warp per row, without the joining warp
        if (!(ok = __all_sync(0xffffffffu, mbar_wait(&bars->join_full, joins & 1, abort_flag, budget)))) break;
        const int row = nt * 8 + warp;
        if (row < rows) {
          float acc[D / 32], top, sum;
          join_warps<D, E>(join, join_ml, warp, acc, top, sum);
          if (w.whole()) {
            store_row<D>(a, w.item, w.head, row, acc, sum);
          } else {
            store_piece<D>(a, w.slot(blockIdx.x) * a.layout.rows + row, acc, top, sum);
            __threadfence();
            __syncwarp();
            int before = 0;
            if (lane == 0)
              before = atomicAdd(reinterpret_cast<int32_t*>(a.ws + a.line.arrived) + w.first() * kSpanRows + row, 1);
            if (__shfl_sync(0xffffffffu, before, 0) == w.parts() - 1) {
              __threadfence();
              join_pieces<D>(a, w.item, w.head, row, w.first(), w.parts());
            }
          }
        }
        if (NT > 1) mbar_arrive_warp(&bars->join_empty8);
      }
    }
    if (!ok && lane == 0) timeout();
  }
}

template <int D, int E, int NT>
cudaError_t launch(const SpanArgs& a, bool write, cudaStream_t s) {
  using L = Smem<D, E, NT>;
  RowsArgs p;
  p.s = a;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wait_budget = wait_budget_cycles();
  p.write = write;
  p.test_stall = test_stall_requested();
  CUtensorMap mk, mv;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)a.n_blocks * a.h_kv * kPage};
  const cuuint32_t box[2] = {(cuuint32_t)(L::kPitch / E), 16};
  const CUtensorMapSwizzle swizzle = L::kPitch == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!span_tensor_map(&mk, a.pool_k, E, 2, dims, box, swizzle) || !span_tensor_map(&mv, a.pool_v, E, 2, dims, box, swizzle))
    return cudaErrorInvalidValue;
  static_assert(L::kStages >= 2 && L::kCtas * (L::kBytes + 1024) <= 228 * 1024, "shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(span_rows_kernel<D, E, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(span_rows_kernel<D, E, NT>, dim3(a.ctas), dim3(kThreads), (size_t)L::kBytes, s, mk, mv, p);
}

template <int D, int E>
cudaError_t launch_nt(const SpanArgs& a, bool write, cudaStream_t s) {
  return a.tile_rows == 8 ? launch<D, E, 1>(a, write, s) : launch<D, E, 2>(a, write, s);
}

}  // namespace

int span_rows_ctas(int d, int rows) { return few_rows_ctas(d, rows / 8); }

cudaError_t launch_span_rows(const SpanArgs& a, bool write, cudaStream_t s) {
  if (a.pool_elem == 1) return a.d == 64 ? launch_nt<64, 1>(a, write, s) : launch_nt<128, 1>(a, write, s);
  return a.d == 64 ? launch_nt<64, 2>(a, write, s) : launch_nt<128, 2>(a, write, s);
}

}  // namespace kev
