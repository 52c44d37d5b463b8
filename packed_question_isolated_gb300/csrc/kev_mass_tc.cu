// Attention mass on the 5th-generation tensor cores, for chunks of new tokens: bf16 q, cache bf16 or e4m3, fp32 scores.
//
// Two kernels over the same scores, which are computed twice (their exponentials, not the products, are what both cost):
//   mass_rows_tc   S[128 rows x 128 keys] = Q K^T of a row tile -- (token, q-head of the group) rows of one question and kv
//                  head -- against the key tiles its tokens see; a thread owns a row (its TMEM lane) and keeps its running
//                  maximum and sum.  A unit is one or two row tiles and a kv head; every CTA has an equal part of all units'
//                  key tiles (kev_span.cuh).
//   mass_keys_tc   S^T[128 keys x 128 rows] = K Q^T of a key tile against the row tiles that see it; a thread owns a key, so
//                  the sum of its weights exp2(S^T - lse) over the rows needs no exchange.  A unit is a key tile and a kv
//                  head; every CTA has an equal part of all units' row tiles, cut by mass_cuts; the pieces of a unit that a
//                  cut goes through are added in their order by the CTA that finishes last.
// Both have the same shape, one persistent CTA per SM of 16 warps:
//   warps 0-3, 4-7   exponentials; tile x of the CTA's sequence goes to group x % 2 and to one of four S buffers in tensor
//                    memory, so two tiles' MMAs run ahead of them
//   warp 8           loads key tiles (TMA; e4m3: bulk copies of a page's codes and scales)
//   warp 9           issues the MMAs
//   warp 10          loads q tiles: boxes of tokens x group heads x 64 dims
//   warps 12-15      e4m3: codes to bf16, which holds each exactly, in the MMA's swizzled layout; the scale multiplies the
//                    score instead
// A masked score is replaced, not multiplied, so what lies in keys that a row does not see never counts.  Every wait is
// bounded, as in the other tensor-core kernels.
//
// What bounds it.  8 chunks of 128 to 1024 tokens behind up to 8192 positions (28/4 heads, bf16) take 208 us, 87 of them
// the first kernel and 121 the second; over e4m3 248; 32 tokens of each of 8 e4m3 caches of 4 to 16 Ki positions 111 (49
// and 60), of bf16 ones 90.  The tensor pipe is busy 38 and 30 % of the time (19 and 16 over e4m3), the exponentials' pipe
// about as much, L2 and DRAM under 15 %.  Neither the exponentials (without them 200 us), nor the MMAs (with one of a
// tile's eight 186) nor the copies (of half the bytes: no change) carry it alone: what is left is the hand-over of a tile,
// MMA - barrier - tensor memory - barrier, some 1500 clocks each, and in the second kernel a key tile's beginning and end.
// Measured and left: four groups of four warps at 96 registers, which spill (235 and 157 us); three groups at 128 that
// take 32 columns at a time (207 and 124); polling instead of suspended waits, shorter chains for the maximum (no
// difference).  A second key tile against each loaded q tile is not built.
#include <cuda.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "kev_mass.cuh"
#include "kev_sm100.cuh"

namespace kev {
namespace {

using namespace sm100;

constexpr int kM = 128;
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kQWarp = 10, kReadyWarp = 12;
constexpr int kRegsExp = 200, kRegsOther = 56;  // 128 registers a thread at launch: 256 x 200 + 256 x 56 = 512 x 128
constexpr uint32_t kTmemCols = 512;             // four S buffers of 128 columns
constexpr long long kDrainBudget = 4000000000ll;
// Of a unit of mass_keys_tc beside its row tiles, in row tiles: 8 chunks of 128 to 1024 tokens (32/8 heads) take 180 us with
// 1, 191 with 0, 179 with 2, 185 with 4 (28/4 heads 157, 159, 158, 161); 32 tokens of each of 8 caches the same with all
constexpr int kUnitCost = 1;

// Where a part of mass_keys_tc's work line begins: key tile `tile` of question and head, its row tile r; r > 0: the cut is
// inside the unit, which has `parts` parts from part `first` on.
struct alignas(16) KeyCut {
  int32_t question, head, tile, r;
  int32_t first, parts, pad[2];
};

struct TcArgs {
  MassArgs m;
  float scale_log2;
  long long wait_budget;
  int32_t test_stall;  // timeout test hook
};

// kQ q tiles and kK key tiles of bf16 in shared memory, and for e4m3 kStages tiles of codes
template <int D, bool Q8, int kQTiles, int kKTiles, int kStages>
struct Smem {
  static constexpr int kSub = D / 64;        // 128-byte sub-tiles of a row
  static constexpr int kSubBytes = kM * 128;
  static constexpr int kTile = kM * D * 2;
  static constexpr int kCodes = kM * D;
  static constexpr int kNQ = kQTiles, kNK = kKTiles, kNS = kStages;
  static constexpr int kQ = 0;
  static constexpr int kK = kQTiles * kTile;
  static constexpr int kStage = kK + kKTiles * kTile;
  static constexpr int kScale = kStage + (Q8 ? kStages * kCodes : 0);  // scales of four key tiles
  static constexpr int kExtra = kScale + (Q8 ? 4 * kM * 4 : 0);        // floats of the exponentials' groups
  static constexpr int kBar = kExtra + 4 * kM * 4 * 2;
  static constexpr int kBytes = kBar + 512 + 1024;  // slack for 1024-byte alignment
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Bars {
  uint64_t q_full[4], q_empty[4];
  uint64_t k_full[4], k_empty[4], ready[4];
  uint64_t st_full[4], st_empty[4], sc_full[4], sc_empty[4];
  uint64_t s_full[4], s_free[4];
  uint64_t drain, stall;
  uint32_t tmem;
  int abort, never, last[2];
};
static_assert(sizeof(Bars) <= 512, "barriers");

__device__ __forceinline__ void raise_timeout(const TcArgs& p, Bars* b) {
  atomicCAS(&reinterpret_cast<SpanHeader*>(p.m.s.ws)->status, 0, ST_TIMEOUT);
  set_status(p.m.s.dev_status, ST_TIMEOUT);
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag, long long budget) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, budget));
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void e4m3_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  lo = pack_bf16x2(x.x, x.y);
  hi = pack_bf16x2(y.x, y.y);
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A tile of codes as bf16 in the swizzled layout, by 128 threads (x: which).
template <typename L>
__device__ __forceinline__ void convert_tile(const unsigned char* from, unsigned char* to, int D, int x) {
  const uint4* codes = reinterpret_cast<const uint4*>(from);
  const uint32_t dst = smem_u32(to);
  const int groups = D / 16;  // 16-code groups of a row
#pragma unroll 4
  for (int e = 0; e < kM * groups / 128; ++e) {
    const int at = e * 128 + x, r = at / groups, g = at % groups;
    const uint4 c = codes[at];
    uint32_t o[8];
    e4m3_to_bf16(c.x, o[0], o[1]);
    e4m3_to_bf16(c.y, o[2], o[3]);
    e4m3_to_bf16(c.z, o[4], o[5]);
    e4m3_to_bf16(c.w, o[6], o[7]);
    // 16-byte chunks 2 (g % 4) and + 1 of sub-tile g / 4, XOR-ed with r % 8; lanes of the second sub-tile store
    // theirs the other way round, so a quarter warp hits every bank once
    const uint32_t base = dst + (g >> 2) * L::kSubBytes + r * 128, k = 2 * (g & 3), sw = r & 7;
    const bool flip = g >= 4;
    const uint32_t a0 = base + (((k + (flip ? 1 : 0)) ^ sw) << 4), a1 = base + (((k + (flip ? 0 : 1)) ^ sw) << 4);
    if (flip) {
      st_shared_v4(a0, o[4], o[5], o[6], o[7]);
      st_shared_v4(a1, o[0], o[1], o[2], o[3]);
    } else {
      st_shared_v4(a0, o[0], o[1], o[2], o[3]);
      st_shared_v4(a1, o[4], o[5], o[6], o[7]);
    }
  }
}

// S = A B^T of two 128-row tiles into a buffer of tensor memory, by one thread
template <int D, typename L>
__device__ __forceinline__ void issue_scores(uint32_t tmem, const unsigned char* a, const unsigned char* b) {
  constexpr uint32_t idesc = idesc_bf16(kM, kM, false, false);
  // the descriptors' address field counts 16 bytes: one addition a step instead of building each anew (8 chunks 212 -> 208 us)
  const uint64_t a_desc = sdesc_sw128(smem_u32(a), 16, 1024), b_desc = sdesc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * L::kSubBytes + (kk & 3) * 32) / 16;
    umma_bf16(tmem, a_desc + off, b_desc + off, idesc, kk > 0);
  }
}

// Barriers, tensor memory; the whole CTA.  q tiles start as zeros: rows behind a box's stay so.
template <typename L>
__device__ __forceinline__ uint32_t begin(unsigned char* smem, Bars* b, int warp) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) {
      mbar_init(&b->q_full[s], 1);
      mbar_init(&b->q_empty[s], 1);
      mbar_init(&b->k_full[s], 1);
      mbar_init(&b->k_empty[s], 1);
      mbar_init(&b->ready[s], 4);
      mbar_init(&b->st_full[s], 1);
      mbar_init(&b->st_empty[s], 4);
      mbar_init(&b->sc_full[s], 4);
      mbar_init(&b->sc_empty[s], 8);
      mbar_init(&b->s_full[s], 1);
      mbar_init(&b->s_free[s], 4);
    }
    mbar_init(&b->drain, 1);
    mbar_init(&b->stall, 1);
    b->abort = 0;
    b->never = 0;
    fence_mbar_init();
  }
  uint4* q = reinterpret_cast<uint4*>(smem + L::kQ);
  for (int x = threadIdx.x; x < L::kNQ * L::kTile / 16; x += kThreads) q[x] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == kMmaWarp) {
    tmem_alloc(&b->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return b->tmem;
}

// Group g's 128 threads
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(4 + g) : "memory"); }
__device__ __forceinline__ void both_sync() { asm volatile("bar.sync 6, 256;" ::: "memory"); }

// A key tile's copies by one thread: ring slot `slot` (bf16) or code stage (e4m3)
template <int D, bool Q8, typename L>
__device__ __forceinline__ void load_keys(const SpanArgs& a, const CUtensorMap* tm_k, unsigned char* smem, int slot, uint32_t n,
                                          int block, int head, uint64_t* bar) {
  const int64_t cell = ((int64_t)block * a.h_kv + head) * kPage;
  if (Q8) {
    mbar_arrive_expect_tx(bar, L::kCodes + kM * 4);
    bulk_load(smem + L::kStage + slot * L::kCodes, static_cast<const char*>(a.pool_k) + cell * D, L::kCodes, bar);
    bulk_load(smem + L::kScale + n % 4 * (kM * 4), a.scale_k + cell, kM * 4, bar);
  } else {
    mbar_arrive_expect_tx(bar, L::kTile);
    for (int c = 0; c < L::kSub; ++c)
      tma_load_2d(smem + L::kK + slot * L::kTile + c * L::kSubBytes, tm_k, c * 64, (int)cell, bar);
  }
}

// ---------------------------------------------------------------------------------------
// the rows' log sums
// ---------------------------------------------------------------------------------------
template <int D, bool Q8> using RowsSmem = Smem<D, Q8, 2, Q8 ? 3 : 4, 3>;

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    mass_rows_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ TcArgs p) {
  using L = RowsSmem<D, Q8>;
  const SpanArgs& a = p.m.s;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = begin<L>(smem, bars, warp);
  volatile int* abort_flag = &bars->abort;
  const volatile int* never = &bars->never;
  const long long budget = p.wait_budget;
  pdl_wait();
  pdl_trigger();
  const bool go = reinterpret_cast<const SpanHeader*>(a.ws)->status == ST_OK;

  if (warp >= kLoadWarp) {
    regs_dec<kRegsOther>();
    if (!go) {
    } else if (warp == kLoadWarp) {
      if (lane == 0) {
        constexpr int kSlots = Q8 ? L::kNS : L::kNK;
        uint64_t* full = Q8 ? bars->st_full : bars->k_full;
        uint64_t* empty = Q8 ? bars->st_empty : bars->k_empty;
        uint32_t n = 0;
        bool ok = !(p.test_stall && blockIdx.x == 0) || mbar_wait(&bars->stall, 0, abort_flag, budget);
        for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next()) {
          const int32_t* table = a.table + (int64_t)w.item.question * a.max_blocks;
          int block = table[w.j0];
          for (int j = w.j0; j < w.j1; ++j, ++n) {
            const int here = block;
            if (j + 1 < w.j1) block = table[j + 1];  // one tile ahead
            const int s = n % kSlots;
            if ((n >= kSlots && !mbar_wait(&empty[s], (n / kSlots - 1) & 1, abort_flag, budget)) ||
                (Q8 && n >= 4 && !mbar_wait(&bars->sc_empty[n % 4], (n / 4 - 1) & 1, abort_flag, budget))) {
              ok = false;
              break;
            }
            load_keys<D, Q8, L>(a, &tm_k, smem, s, n, here, w.head, &full[s]);
          }
        }
        if (!ok) raise_timeout(p, bars);
        // every copy issued lands before the CTA leaves, whoever gave up
        for (uint32_t q = n < kSlots ? 0 : n - kSlots; q < n; ++q) mbar_wait(&full[q % kSlots], (q / kSlots) & 1, never, kDrainBudget);
      }
    } else if (warp == kQWarp) {
      if (lane == 0) {
        uint32_t n = 0;
        bool ok = true;
        for (SpanWalk w(a, blockIdx.x); w.live(); w.next(), ++n) {
          if (n > 0 && !mbar_wait(&bars->q_empty[0], (n - 1) & 1, abort_flag, budget)) {
            ok = false;
            break;
          }
          const int nt = w.item.tokens > a.tile_tokens ? 2 : 1;
          mbar_arrive_expect_tx(&bars->q_full[0], nt * L::kSub * 128 * a.group * a.tile_tokens);
          for (int t = 0; t < nt; ++t)
            for (int c = 0; c < L::kSub; ++c)
              tma_load_3d(smem + L::kQ + t * L::kTile + c * L::kSubBytes, &tm_q, c * 64, w.head * a.group,
                          w.item.row0 + t * a.tile_tokens, &bars->q_full[0]);
        }
        if (!ok) raise_timeout(p, bars);
        if (n) mbar_wait(&bars->q_full[0], (n - 1) & 1, never, kDrainBudget);
      }
    } else if (warp == kMmaWarp) {
      uint32_t n = 0, x = 0, units = 0;
      bool ok = true;
      auto wait_ok = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = warp_wait(bar, parity, abort_flag, budget);
      };
      for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next(), ++units) {
        const int nt = w.item.tokens > a.tile_tokens ? 2 : 1;
        wait_ok(&bars->q_full[0], units & 1);
        for (int j = w.j0; ok && j < w.j1; ++j, ++n) {
          const int s = n % L::kNK;
          wait_ok(Q8 ? &bars->ready[s] : &bars->k_full[s], (n / L::kNK) & 1);
          for (int t = 0; t < nt; ++t, ++x) {
            if (x >= 4) wait_ok(&bars->s_free[x % 4], (x / 4 - 1) & 1);
            if (ok && lane == 0) {
              tc_fence_after();
              issue_scores<D, L>(tmem + x % 4 * kM, smem + L::kQ + t * L::kTile, smem + L::kK + s * L::kTile);
              umma_commit(&bars->s_full[x % 4]);
            }
            __syncwarp();
          }
          if (ok && lane == 0) {
            umma_commit(&bars->k_empty[s]);
            if (j + 1 == w.j1) umma_commit(&bars->q_empty[0]);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
      if (lane == 0) {  // every MMA issued is complete before TMEM is freed
        umma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, never, kDrainBudget);
      }
      __syncwarp();
    } else if (Q8 && warp >= kReadyWarp) {
      const int x = threadIdx.x - kReadyWarp * 32;
      uint32_t n = 0;
      bool ok = true;
      for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next())
        for (int j = w.j0; j < w.j1; ++j, ++n) {
          const int s = n % L::kNK, st = n % L::kNS;
          if (!warp_wait(&bars->st_full[st], (n / L::kNS) & 1, abort_flag, budget) ||
              (n >= L::kNK && !warp_wait(&bars->k_empty[s], (n / L::kNK - 1) & 1, abort_flag, budget))) {
            ok = false;
            break;
          }
          float* sc = reinterpret_cast<float*>(smem + L::kScale) + n % 4 * kM + x;
          *sc *= p.scale_log2;
          mbar_arrive_warp(&bars->sc_full[n % 4]);
          convert_tile<L>(smem + L::kStage + st * L::kCodes, smem + L::kK + s * L::kTile, D, x);
          fence_proxy_async_smem();
          mbar_arrive_warp(&bars->ready[s]);
          mbar_arrive_warp(&bars->st_empty[st]);
        }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  } else {
    regs_inc<kRegsExp>();
    if (go) {
      const int grp = warp >> 2, r = (warp & 3) * 32 + lane;  // a warp reaches TMEM lanes 32 (warp % 4) ..
      const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const int tok = r / a.group;
      float* lse = reinterpret_cast<float*>(a.ws + p.m.lse);
      float2* other = reinterpret_cast<float2*>(smem + L::kExtra);  // [2][128] group 1's sums of one row tile
      uint32_t n = 0, x = 0, single = 0;
      bool ok = true;  // false: a wait gave up; the walk goes on, for the barriers that the groups' threads share
      for (SpanWalk w(a, blockIdx.x); w.live(); w.next()) {
        const int p0 = w.item.p0, nt = w.item.tokens > a.tile_tokens ? 2 : 1;
        // two row tiles: this group's is always the same; one: the groups take its key tiles in turns
        const int t = nt == 2 ? grp ^ (int)(x & 1) : 0;
        const int token = t * a.tile_tokens + tok, pos = p0 + token;
        const bool row_ok = tok < a.tile_tokens && token < w.item.tokens;
        float m = -INFINITY, l = 0.f;
        for (int j = w.j0; j < w.j1; ++j, ++n, x += nt) {
          const uint32_t y = x + t;  // tile of the CTA's sequence
          const bool mine = (y & 1) == (uint32_t)grp;
          if (Q8) ok = ok && warp_wait(&bars->sc_full[n % 4], (n / 4) & 1, abort_flag, budget);
          if (mine) {
            ok = ok && warp_wait(&bars->s_full[y % 4], (y / 4) & 1, abort_flag, budget);
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tm + y % 4 * kM + 32 * c, v[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_wait(v[c]);
            tc_fence_before();
            mbar_arrive_warp(&bars->s_free[y % 4]);
            // scores in log2 units
            if (Q8) {
              const float4* sc = reinterpret_cast<const float4*>(smem + L::kScale + n % 4 * (kM * 4));
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float4 f = sc[8 * c + e];
                  v[c][4 * e] = __float_as_uint(__uint_as_float(v[c][4 * e]) * f.x);
                  v[c][4 * e + 1] = __float_as_uint(__uint_as_float(v[c][4 * e + 1]) * f.y);
                  v[c][4 * e + 2] = __float_as_uint(__uint_as_float(v[c][4 * e + 2]) * f.z);
                  v[c][4 * e + 3] = __float_as_uint(__uint_as_float(v[c][4 * e + 3]) * f.w);
                }
            }
            const int u0 = j * kM;
            if (u0 + kM - 1 > p0) {  // a key that some row does not see
              const int seen = pos - u0 + 1;
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (32 * c + e >= seen) v[c][e] = 0xff800000u;
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 2)
#pragma unroll
              for (int c = 0; c < 4; ++c) tops[c] = fmax3(tops[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
            float top = fmax3(fmaxf(tops[0], tops[1]), tops[2], tops[3]);
            const float sl2 = Q8 ? 1.f : p.scale_log2;
            top *= sl2;
            if (top > m) {
              l *= ex2_approx(m - top);  // (0 at the beginning: m is -infinity)
              m = top;
            }
            const float base = m == -INFINITY ? 0.f : m;
            const unsigned long long sl2x2 = f2pack(sl2, sl2), basex2 = f2pack(-base, -base);
            unsigned long long sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const unsigned long long s2 = (unsigned long long)v[c][e] | (unsigned long long)v[c][e + 1] << 32;
                const float2 z = unpack2(Q8 ? add2(s2, basex2) : fma2(s2, sl2x2, basex2));
                sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], f2pack(ex2_approx(z.x), ex2_approx(z.y)));
              }
            const float2 s0 = unpack2(add2(sum[0], sum[1]));
            l += s0.x + s0.y;
          }
          if (Q8) mbar_arrive_warp(&bars->sc_empty[n % 4]);
        }
        if (nt == 1) {  // both groups have sums of the same rows
          if (grp == 1) other[(single & 1) * kM + r] = make_float2(m, l);
          both_sync();
          if (grp == 0) {
            const float2 y = other[(single & 1) * kM + r];
            const float top = fmaxf(m, y.x), base = top == -INFINITY ? 0.f : top;
            l = l * ex2_approx(m - base) + y.y * ex2_approx(y.x - base);
            m = top;
          }
          ++single;
        }
        if (ok && row_ok && (nt == 2 || grp == 0)) {
          if (w.whole())
            lse[(int64_t)(w.item.row0 + token) * a.h_q + w.head * a.group + r % a.group] = m + log2f(l);
          else
            reinterpret_cast<float2*>(a.ws + a.layout.part_ml)[w.slot(blockIdx.x) * a.layout.rows + t * kM + r] = make_float2(m, l);
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------------------
// between them: the rows' pieces joined, and the work line of the second kernel
// ---------------------------------------------------------------------------------------
// Row tiles that see key tile j of a question with L new tokens behind `prefix` ones
struct KeyTiles {
  int L, prefix, tokens, tiles, whole, most;  // whole: tiles that all of the tokens see, of `most` row tiles each
  __device__ KeyTiles(const SpanArgs& a, int i) {
    const kev_interval v = a.intervals[i];
    L = v.end - v.begin;
    prefix = a.prefix[i];
    tokens = a.tile_tokens;
    tiles = L > 0 ? (prefix + L - 1) / kM + 1 : 0;
    whole = L > 0 ? prefix / kM + 1 : 0;
    most = (L + tokens - 1) / tokens;
  }
  __device__ int token(int j) const { return max(0, j * kM - prefix); }  // the first token that sees tile j
  __device__ int rows(int j) const { return (L - token(j) + tokens - 1) / tokens; }
};

__global__ void __launch_bounds__(256) mass_cuts_kernel(const __grid_constant__ MassArgs p) {
  extern __shared__ long long s_before[];  // [n + 1] cost before each question
  __shared__ long long s_sum[9];
  const SpanArgs& a = p.s;
  pdl_wait();
  pdl_trigger();
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  if (h->status != ST_OK) return;
  const int t = threadIdx.x;
  if (blockIdx.x > 0) {  // a thread per row of the units that the plan lists
    const SpanCut* cuts = reinterpret_cast<const SpanCut*>(a.ws + a.line.cuts);
    const int32_t* joins = reinterpret_cast<const int32_t*>(a.ws + a.line.joins);
    const float2* ml = reinterpret_cast<const float2*>(a.ws + a.layout.part_ml);
    float* lse = reinterpret_cast<float*>(a.ws + p.lse);
    const int todo = h->n_joins * a.layout.rows;
    for (int x = (blockIdx.x - 1) * 256 + t; x < todo; x += (gridDim.x - 1) * 256) {
      const SpanCut& cut = cuts[joins[x / a.layout.rows]];
      const int row = x % a.layout.rows, rr = row % a.tile_rows, token = row / a.tile_rows * a.tile_tokens + rr / a.group;
      if (rr >= a.tile_tokens * a.group || token >= cut.record.tokens) continue;
      // slot 1 of the part the unit begins in, slot 0 of the later ones
      auto piece = [&](int i) { return ml[(2 * (int64_t)(cut.first + i) + (i == 0)) * a.layout.rows + row]; };
      float m = -INFINITY, l = 0.f;
#pragma unroll 4
      for (int i = 0; i < cut.parts; ++i) m = fmaxf(m, piece(i).x);
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll 4
      for (int i = 0; i < cut.parts; ++i) {
        const float2 y = piece(i);
        l = fmaf(y.y, ex2_approx(y.x - base), l);
      }
      lse[(int64_t)(cut.record.row0 + token) * a.h_q + cut.head * a.group + rr % a.group] = base + log2f(l);
    }
    return;
  }
  // one CTA: cut c of the line that lays all units' row tiles (and kUnitCost before each) end to end -- question by
  // question, kv head by kv head, key tile by key tile -- at place floor(c * total / parts)
  const int per = (a.n + 255) / 256;
  auto cost = [&](int i) {  // of a kv head
    const KeyTiles k(a, i);
    long long w = (long long)k.whole * (k.most + kUnitCost);
    for (int j = k.whole; j < k.tiles; ++j) w += k.rows(j) + kUnitCost;
    return w * a.h_kv;
  };
  long long mine = 0;
  for (int e = 0; e < per; ++e) {
    const int i = t * per + e;
    if (i < a.n) mine += s_before[i] = cost(i);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if ((t & 31) >= o) incl += y;
  }
  if ((t & 31) == 31) s_sum[t >> 5] = incl;
  __syncthreads();
  long long at = incl - mine;
  for (int w = 0; w < t >> 5; ++w) at += s_sum[w];
  for (int e = 0; e < per; ++e) {
    const int i = t * per + e;
    if (i < a.n) {
      const long long c = s_before[i];
      s_before[i] = at;
      at += c;
    }
  }
  if (t == 255) s_before[a.n] = at;
  __syncthreads();
  const long long total = s_before[a.n];
  const int parts = (int)min((long long)a.ctas, total);
  KeyCut* cuts = reinterpret_cast<KeyCut*>(a.ws + p.cuts);
  for (int c = t; c <= a.ctas; c += 256) {
    KeyCut cut = {a.n, 0, 0, 0, 0, 0, {0, 0}};
    if (c < parts) {
      const long long x = c * total / parts;
      int lo = 0, hi = a.n - 1;  // the last question that begins at or before x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_before[mid] <= x) lo = mid;
        else hi = mid - 1;
      }
      const KeyTiles k(a, lo);
      const long long head_cost = (s_before[lo + 1] - s_before[lo]) / a.h_kv, in = x - s_before[lo];
      cut.question = lo;
      cut.head = (int)(in / head_cost);
      long long y = in - cut.head * head_cost;
      const int size = k.most + kUnitCost;
      int j = (int)min((long long)k.whole, y / size);
      y -= (long long)j * size;
      while (y >= k.rows(j) + kUnitCost) y -= k.rows(j++) + kUnitCost;
      cut.tile = j;
      cut.r = (int)max(0ll, y - kUnitCost);
      if (cut.r > 0) {
        auto part_of = [&](long long z) { return (int)(((z + 1) * parts - 1) / total); };  // the last part that begins at or before z
        cut.first = part_of(x - cut.r);
        cut.parts = part_of(x - cut.r + k.rows(j) - 1) - cut.first + 1;
      }
    }
    cuts[c] = cut;
  }
}

// ---------------------------------------------------------------------------------------
// the positions' sums
// ---------------------------------------------------------------------------------------
template <int D, bool Q8> using KeysSmem = Smem<D, Q8, Q8 ? 3 : 4, 2, 2>;

// The units of a part: key tile j of a question and head, and its row tiles [r0, r1).
struct KeyWalk {
  const SpanArgs& a;
  KeyCut from, to;
  int i, head, j, r0, r1;
  KeyTiles k;
  __device__ __forceinline__ KeyWalk(const MassArgs& p, int part)
      : a(p.s),
        from(reinterpret_cast<const KeyCut*>(p.s.ws + p.cuts)[part]),
        to(reinterpret_cast<const KeyCut*>(p.s.ws + p.cuts)[part + 1]),
        i(from.question), head(from.head), j(from.tile), r0(from.r), r1(0), k(a, min(i, a.n - 1)) {
    settle();
  }
  __device__ __forceinline__ bool at_end() const { return i == to.question && head == to.head && j == to.tile; }
  __device__ __forceinline__ void settle() { r1 = live() ? (at_end() ? to.r : k.rows(j)) : 0; }
  __device__ __forceinline__ bool live() const { return i < to.question || (i == to.question && (head < to.head || (head == to.head && (j < to.tile || (j == to.tile && r0 < to.r))))); }
  __device__ __forceinline__ bool whole() const { return r0 == 0 && r1 == k.rows(j); }
  __device__ __forceinline__ int first(int part) const { return r0 ? from.first : part; }
  __device__ __forceinline__ int parts() const { return r0 ? from.parts : to.parts; }
  __device__ __forceinline__ void next() {
    r0 = 0;
    if (++j >= k.tiles) {
      j = 0;
      if (++head == a.h_kv) {
        head = 0;
        do {  // (questions without new tokens have no tiles)
          if (++i >= a.n) break;
          k = KeyTiles(a, i);
        } while (k.tiles == 0 && i < to.question);
      }
    }
    settle();
  }
};

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    mass_keys_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ TcArgs p) {
  using L = KeysSmem<D, Q8>;
  const SpanArgs& a = p.m.s;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmem = begin<L>(smem, bars, warp);
  volatile int* abort_flag = &bars->abort;
  const volatile int* never = &bars->never;
  const long long budget = p.wait_budget;
  pdl_wait();
  pdl_trigger();
  const bool go = reinterpret_cast<const SpanHeader*>(a.ws)->status == ST_OK;

  if (warp >= kLoadWarp) {
    regs_dec<kRegsOther>();
    if (!go) {
    } else if (warp == kLoadWarp) {
      if (lane == 0) {
        constexpr int kSlots = Q8 ? L::kNS : L::kNK;
        uint64_t* full = Q8 ? bars->st_full : bars->k_full;
        uint64_t* empty = Q8 ? bars->st_empty : bars->k_empty;
        uint32_t n = 0;
        bool ok = !(p.test_stall && blockIdx.x == 0) || mbar_wait(&bars->stall, 0, abort_flag, budget);
        for (KeyWalk w(p.m, blockIdx.x); ok && w.live(); w.next(), ++n) {
          const int s = n % kSlots, block = a.table[(int64_t)w.i * a.max_blocks + w.j];
          if ((n >= kSlots && !mbar_wait(&empty[s], (n / kSlots - 1) & 1, abort_flag, budget)) ||
              (Q8 && n >= 4 && !mbar_wait(&bars->sc_empty[n % 4], (n / 4 - 1) & 1, abort_flag, budget))) {
            ok = false;
            break;
          }
          load_keys<D, Q8, L>(a, &tm_k, smem, s, n, block, w.head, &full[s]);
        }
        if (!ok) raise_timeout(p, bars);
        // every copy issued lands before the CTA leaves, whoever gave up
        for (uint32_t q = n < kSlots ? 0 : n - kSlots; q < n; ++q) mbar_wait(&full[q % kSlots], (q / kSlots) & 1, never, kDrainBudget);
      }
    } else if (warp == kQWarp) {
      if (lane == 0) {
        uint32_t x = 0;
        bool ok = true;
        for (KeyWalk w(p.m, blockIdx.x); ok && w.live(); w.next()) {
          const int row = a.intervals[w.i].begin + w.k.token(w.j);
          for (int r = w.r0; r < w.r1; ++r, ++x) {
            const int s = x % L::kNQ;
            if (x >= L::kNQ && !mbar_wait(&bars->q_empty[s], (x / L::kNQ - 1) & 1, abort_flag, budget)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&bars->q_full[s], L::kSub * 128 * a.group * a.tile_tokens);
            for (int c = 0; c < L::kSub; ++c)
              tma_load_3d(smem + L::kQ + s * L::kTile + c * L::kSubBytes, &tm_q, c * 64, w.head * a.group, row + r * a.tile_tokens,
                          &bars->q_full[s]);
          }
        }
        if (!ok) raise_timeout(p, bars);
        for (uint32_t q = x < L::kNQ ? 0 : x - L::kNQ; q < x; ++q) mbar_wait(&bars->q_full[q % L::kNQ], (q / L::kNQ) & 1, never, kDrainBudget);
      }
    } else if (warp == kMmaWarp) {
      uint32_t n = 0, x = 0;
      bool ok = true;
      auto wait_ok = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = warp_wait(bar, parity, abort_flag, budget);
      };
      for (KeyWalk w(p.m, blockIdx.x); ok && w.live(); w.next(), ++n) {
        const int ks = n % L::kNK;
        wait_ok(Q8 ? &bars->ready[ks] : &bars->k_full[ks], (n / L::kNK) & 1);
        for (int r = w.r0; ok && r < w.r1; ++r, ++x) {
          const int qs = x % L::kNQ;
          wait_ok(&bars->q_full[qs], (x / L::kNQ) & 1);
          if (x >= 4) wait_ok(&bars->s_free[x % 4], (x / 4 - 1) & 1);
          if (ok && lane == 0) {
            tc_fence_after();
            issue_scores<D, L>(tmem + x % 4 * kM, smem + L::kK + ks * L::kTile, smem + L::kQ + qs * L::kTile);
            umma_commit(&bars->s_full[x % 4]);
            umma_commit(&bars->q_empty[qs]);
            if (r + 1 == w.r1) umma_commit(&bars->k_empty[ks]);
          }
          __syncwarp();
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
      if (lane == 0) {  // every MMA issued is complete before TMEM is freed
        umma_commit(&bars->drain);
        mbar_wait(&bars->drain, 0, never, kDrainBudget);
      }
      __syncwarp();
    } else if (Q8 && warp >= kReadyWarp) {
      const int x = threadIdx.x - kReadyWarp * 32;
      uint32_t n = 0;
      bool ok = true;
      for (KeyWalk w(p.m, blockIdx.x); ok && w.live(); w.next(), ++n) {
        const int s = n % L::kNK, st = n % L::kNS;
        if (!warp_wait(&bars->st_full[st], (n / L::kNS) & 1, abort_flag, budget) ||
            (n >= L::kNK && !warp_wait(&bars->k_empty[s], (n / L::kNK - 1) & 1, abort_flag, budget))) {
          ok = false;
          break;
        }
        float* sc = reinterpret_cast<float*>(smem + L::kScale) + n % 4 * kM + x;
        *sc *= p.scale_log2;
        mbar_arrive_warp(&bars->sc_full[n % 4]);
        convert_tile<L>(smem + L::kStage + st * L::kCodes, smem + L::kK + s * L::kTile, D, x);
        fence_proxy_async_smem();
        mbar_arrive_warp(&bars->ready[s]);
        mbar_arrive_warp(&bars->st_empty[st]);
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  } else {
    regs_inc<kRegsExp>();
    if (go) {
      const int grp = warp >> 2, r = (warp & 3) * 32 + lane;  // this thread's key of the tile, and its column of the lse
      const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const float* lse = reinterpret_cast<const float*>(a.ws + p.m.lse);
      float* minus = reinterpret_cast<float*>(smem + L::kExtra) + grp * 2 * kM;       // [2][128] -lse of a row tile
      float* other = reinterpret_cast<float*>(smem + L::kExtra) + 4 * kM;             // [2][128] group 1's sums
      float* part = reinterpret_cast<float*>(a.ws + a.layout.part_o);                 // [2 * parts][128]
      int32_t* arrived = reinterpret_cast<int32_t*>(a.ws + a.line.arrived);
      const int tok = r / a.group;
      // Columns that are rows of a full tile.  Those behind them (a group that does not divide 128 leaves fewer than 16) are
      // q rows of zeros, and beside an infinite key not 0 but NaN: masked in whole tiles too.
      const int live = a.tile_tokens * a.group;
      uint32_t n = 0, x = 0, mine_n = 0, joins = 0;
      bool ok = true;  // as above
      for (KeyWalk w(p.m, blockIdx.x); w.live(); w.next(), ++n) {
        const int u0 = w.j * kM, u = u0 + r, size = w.k.prefix + w.k.L, row0 = a.intervals[w.i].begin;
        const int count = w.r1 - w.r0;
        float f = p.scale_log2;
        if (Q8) {
          ok = ok && warp_wait(&bars->sc_full[n % 4], (n / 4) & 1, abort_flag, budget);
          f = reinterpret_cast<const float*>(smem + L::kScale)[n % 4 * kM + r];
          mbar_arrive_warp(&bars->sc_empty[n % 4]);
        }
        const unsigned long long fx2 = f2pack(f, f);
        float sum = 0.f;
        auto fetch = [&](int q) {  // -lse of this thread's column of row tile q
          const int token = w.k.token(w.j) + q * a.tile_tokens + tok;
          return q < w.r1 && tok < a.tile_tokens && token < w.k.L
                     ? -lse[(int64_t)(row0 + token) * a.h_q + w.head * a.group + r % a.group]
                     : -INFINITY;
        };
        const int q0 = w.r0 + (int)((x + grp) & 1);  // this group's first row tile: the sequence's tiles of its parity
        float ahead = fetch(q0);
        for (int q = q0; q < w.r1; q += 2, ++mine_n) {
          const uint32_t y = x + (q - w.r0);
          float* ml = minus + (mine_n & 1) * kM;
          ml[r] = ahead;
          ahead = fetch(q + 2);
          group_sync(grp);
          ok = ok && warp_wait(&bars->s_full[y % 4], (y / 4) & 1, abort_flag, budget);
          tc_fence_after();
          const int token0 = w.k.token(w.j) + q * a.tile_tokens;
          const int rows = min(a.tile_tokens, w.k.L - token0) * a.group;       // columns that are rows of the question
          const int from = max(0, u - w.k.prefix - token0) * a.group;          // the first that sees this thread's key
          // whole: every row of the tile sees every key
          const bool whole = rows == live && u0 + kM - 1 <= w.k.prefix + token0;
          const ulonglong2* ml2 = reinterpret_cast<const ulonglong2*>(ml);
          unsigned long long s2[4] = {0, 0, 0, 0};
          uint32_t v[2][32];
          tmem_ld32(tm + y % 4 * kM, v[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 32 columns at a time, the next ones on their way
            uint32_t(&s)[32] = v[c & 1];
            tmem_ld_wait(s);
            if (c < 3) {
              tmem_ld32(tm + y % 4 * kM + 32 * (c + 1), v[(c + 1) & 1]);
            } else {
              tc_fence_before();
              mbar_arrive_warp(&bars->s_free[y % 4]);
            }
            auto weights = [&](auto masked) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const ulonglong2 nl = ml2[8 * c + e / 4];
                float2 z0 = unpack2(fma2((unsigned long long)s[e] | (unsigned long long)s[e + 1] << 32, fx2, nl.x));
                float2 z1 = unpack2(fma2((unsigned long long)s[e + 2] | (unsigned long long)s[e + 3] << 32, fx2, nl.y));
                const int col = 32 * c + e;
                if (decltype(masked)::value == 1 && e >= 16) {
                  z0.x = col >= live ? -INFINITY : z0.x;
                  z0.y = col + 1 >= live ? -INFINITY : z0.y;
                  z1.x = col + 2 >= live ? -INFINITY : z1.x;
                  z1.y = col + 3 >= live ? -INFINITY : z1.y;
                }
                if (decltype(masked)::value == 2) {
                  z0.x = col < from || col >= rows ? -INFINITY : z0.x;
                  z0.y = col + 1 < from || col + 1 >= rows ? -INFINITY : z0.y;
                  z1.x = col + 2 < from || col + 2 >= rows ? -INFINITY : z1.x;
                  z1.y = col + 3 < from || col + 3 >= rows ? -INFINITY : z1.y;
                }
                s2[(e >> 1) & 3] = add2(s2[(e >> 1) & 3], f2pack(ex2_approx(z0.x), ex2_approx(z0.y)));
                s2[((e >> 1) + 1) & 3] = add2(s2[((e >> 1) + 1) & 3], f2pack(ex2_approx(z1.x), ex2_approx(z1.y)));
              }
            };
            if (!whole) weights(std::integral_constant<int, 2>{});
            else if (c == 3 && live < kM) weights(std::integral_constant<int, 1>{});
            else weights(std::integral_constant<int, 0>{});
          }
          const float2 s0 = unpack2(add2(add2(s2[0], s2[1]), add2(s2[2], s2[3])));
          sum += s0.x + s0.y;
        }
        x += count;
        bool writes = q0 == w.r0;  // of a unit of one row tile, the group that had it
        if (count > 1) {
          if (grp == 1) other[(joins & 1) * kM + r] = sum;
          both_sync();
          if (grp == 0) sum += other[(joins & 1) * kM + r];
          ++joins;
          writes = grp == 0;
        }
        if (!writes) continue;
        const int64_t cell = ((int64_t)a.table[(int64_t)w.i * a.max_blocks + w.j] * a.h_kv + w.head) * kPage + r;
        bool last = true;
        if (!w.whole()) {
          const int first = w.first(blockIdx.x), parts = w.parts();
          __stcg(part + (2 * (int64_t)blockIdx.x + (w.r0 == 0)) * kM + r, sum);
          __threadfence();
          group_sync(grp);
          if (r == 0) *reinterpret_cast<volatile int*>(&bars->last[grp]) = atomicAdd(arrived + first * kSpanRows, 1) == parts - 1;
          group_sync(grp);
          last = *reinterpret_cast<volatile int*>(&bars->last[grp]);
          group_sync(grp);
          if (last) {
            __threadfence();
            sum = 0.f;
            for (int c = 0; c < parts; ++c) sum += __ldcg(part + (2 * (int64_t)(first + c) + (c == 0)) * kM + r);
          }
        }
        if (ok && last && u < size) {
          float* to = p.m.mass + cell;
          *to = u < w.k.prefix && p.m.decay != 0.f ? fmaf(p.m.decay, *to, sum) : sum;
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool Q8>
cudaError_t launch(const MassArgs& m, int num_sms, cudaStream_t s) {
  const SpanArgs& a = m.s;
  TcArgs p;
  p.m = m;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wait_budget = wait_budget_cycles();
  p.test_stall = test_stall_requested();
  CUtensorMap mq = {}, mk = {};
  const cuuint64_t q_dims[3] = {(cuuint64_t)D, (cuuint64_t)a.h_q, (cuuint64_t)a.T};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.tile_tokens};
  bool ok = span_tensor_map(&mq, a.q, 2, 3, q_dims, q_box, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!Q8) {
    const cuuint64_t pool[2] = {(cuuint64_t)D, (cuuint64_t)a.n_blocks * a.h_kv * kPage};
    const cuuint32_t box[2] = {64, 128};
    ok = ok && span_tensor_map(&mk, a.pool_k, 2, 2, pool, box, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  if (!ok) return cudaErrorInvalidValue;
  constexpr int rows_smem = RowsSmem<D, Q8>::kBytes, keys_smem = KeysSmem<D, Q8>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(mass_rows_tc_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(mass_keys_tc_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, keys_smem);
  if (e == cudaSuccess) e = launch_pdl(mass_rows_tc_kernel<D, Q8>, dim3(a.ctas), dim3(kThreads), rows_smem, s, mq, mk, p);
  if (e == cudaSuccess) e = launch_pdl(mass_cuts_kernel, dim3(1 + num_sms), dim3(256), sizeof(long long) * ((size_t)a.n + 1), s, m);
  if (e == cudaSuccess) e = launch_pdl(mass_keys_tc_kernel<D, Q8>, dim3(a.ctas), dim3(kThreads), keys_smem, s, mq, mk, p);
  return e;
}

}  // namespace

size_t mass_cuts_bytes() { return sizeof(KeyCut) * (kSpanMaxCtas + 1); }

cudaError_t launch_mass_tc(const MassArgs& m, int num_sms, cudaStream_t s) {
  if (m.s.pool_elem == 1) return m.s.d == 64 ? launch<64, true>(m, num_sms, s) : launch<128, true>(m, num_sms, s);
  return m.s.d == 64 ? launch<64, false>(m, num_sms, s) : launch<128, false>(m, num_sms, s);
}

}  // namespace kev
