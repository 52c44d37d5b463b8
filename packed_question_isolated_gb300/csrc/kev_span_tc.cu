// Span attention on the 5th-generation tensor cores: bf16 q and out, cache (or packed rows) bf16
// or e4m3, fp32 accumulation.
//
// out = softmax(scale q K^T + M) V over the visible positions, tile by tile with a running
// reference maximum m and sum l per row.  A row tile is 128 (token, q-head of the group) rows of
// one question and kv head -- 32 tokens at G = 4 -- so all G heads share every K/V tile that is
// loaded, and a short chunk still fills most of an MMA.  A unit is up to two row tiles A and B of
// consecutive tokens over the same key tiles (128 positions: one page).
//
// One persistent CTA per SM, 16 warps; each walks its equal part of the work line (kev_span.cuh):
//   warps 0-3, 4-7   softmax of tiles A, B: a thread owns a row (its TMEM lane): S from TMEM, mask on
//                    tiles where some row does not see every key, P = exp2(scale log2e s - m) as bf16
//                    over S in TMEM; the accumulator is rescaled only when the exponentials
//                    outgrow 2^64 (m is a reference, not the exact maximum: exact either way, since
//                    O and l share it); the epilogue divides by l, or stores a partial result
//   warp 8           loads K and V tiles (TMA; e4m3: bulk copies of the codes and scales of a page)
//   warps 9, 11      issue the MMAs of A and B in turns: S = Q K^T, then O += P V with P from TMEM
//   warp 10          loads the q tiles: a 3-D box of tokens x group heads x 64 dims
//   warps 12-15      make the loaded tiles ready.  bf16: on tiles with masked keys, NaN and infinities
//                    in V become zeros (0 x NaN would reach rows that do not see the key; the
//                    epilogue puts them back for the rows that do, by a flag per unit; where it
//                    reads the flag moves the whole kernel by up to 2 %).  e4m3: the codes become
//                    bf16, which holds every e4m3 value exactly, in the MMA's swizzled layout; the
//                    scales multiply S (K) and P (V) in fp32 instead, so quantisation is the only
//                    loss.
// What bounds it.  With many rows the shared-memory reads of the MMA operands, which share the 128 bytes a
// clock with the loads: S and PV of a 128 x 128 x 128 tile take about 750 clocks instead of 512, and the two
// row tiles' softmax (about 1450 clocks each) and MMAs then fill each other's gaps to about 3300 clocks a key
// tile.  Over e4m3 the codes' way through shared memory adds 96 KB a key tile and bounds it at about 4100.
// With few rows the latency of one key tile's chain, S - softmax - PV.  Measured on a GB300 at the clocks it
// keeps under load: 27k tokens under a window of 2048 715 to 750 us, from one GPU to the next (766 GFLOP useful,
// 1.02 to 1.07 PFLOP/s, 53 to 56 % of the measured burst peak); 8 chunks of 128 to 1024 tokens over bf16 caches
// 132 us, over e4m3 ones of up to 16k positions 337 us (0.64 PFLOP/s); 8 prompts under a window of 512 99 us, 64
// short ones at d = 64 59 us.
// Why these tiles: all G heads of a group on one row tile load each K/V tile once and waste nothing on short
// chunks; two row tiles per CTA are what 512 columns of tensor memory hold (S and O in fp32, P over S).
// Measured and left: scores in pieces of 32 keys, for fewer registers (855 us against 729); a ring of 5
// slots (734 against 729); q and K as fp16 over e4m3, whose conversion is a quarter of the bf16 one's
// instructions (370 against 338: shared memory bounds it, not they).  Every wait is bounded, as in the
// other tensor-core kernels.
#include <cuda.h>
#include <cuda_fp16.h>

#include "kev_sm100.cuh"
#include "kev_span.cuh"

namespace kev {
namespace {

using namespace sm100;

constexpr int kBM = 128, kBN = kSpanKeys;
constexpr int kThreads = 512;
constexpr int kLoadWarp = 8, kMmaWarpA = 9, kQWarp = 10, kMmaWarpB = 11, kReadyWarp = 12;
// 128 registers a thread at launch: 256 x 200 + 256 x 56 = 512 x 128
constexpr int kRegsSoftmax = 200, kRegsOther = 56;
constexpr uint32_t kTmemCols = 512;
constexpr float kOverflowSum = 1.8446744e19f;  // 2^64
constexpr long long kDrainBudget = 4000000000ll;
constexpr int kScaleSlots = 4;
// Over e4m3 the weight times V's scale is what becomes bf16, and a bf16 value's scale may be 2^-135 (of a subnormal
// one 2^-142): the weights start 2^24 higher, so the product stays a normal bf16 number down to weights of 2^-15 at
// that scale.  O and l share the factor.
constexpr float kLift = 24.f;

template <int D, bool Q8>
struct Smem {
  static constexpr int kSub = D / 64;             // 128-byte sub-tiles of a row
  static constexpr int kSubBytes = kBM * 128;
  static constexpr int kTile = kBM * D * 2;       // one bf16 tile
  static constexpr int kCodes = kBN * D;          // one tile of codes
  // K and V tiles share a ring, K(0) V(0) K(1) V(1) ...; with e4m3 it is fed from a ring of code tiles
  static constexpr int kRing = Q8 ? 3 : 4;
  static constexpr int kStages = Q8 ? 3 : 1;
  static constexpr int kQ = 0;
  static constexpr int kKv = 2 * kTile;
  static constexpr int kStage = kKv + kRing * kTile;
  static constexpr int kScale = kStage + (Q8 ? kStages * kCodes : 0);  // {K, V} scales of 4 key tiles
  static constexpr int kBar = kScale + (Q8 ? kScaleSlots * 2 * kBN * 4 : 0);
  static constexpr int kBytes = kBar + 1024 + 1024;  // slack for 1024-byte alignment
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t full[4], empty[4], ready[4];  // ring slot: loaded (bf16), read by both MMAs, ready for them
  uint64_t st_full[4], st_empty[4];      // e4m3: code tile loaded, converted
  uint64_t sc_full[kScaleSlots];         // e4m3: scales of a key tile visible
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t drain[2];
  uint64_t stall;  // timeout test hook: nothing ever arrives on it
  uint32_t tmem;
  int abort;
  int never;
  // [u % 64]: unit u (or one that many times 64 before it) has NaN or infinities in V (e4m3: in its scales) at
  // tiles with masked keys.  Never cleared: nothing holds the next units' tiles back until an epilogue has read it
  int bad[64];
};
static_assert(sizeof(Bars) <= 1024, "barriers");

struct TcArgs {
  SpanArgs s;
  float scale_log2;
  long long wait_budget;
  int32_t test_stall;  // timeout test hook
};

__device__ __forceinline__ void raise_timeout(const TcArgs& p, Bars* b) {
  atomicCAS(&reinterpret_cast<SpanHeader*>(p.s.ws)->status, 0, ST_TIMEOUT);
  set_status(p.s.dev_status, ST_TIMEOUT);
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

// Tile at(j) has a key that some row of the item does not see.
__device__ __forceinline__ bool edge_tile(const SpanArgs& a, int u0, int p0, int p1) {
  const int u1 = u0 + kBN - 1;
  return !(u1 <= p0 && (a.window == 0 || p1 - u0 < a.window || u1 < a.sinks));
}

// four e4m3 codes as bf16 pairs, exactly: by way of fp16 and fp32 (placing the bits takes four integer
// operations per pair, on the pipe that the softmax needs most)
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

// bits e of word c (keys 32 c + e) with lo <= key <= hi, or key < below
__device__ __forceinline__ uint32_t seen_bits(int c, int hi, int lo, int below) {
  auto under = [&](int n) {  // keys < n
    n -= 32 * c;
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
  };
  return under(hi + 1) & (~under(lo) | under(below));
}

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    span_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ TcArgs p) {
  using L = Smem<D, Q8>;
  const SpanArgs& a = p.s;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 2);
      mbar_init(&bars->ready[s], 4);
      mbar_init(&bars->st_full[s], 1);
      mbar_init(&bars->st_empty[s], 4);
      mbar_init(&bars->sc_full[s], 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->o_done[t], 1);
      mbar_init(&bars->o_free[t], 4);
      mbar_init(&bars->drain[t], 1);
    }
    mbar_init(&bars->stall, 1);
    bars->abort = 0;
    bars->never = 0;
    for (int u = 0; u < 64; ++u) bars->bad[u] = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tm_q);
    if (!Q8) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  if (warp == kMmaWarpA) {
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  // TMEM columns: S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [256+D,256+2D)
  volatile int* abort_flag = &bars->abort;
  const volatile int* never = &bars->never;
  const long long budget = p.wait_budget;

  pdl_wait();  // the plan, and the chunk's rows in the cache
  pdl_trigger();
  const bool go = reinterpret_cast<const SpanHeader*>(a.ws)->status == ST_OK;

  if (warp >= kLoadWarp) {
    regs_dec<kRegsOther>();
    if (!go) {
    } else if (warp == kLoadWarp) {
      // ------------------------------------------------------------------ K/V loads
      if (lane == 0) {
        constexpr int kSlots = Q8 ? L::kStages : L::kRing;
        uint64_t* full = Q8 ? bars->st_full : bars->full;
        uint64_t* empty = Q8 ? bars->st_empty : bars->empty;
        uint32_t seq = 0, tiles_done = 0;
        bool ok = !(p.test_stall && blockIdx.x == 0) || mbar_wait(&bars->stall, 0, abort_flag, budget);
        for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next()) {
          const SpanTiles tiles(w.item.p0, w.item.p0 + w.item.tokens - 1, a.window, a.sinks);
          const int32_t* row = a.table ? a.table + (int64_t)w.item.question * a.max_blocks : nullptr;
          int block = a.table ? row[tiles.at(w.j0)] : 0;
          for (int j = w.j0; ok && j < w.j1; ++j, ++tiles_done) {
            const int here = block;
            if (a.table && j + 1 < w.j1) block = row[tiles.at(j + 1)];  // one tile ahead
            for (int is_v = 0; is_v < 2; ++is_v, ++seq) {
              const int s = seq % kSlots;
              if (seq >= kSlots && !mbar_wait(&empty[s], (seq / kSlots - 1) & 1, abort_flag, budget)) {
                ok = false;
                break;
              }
              if (Q8) {
                const int64_t cell = ((int64_t)here * a.h_kv + w.head) * kPage;
                mbar_arrive_expect_tx(&full[s], L::kCodes + (is_v ? 0 : 2 * kBN * 4));
                bulk_load(smem + L::kStage + s * L::kCodes, static_cast<const char*>(is_v ? a.pool_v : a.pool_k) + cell * D,
                          L::kCodes, &full[s]);
                if (!is_v) {  // both scales with the K tile: the softmax wants them before V
                  unsigned char* sc = smem + L::kScale + tiles_done % kScaleSlots * (2 * kBN * 4);
                  bulk_load(sc, a.scale_k + cell, kBN * 4, &full[s]);
                  bulk_load(sc + kBN * 4, a.scale_v + cell, kBN * 4, &full[s]);
                }
              } else {
                mbar_arrive_expect_tx(&full[s], L::kTile);
                const int x = a.table ? 0 : w.head * D;
                const int y = a.table ? (here * a.h_kv + w.head) * kPage : w.item.row0 - w.item.p0 + tiles.at(j) * kBN;
                for (int c = 0; c < L::kSub; ++c)
                  tma_load_2d(smem + L::kKv + s * L::kTile + c * L::kSubBytes, is_v ? &tm_v : &tm_k, x + c * 64, y, &full[s]);
              }
            }
          }
        }
        if (!ok) raise_timeout(p, bars);
        if (*abort_flag)  // every copy issued lands before the CTA leaves
          for (uint32_t q = seq < kSlots ? 0 : seq - kSlots; q < seq; ++q)
            mbar_wait(&full[q % kSlots], (q / kSlots) & 1, never, kDrainBudget);
      }
    } else if (warp == kQWarp) {
      // ------------------------------------------------------------------ q loads
      if (lane == 0) {
        uint32_t n = 0;
        bool ok = true;
        for (SpanWalk w(a, blockIdx.x); w.live(); w.next(), ++n) {
          if (n > 0 && !mbar_wait(&bars->q_empty, (n - 1) & 1, abort_flag, budget)) {
            ok = false;
            break;
          }
          const int nt = w.item.tokens > a.tile_tokens ? 2 : 1;
          mbar_arrive_expect_tx(&bars->q_full, nt * L::kSub * 128 * a.group * a.tile_tokens);
          for (int t = 0; t < nt; ++t)
            for (int c = 0; c < L::kSub; ++c)
              tma_load_3d(smem + L::kQ + t * L::kTile + c * L::kSubBytes, &tm_q, c * 64, w.head * a.group,
                          w.item.row0 + t * a.tile_tokens, &bars->q_full);
        }
        if (!ok) raise_timeout(p, bars);
        if (*abort_flag && n) mbar_wait(&bars->q_full, (n - 1) & 1, never, kDrainBudget);
      }
    } else if (warp == kMmaWarpA || warp == kMmaWarpB) {
      // ------------------------------------------------------------------ MMA issue
      // Strict turns on the tensor core (as in the single-CTA prefill kernel): a group is PV of one
      // key tile, then S of the next, of one row tile; B's softmax runs while A's group executes.
      const int t = warp == kMmaWarpA ? 0 : 1;
      const bool leader = lane == 0;
      constexpr uint32_t idesc_s = idesc_bf16(kBM, kBN, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(kBM, D, false, true);
      uint32_t seq = 0, n = 0, p_cnt = 0, units = 0;
      bool ok = true, first_turn = true;
      auto wait_ok = [&](uint64_t* bar, uint32_t parity) {
        if (!ok) return;
        ok = warp_wait(bar, parity, abort_flag, budget);
        if (!ok) *abort_flag = 1;
      };
      auto take_turn = [&]() {
        if (t == 1) asm volatile("bar.sync 2, 64;" ::: "memory");
        else if (!first_turn) asm volatile("bar.sync 3, 64;" ::: "memory");
        first_turn = false;
      };
      auto pass_turn = [&]() {
        __syncwarp();
        if (t == 0) asm volatile("bar.arrive 2, 64;" ::: "memory");
        else asm volatile("bar.arrive 3, 64;" ::: "memory");
      };
      auto issue_s = [&](int slot) {
        const uint32_t q_addr = smem_u32(smem + L::kQ + t * L::kTile), k_addr = smem_u32(smem + L::kKv + slot * L::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * L::kSubBytes + (kk & 3) * 32;
          umma_bf16(tmem + t * kBN, sdesc_sw128(q_addr + off, 16, 1024), sdesc_sw128(k_addr + off, 16, 1024), idesc_s, kk > 0);
        }
        umma_commit(&bars->s_full[t]);
      };
      auto issue_pv = [&](int slot, bool accumulate) {
        const uint32_t v_addr = smem_u32(smem + L::kKv + slot * L::kTile);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          umma_bf16_ts(tmem + 256 + t * D, tmem + t * kBN + kk * 8, sdesc_sw128(v_addr + kk * 16 * 128, L::kSubBytes, 1024),
                       idesc_o, (accumulate || kk > 0) ? 1u : 0u);
      };
      auto slot = [](uint32_t q) { return (int)(q % L::kRing); };
      auto phase = [](uint32_t q) { return (q / L::kRing) & 1; };

      for (SpanWalk w(a, blockIdx.x); w.live(); w.next(), ++n) {
        const bool mine = t == 0 || w.item.tokens > a.tile_tokens;
        const int nkv = w.j1 - w.j0;
        wait_ok(&bars->q_full, n & 1);
        wait_ok(&bars->ready[slot(seq)], phase(seq));
        take_turn();
        if (ok && leader) {
          tc_fence_after();
          if (mine) issue_s(slot(seq));
          umma_commit(&bars->empty[slot(seq)]);
          if (nkv == 1) umma_commit(&bars->q_empty);
        }
        pass_turn();
        for (int j = 0; j < nkv; ++j, seq += 2) {
          const int vs = slot(seq + 1), kn = slot(seq + 2);
          const bool more = j + 1 < nkv;
          wait_ok(&bars->ready[vs], phase(seq + 1));
          if (more) wait_ok(&bars->ready[kn], phase(seq + 2));
          if (mine) {
            wait_ok(&bars->p_full[t], p_cnt & 1);
            if (j == 0 && units > 0) wait_ok(&bars->o_free[t], (units - 1) & 1);
            ++p_cnt;
          }
          take_turn();
          if (ok && leader) {
            tc_fence_after();
            if (mine) issue_pv(vs, j > 0);
            umma_commit(&bars->empty[vs]);
            if (mine && !more) umma_commit(&bars->o_done[t]);
            if (more) {
              if (mine) issue_s(kn);  // over S_t / P_t, which the PV above has read (in order)
              umma_commit(&bars->empty[kn]);
              if (j + 2 == nkv) umma_commit(&bars->q_empty);
            }
          }
          pass_turn();
        }
        if (mine) ++units;
      }
      if (t == 0 && !first_turn) asm volatile("bar.sync 3, 64;" ::: "memory");  // B's last hand-over
      if (!ok && leader) raise_timeout(p, bars);
      if (leader) {  // every MMA issued is complete before TMEM is freed
        umma_commit(&bars->drain[t]);
        mbar_wait(&bars->drain[t], 0, never, kDrainBudget);
      }
      __syncwarp();
    } else if (warp >= kReadyWarp) {
      // ------------------------------------------------------------------ tiles made ready
      const int x = threadIdx.x - kReadyWarp * 32;
      uint32_t seq = 0, n = 0, tiles_done = 0;
      bool ok = true;
      for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next(), ++n) {
        const int p0 = w.item.p0, p1 = p0 + w.item.tokens - 1;
        const SpanTiles tiles(p0, p1, a.window, a.sinks);
        for (int j = w.j0; ok && j < w.j1; ++j, ++tiles_done) {
          const bool edge = edge_tile(a, tiles.at(j) * kBN, p0, p1);
          for (int is_v = 0; is_v < 2; ++is_v, ++seq) {
            const int s = seq % L::kRing;
            unsigned char* tile = smem + L::kKv + s * L::kTile;
            if (!Q8) {
              if (!warp_wait(&bars->full[s], (seq / L::kRing) & 1, abort_flag, budget)) {
                ok = false;
                break;
              }
              if (is_v && edge) {
                uint4* at = reinterpret_cast<uint4*>(tile) + x;
                // a half with all exponent bits carries into its top bit
                auto bad_bits = [](uint32_t u) { return ((u & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                uint32_t any = 0;
#pragma unroll 8
                for (int e = 0; e < L::kTile / 16 / 128; ++e) {
                  const uint4 v = at[e * 128];
                  any |= bad_bits(v.x) | bad_bits(v.y) | bad_bits(v.z) | bad_bits(v.w);
                }
                if (any) {
#pragma unroll 1
                  for (int e = 0; e < L::kTile / 16 / 128; ++e) {
                    uint4 v = at[e * 128];
                    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                      const uint32_t b = bad_bits(u[i]);
                      if (b & 0x8000u) u[i] &= 0xffff0000u;
                      if (b & 0x80000000u) u[i] &= 0x0000ffffu;
                    }
                    at[e * 128] = v;
                  }
                }
                if (__any_sync(0xffffffffu, any != 0)) {
                  if (lane == 0) *reinterpret_cast<volatile int*>(&bars->bad[n & 63]) = 1;
                  fence_proxy_async_smem();
                }
              }
              mbar_arrive_warp(&bars->ready[s]);
            } else {
              const int st = seq % L::kStages;
              if (!warp_wait(&bars->st_full[st], (seq / L::kStages) & 1, abort_flag, budget) ||
                  (seq >= L::kRing && !warp_wait(&bars->empty[s], (seq / L::kRing - 1) & 1, abort_flag, budget))) {
                ok = false;
                break;
              }
              if (!is_v) {
                // This thread's key: K's factor with the softmax's (1 for a row of zeros, whose scores are 0;
                // a row with a NaN scale has NaN codes), never 0, which would make NaN of the -inf of a row that
                // does not see the key (as a normal number at the least: scores of such keys are 0 to within
                // 2^-126 q . codes); and V's, where a NaN or an infinity at a tile with masked keys becomes 0: the
                // epilogue makes NaN of the rows that see it
                float* sc = reinterpret_cast<float*>(smem + L::kScale) + tiles_done % kScaleSlots * (2 * kBN) + x;
                const float k = sc[0], v = sc[kBN];
                sc[0] = k > 0.f ? fmaxf(k * p.scale_log2, 1.17549435e-38f) : 1.f;
                if (edge && !(fabsf(v) <= 3.4028235e38f)) {
                  sc[kBN] = 0.f;
                  *reinterpret_cast<volatile int*>(&bars->bad[n & 63]) = 1;
                }
                mbar_arrive_warp(&bars->sc_full[tiles_done % kScaleSlots]);
              }
              const uint4* codes = reinterpret_cast<const uint4*>(smem + L::kStage + st * L::kCodes);
              const uint32_t dst = smem_u32(tile);
              constexpr int kGroups = D / 16;  // 16-code groups of a row
#pragma unroll 4
              for (int e = 0; e < kBN * kGroups / 128; ++e) {
                const int at = e * 128 + x, r = at / kGroups, g = at % kGroups;
                uint4 c = codes[at];
                if (is_v && edge) {  // and NaN codes become 0
                  uint32_t* u = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
                  for (int i = 0; i < 4; ++i) u[i] &= ~(((((u[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
                }
                uint32_t o[8];
                e4m3_to_bf16(c.x, o[0], o[1]);
                e4m3_to_bf16(c.y, o[2], o[3]);
                e4m3_to_bf16(c.z, o[4], o[5]);
                e4m3_to_bf16(c.w, o[6], o[7]);
                // 16-byte chunks 2 (g % 4) and + 1 of sub-tile g / 4, XOR-ed with r % 8; lanes of the second
                // sub-tile store theirs the other way round, so a quarter warp hits every bank once
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
              fence_proxy_async_smem();
              mbar_arrive_warp(&bars->ready[s]);
              mbar_arrive_warp(&bars->st_empty[st]);
            }
          }
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax and epilogue
    if (go) {
      span_zero_gaps(a, 256);
      const int t = warp >> 2, r = (warp & 3) * 32 + lane;  // row tile, row (a warp reaches TMEM lanes 32 (warp % 4) ..)
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tm_s = tmem + t * kBN + lane_off, tm_o = tmem + 256 + t * D + lane_off;
      const float sl2 = Q8 ? 1.f : p.scale_log2;  // e4m3: in the keys' factors
      constexpr float lift = Q8 ? kLift : 0.f;
      const unsigned long long sl2x2 = f2pack(sl2, sl2);
      const int tok = r / a.group;  // token of the tile
      uint32_t s_cnt = 0, o_cnt = 0, n = 0, tiles_done = 0;
      bool ok = true;

      for (SpanWalk w(a, blockIdx.x); ok && w.live(); w.next(), ++n) {
        const int p0 = w.item.p0, p1 = p0 + w.item.tokens - 1;
        if (t == 1 && w.item.tokens <= a.tile_tokens) {  // no tile B
          tiles_done += w.j1 - w.j0;
          continue;
        }
        const SpanTiles tiles(p0, p1, a.window, a.sinks);
        const int token = t * a.tile_tokens + tok;
        const bool row_ok = tok < a.tile_tokens && token < w.item.tokens;
        const int pos = p0 + token;
        const bool warp_ok = __any_sync(0xffffffffu, row_ok);  // else: nothing of these rows is stored
        float m_run = -INFINITY, l_run = 0.f;

        for (int j = w.j0; j < w.j1; ++j, ++tiles_done) {
          const int u0 = tiles.at(j) * kBN;
          const bool edge = edge_tile(a, u0, p0, p1);
          const float4* sc = reinterpret_cast<const float4*>(smem + L::kScale + tiles_done % kScaleSlots * (2 * kBN * 4));
          // Keys this row sees, as bits.  A warp's few tokens agree on most words of 32 keys: bit c of `full` where
          // all its rows see all of word c.
          uint32_t seen[4], full = 0;
          auto look = [&]() {
            if (!edge) return;
            const int hi = pos - u0, lo = a.window ? hi - a.window + 1 : 0, below = a.sinks - u0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              seen[c] = seen_bits(c, hi, lo, below);
              full |= (unsigned)__all_sync(0xffffffffu, seen[c] == 0xffffffffu) << c;
            }
          };
          if (!Q8) look();  // while S is computed (over e4m3 the registers are short: 344 us against 339 so)
          if (!warp_wait(&bars->s_full[t], s_cnt & 1, abort_flag, budget) ||
              (Q8 && !warp_wait(&bars->sc_full[tiles_done % kScaleSlots], (tiles_done / kScaleSlots) & 1, abort_flag, budget))) {
            ok = false;
            break;
          }
          ++s_cnt;
          tc_fence_after();
          if (!warp_ok) {
            tc_fence_before();
            mbar_arrive_warp(&bars->p_full[t]);
            continue;
          }
          uint32_t sr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tm_s + c * 32, sr[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_wait(sr[c]);
          if (Q8) look();
          if (edge) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (full >> c & 1u) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(seen[c] >> e & 1u)) sr[c][e] = __float_as_uint(-INFINITY);
            }
          }
          auto row_max = [&]() -> float {
            float mp[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) mp[q] = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                float4 k = make_float4(1.f, 1.f, 1.f, 1.f);
                if (Q8) k = sc[c * 8 + e / 4];
                const int q = e / 4;
                mp[q] = fmax3(mp[q], __uint_as_float(sr[c][e]) * k.x, __uint_as_float(sr[c][e + 1]) * k.y);
                mp[q] = fmax3(mp[q], __uint_as_float(sr[c][e + 2]) * k.z, __uint_as_float(sr[c][e + 3]) * k.w);
              }
            return fmax3(fmax3(mp[0], mp[1], mp[2]), fmax3(mp[3], mp[4], mp[5]), fmaxf(mp[6], mp[7])) * sl2;
          };
          // P into the first 64 columns of S_t; returns the row's sum of the weights
          auto exp_tile = [&](float m) -> float {
            const unsigned long long negm = f2pack(-m, -m);
            unsigned long long accs[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const unsigned long long sv = (unsigned long long)sr[c][2 * e] | ((unsigned long long)sr[c][2 * e + 1] << 32);
                const unsigned long long k = Q8 ? reinterpret_cast<const unsigned long long*>(sc)[c * 16 + e] : sl2x2;
                const float2 z = unpack2(fma2(sv, k, negm));
                unsigned long long w = f2pack(ex2_approx(z.x), ex2_approx(z.y));
                accs[e & 3] = add2(accs[e & 3], w);
                if (Q8) w = mul2(w, reinterpret_cast<const unsigned long long*>(sc)[kBN / 2 + c * 16 + e]);  // V's scales
                const float2 x = unpack2(w);
                pk[e] = pack_bf16x2(x.x, x.y);
              }
              tmem_st16(tm_s + c * 16, pk);
            }
            const float2 acc = unpack2(add2(add2(accs[0], accs[1]), add2(accs[2], accs[3])));
            return acc.x + acc.y;
          };
          // The first tile in which a row sees a key sets its reference; a later one moves it only
          // when the weights approach the end of the fp32 range.
          if (__any_sync(0xffffffffu, row_ok && m_run == -INFINITY)) {
            const float mt = row_max() - lift;
            if (m_run == -INFINITY) m_run = mt;
          }
          float lt = exp_tile(m_run == -INFINITY ? 0.f : m_run);
          const bool big = row_ok && !(lt <= kOverflowSum);
          if (__any_sync(0xffffffffu, big)) {
            float alpha = 1.f;
            if (big) {
              const float mt = fmaxf(row_max() - lift, m_run);
              alpha = ex2_approx(m_run - mt);
              m_run = mt;
              l_run *= alpha;
            }
            lt = exp_tile(m_run == -INFINITY ? 0.f : m_run);
            if (j > w.j0) {  // PV of the tile before is complete (S_t came after it); the first PV overwrites O
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tm_o + c * 32, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st32(tm_o + c * 32, o);
              }
            }
          }
          l_run += lt;
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(&bars->p_full[t]);
        }
        if (!ok) break;

        if (!warp_wait(&bars->o_done[t], o_cnt & 1, abort_flag, budget)) {
          ok = false;
          break;
        }
        ++o_cnt;
        tc_fence_after();
        const bool bad = *reinterpret_cast<volatile int*>(&bars->bad[n & 63]);  // at worst nothing is found to put back
        uint32_t o[D / 32][32];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tm_o + c * 32, o[c]);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld_wait(o[c]);
        tc_fence_before();
        mbar_arrive_warp(&bars->o_free[t]);
        if (bad && row_ok) {
          // V's NaN and infinities at tiles with masked keys were left out of the products: add those
          // that this row sees
          for (int j = w.j0; j < w.j1; ++j) {
            const int u0 = tiles.at(j) * kBN;
            if (!edge_tile(a, u0, p0, p1)) continue;
            for (int u = u0; u < u0 + kBN && u <= pos; ++u) {
              if (!span_sees(pos, u, a.window, a.sinks)) continue;
              if (Q8) {
                const int64_t cell =
                    ((int64_t)a.table[(int64_t)w.item.question * a.max_blocks + u / kPage] * a.h_kv + w.head) * kPage + u % kPage;
                if (!(fabsf(a.scale_v[cell]) <= 3.4028235e38f)) l_run = __int_as_float(0x7fffffff);
                continue;
              }
              const uint4* v = reinterpret_cast<const uint4*>(
                  a.table ? static_cast<const __nv_bfloat16*>(a.pool_v) +
                                (((int64_t)a.table[(int64_t)w.item.question * a.max_blocks + u / kPage] * a.h_kv + w.head) * kPage +
                                 u % kPage) * D
                          : static_cast<const __nv_bfloat16*>(a.v) +
                                ((int64_t)(w.item.row0 - p0 + u) * a.h_kv + w.head) * D);
#pragma unroll
              for (int c = 0; c < D / 8; ++c) {
                const uint4 x = v[c];
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t& o0 = o[c / 4][c % 4 * 8 + 2 * e];
                  uint32_t& o1 = o[c / 4][c % 4 * 8 + 2 * e + 1];
                  if ((y[e] & 0x7f80u) == 0x7f80u) o0 = __float_as_uint(__uint_as_float(o0) + __uint_as_float(y[e] << 16));
                  if ((y[e] & 0x7f800000u) == 0x7f800000u)
                    o1 = __float_as_uint(__uint_as_float(o1) + __uint_as_float(y[e] & 0xffff0000u));
                }
              }
            }
          }
        }
        if (!warp_ok) continue;
        if (!w.whole()) {
          // A piece of a unit.  Of two, the warp that comes second joins both, its own from registers and in
          // the order of the pieces; more are left to the merge kernel.
          const int first = w.first(), parts = w.parts(), row = t * kBM + r;
          const bool mine_first = w.j0 == 0;
          float* po = reinterpret_cast<float*>(a.ws + a.layout.part_o);
          float2* ml = reinterpret_cast<float2*>(a.ws + a.layout.part_ml);
          int32_t* arrived = reinterpret_cast<int32_t*>(a.ws + a.line.arrived) + first * kSpanRows + warp;
          int there = 0;
          if (parts == 2) {
            if (lane == 0) asm volatile("ld.acquire.gpu.b32 %0, [%1];" : "=r"(there) : "l"(arrived) : "memory");
            there = __shfl_sync(0xffffffffu, there, 0);
          }
          if (!there) {
            const int64_t slot = w.slot(blockIdx.x);
            if (row_ok) {
              ml[slot * a.layout.rows + row] = make_float2(m_run, l_run);
#pragma unroll
              for (int c = 0; c < D / 8; ++c) st_global_v8(po + span_part(a, slot, c, row), &o[c / 4][c % 4 * 8]);
            }
            if (parts == 2) {
              __threadfence();
              __syncwarp();
              if (lane == 0) there = atomicAdd(arrived, 1);
              there = __shfl_sync(0xffffffffu, there, 0);
            }
          }
          if (!there) continue;
          __threadfence();
          if (row_ok) {
            const int64_t slot = mine_first ? 2 * (int64_t)(first + 1) : 2 * (int64_t)first + 1;  // the other's
            const float2 y = __ldcg(ml + slot * a.layout.rows + row);
            const float top = fmaxf(m_run, y.x), ref = top == -INFINITY ? 0.f : top;
            const float f = ex2_approx(m_run - ref), g = ex2_approx(y.x - ref);
            l_run = mine_first ? fmaf(y.y, g, l_run * f) : fmaf(l_run, f, y.y * g);
#pragma unroll
            for (int c = 0; c < D / 4; ++c) {
              const float4 z = __ldcg(reinterpret_cast<const float4*>(po + span_part(a, slot, c / 2, row)) + c % 2);
              const float zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = __uint_as_float(o[c / 8][c % 8 * 4 + e]);
                o[c / 8][c % 8 * 4 + e] = __float_as_uint(mine_first ? fmaf(zs[e], g, x * f) : fmaf(x, f, zs[e] * g));
              }
            }
          }
        }
        if (row_ok) {
          const float inv = 1.f / l_run;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) +
                               ((int64_t)(w.item.row0 + token) * a.h_q + w.head * a.group + r % a.group) * D;
          const bool out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              x[e] = pack_bf16x2(__uint_as_float(o[c][2 * e]) * inv, __uint_as_float(o[c][2 * e + 1]) * inv);
            if (out32) {
              st_global_v8(dst + c * 32, x);
              st_global_v8(dst + c * 32 + 16, x + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(dst + c * 32)[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
          }
        }
      }
      if (!ok && lane == 0) raise_timeout(p, bars);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarpA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
  }();
  return fn;
}

}  // namespace

bool span_tensor_map(CUtensorMap* m, const void* base, int elem, int rank, const cuuint64_t* dims, const cuuint32_t* box,
                     CUtensorMapSwizzle swizzle) {
  const EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t strides[2] = {dims[0] * elem, dims[0] * dims[1] * elem};
  const cuuint32_t ones[3] = {1, 1, 1};
  return fn(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base),
            dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

// bf16, boxes of 64 x box..., 128-byte swizzle
bool make_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims, const cuuint32_t* box) {
  return span_tensor_map(m, base, 2, rank, dims, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool Q8>
cudaError_t launch(const SpanArgs& a, cudaStream_t s) {
  TcArgs p;
  p.s = a;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.wait_budget = wait_budget_cycles();
  p.test_stall = test_stall_requested();
  CUtensorMap mq = {}, mk = {}, mv = {};
  const cuuint64_t q_dims[3] = {(cuuint64_t)D, (cuuint64_t)a.h_q, (cuuint64_t)a.T};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)a.group, (cuuint32_t)a.tile_tokens};
  bool ok = make_map(&mq, a.q, 3, q_dims, q_box);
  if (!Q8) {
    const cuuint64_t pool[2] = {(cuuint64_t)D, (cuuint64_t)a.n_blocks * a.h_kv * kPage};
    const cuuint64_t packed[2] = {(cuuint64_t)a.h_kv * D, (cuuint64_t)a.T};
    const cuuint32_t box[2] = {64, 128};
    ok = ok && make_map(&mk, a.table ? a.pool_k : a.k, 2, a.table ? pool : packed, box) &&
         make_map(&mv, a.table ? a.pool_v : a.v, 2, a.table ? pool : packed, box);
  }
  if (!ok) return cudaErrorInvalidValue;
  constexpr int smem = Smem<D, Q8>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(span_tc_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(span_tc_kernel<D, Q8>, dim3(a.ctas), dim3(kThreads), smem, s, mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_span_tc(const SpanArgs& a, cudaStream_t s) {
  if (a.pool_elem == 1) return a.d == 64 ? launch<64, true>(a, s) : launch<128, true>(a, s);
  return a.d == 64 ? launch<64, false>(a, s) : launch<128, false>(a, s);
}

}  // namespace kev
