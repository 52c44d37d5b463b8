// Attention mass where a question brings few rows -- above all decode steps: bf16 q, at most 16 (token, q-head) rows per
// question and kv head, cache bf16 or e4m3.
//
// A cluster of up to 8 CTAs takes one question and kv head, each CTA a contiguous part of its pages:
//   1. scores S^T[16 keys x 8 rows] = K q^T by mma.sync m16n8k16, a warp 16 of a page's 128 positions.  The keys go from
//      global memory straight into the A operand's registers (the contraction index of an MMA may be permuted freely, so
//      a lane takes whole 16-byte chunks of a row), one page ahead.  The scores stay in shared memory;
//   2. every row's maximum over the CTA, weights exp2(S - max) in place of the scores, their sums;
//   3. maxima and sums of the cluster's CTAs by distributed shared memory: what each row's weights have to be multiplied
//      by; a position's mass is the sum over its rows.
// K is read once and nothing but the result is written.  Where a CTA's part has more positions than its shared memory has
// room for, those behind are read and computed twice: their sums with a running maximum in step 1, their weights in step 3.
//
// e4m3: the codes become fp16, exactly, one conversion per two; q becomes fp16 with a power of two of its own per row that
// brings its largest element to 2^14, so that what fp16 cannot hold is 2^-39 of it; the power and the key's scale multiply
// the score, the power in two halves, which keeps the product in range where one factor is tiny and the other large.
//
// Bound by memory over long caches: 16 bf16 caches of 2 to 32 Ki positions (32/8 heads) 91 us with the checks (5.0 TB/s, 73 %
// of the measured copy rate; DRAM bytes 1.00 of what has to be read, as long as the scores fit).  32 e4m3 caches of 64 to
// 2400 positions take 19, of which the checks are 4 to 5 and the rest is the chain of a cluster: pages, maxima, two cluster
// barriers.  Why clusters: scores written out for a second kernel cost a workspace as large as the caches, a second reading
// of K costs K again.  Measured and left: the longest caches first (97 us against 95).
#include <cuda_fp16.h>

#include "kev_mass.cuh"

namespace kev {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxRows = 16;
constexpr int kRoom = 100 * 1024;  // bytes of scores: two CTAs share an SM

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
__device__ __forceinline__ float ld_peer(const float* p, uint32_t rank) {
  const uint32_t local = static_cast<uint32_t>(__cvta_generic_to_shared(p));
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, bf16 (E = 2) or fp16 (E = 1) operands
template <int E>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (E == 2)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

struct MassRowsArgs {
  MassArgs m;
  int32_t rows;    // of a unit at most, even
  int32_t room;    // positions of scores in shared memory
};

struct Shared {
  float warp[kWarps][kMaxRows];
  float m[kMaxRows], l[kMaxRows];       // this CTA's, for the peers
  float factor[kMaxRows], lse[kMaxRows];
};

// 16 keys of a page in registers: chunks c, c + 4, ... of the rows of keys g and g + 8
template <int D, int E>
struct Keys {
  static constexpr int kChunks = D * E / 64;
  uint4 w[2][kChunks];
  float scale[2];
};

template <int D, int E, int NT>
__global__ void __launch_bounds__(kThreads, 2) mass_rows_kernel(const __grid_constant__ MassRowsArgs p) {
  extern __shared__ __align__(16) float s_scores[];  // [room][rows]
  __shared__ Shared sm;
  const SpanArgs& a = p.m.s;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, c = lane & 3;
  const int S = (int)cluster_size(), rank = (int)cluster_rank();
  pdl_wait();
  pdl_trigger();
  if (reinterpret_cast<const SpanHeader*>(a.ws)->status != ST_OK) return;
  const int unit = blockIdx.x / S, i = unit / a.h_kv, head = unit % a.h_kv;
  const kev_interval iv = a.intervals[i];
  const int L = iv.end - iv.begin;
  if (L <= 0) return;  // the whole cluster
  const int prefix = a.prefix[i], size = prefix + L, G = a.group, R = L * G, RS = p.rows;
  const int tiles = (size + kPage - 1) / kPage, per = (tiles + S - 1) / S;
  const int t0 = min(tiles, rank * per), t1 = min(tiles, t0 + per);
  const int32_t* table = a.table + (int64_t)i * a.max_blocks;
  const float sl2 = a.scale * 1.4426950408889634f;

  // q as the B operand: row 8 n + g, the chunks that this lane's keys have
  constexpr int kSteps = D / 16;
  uint32_t qf[NT][kSteps][2];
  float c1[NT][2], c2[NT][2];  // what the scores of rows 8 n + 2 c, + 1 are multiplied by
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = 8 * n + g;
    const bool live = r < R;
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) +
                               ((int64_t)(iv.begin + (live ? r / G : 0)) * a.h_q + head * G + (live ? r % G : 0)) * D;
    if constexpr (E == 2) {
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 w = live ? *reinterpret_cast<const uint4*>(row + 8 * (c + 4 * x)) : make_uint4(0u, 0u, 0u, 0u);
        qf[n][2 * x][0] = w.x;
        qf[n][2 * x][1] = w.y;
        qf[n][2 * x + 1][0] = w.z;
        qf[n][2 * x + 1][1] = w.w;
      }
      c1[n][0] = c1[n][1] = sl2;
      c2[n][0] = c2[n][1] = 1.f;
    } else {
      uint4 w[D / 64][2];
      float top = 0.f;
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          w[x][h] = live ? *reinterpret_cast<const uint4*>(row + 16 * (c + 4 * x) + 8 * h) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t u[4] = {w[x][h].x, w[x][h].y, w[x][h].z, w[x][h].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[e] << 16)), fabsf(__uint_as_float(u[e] & 0xffff0000u))));
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int k = top > 0.f && top < INFINITY ? 14 - ilogbf(top) : 0, k1 = k / 2, k2 = k - k1;
      const float f1 = pow2(k1), f2 = pow2(k2);
#pragma unroll
      for (int x = 0; x < D / 64; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u[4] = {w[x][h].x, w[x][h].y, w[x][h].z, w[x][h].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 y = __floats2half2_rn(__uint_as_float(u[e] << 16) * f1 * f2, __uint_as_float(u[e] & 0xffff0000u) * f1 * f2);
            qf[n][4 * x + 2 * h + e / 2][e % 2] = *reinterpret_cast<const uint32_t*>(&y);
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int from = (2 * c + e) * 4;
        c1[n][e] = sl2 * pow2(-__shfl_sync(0xffffffffu, k1, from));
        c2[n][e] = pow2(-__shfl_sync(0xffffffffu, k2, from));
      }
    }
  }

  auto load = [&](int tile, int block) {  // this warp's 16 keys
    Keys<D, E> k;
    const int64_t cell = ((int64_t)block * a.h_kv + head) * kPage + warp * 16 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4* row = reinterpret_cast<const uint4*>(static_cast<const char*>(a.pool_k) + (cell + 8 * h) * (D * E));
#pragma unroll
      for (int x = 0; x < Keys<D, E>::kChunks; ++x) k.w[h][x] = __ldcs(row + c + 4 * x);
      k.scale[h] = E == 1 ? __ldcs(a.scale_k + cell + 8 * h) : 1.f;
    }
    return k;
  };
  // z[n][2 h + e]: score of key g + 8 h and row 8 n + 2 c + e in log2 units, -infinity where the row does not see it
  auto scores = [&](const Keys<D, E>& k, int tile, float (&z)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) z[n][e] = 0.f;
#pragma unroll
    for (int x = 0; x < Keys<D, E>::kChunks; ++x) {
      const uint32_t u[2][4] = {{k.w[0][x].x, k.w[0][x].y, k.w[0][x].z, k.w[0][x].w}, {k.w[1][x].x, k.w[1][x].y, k.w[1][x].z, k.w[1][x].w}};
      if constexpr (E == 2) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma<2>(z[n], u[0][2 * s], u[1][2 * s], u[0][2 * s + 1], u[1][2 * s + 1], qf[n][2 * x + s][0], qf[n][2 * x + s][1]);
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t lo[2], hi[2];
          e4m3_to_f16(u[0][s], lo[0], hi[0]);
          e4m3_to_f16(u[1][s], lo[1], hi[1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma<1>(z[n], lo[0], lo[1], hi[0], hi[1], qf[n][4 * x + s][0], qf[n][4 * x + s][1]);
        }
      }
    }
    const int u0 = tile * kPage + warp * 16 + g;
    const bool edge = tile * kPage + warp * 16 + 15 > prefix;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        z[n][e] *= c1[n][e & 1];
        if (E == 1) z[n][e] = z[n][e] * k.scale[e >> 1] * c2[n][e & 1];
        if (edge && u0 + 8 * (e >> 1) > prefix + (8 * n + 2 * c + (e & 1)) / G) z[n][e] = -INFINITY;
      }
  };
  const int kept = min(t1, t0 + p.room / kPage);  // tiles whose scores stay

  // 1. scores
  float top[NT][2], run_m[NT][2], run_l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      top[n][e] = run_m[n][e] = -INFINITY;
      run_l[n][e] = 0.f;
    }
  auto inside = [&](int tile) { return tile < t1 && tile * kPage + warp * 16 < size; };
  Keys<D, E> next;
  if (inside(t0)) next = load(t0, table[t0]);
  int block = t0 + 1 < t1 ? table[t0 + 1] : 0;
#pragma unroll 1
  for (int tile = t0; inside(tile); ++tile) {
    const Keys<D, E> k = next;
    if (inside(tile + 1)) next = load(tile + 1, block);
    if (tile + 2 < t1) block = table[tile + 2];
    float z[NT][4];
    scores(k, tile, z);
    if (tile < kept) {
      float* to = s_scores + ((tile - t0) * kPage + warp * 16 + g) * RS;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (8 * n + 2 * c < RS) {
          *reinterpret_cast<float2*>(to + 8 * n + 2 * c) = make_float2(z[n][0], z[n][1]);
          *reinterpret_cast<float2*>(to + 8 * RS + 8 * n + 2 * c) = make_float2(z[n][2], z[n][3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) top[n][e] = fmaxf(top[n][e], fmaxf(z[n][e], z[n][2 + e]));
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m = fmaxf(run_m[n][e], fmaxf(z[n][e], z[n][2 + e])), base = m == -INFINITY ? 0.f : m;
          run_l[n][e] = run_l[n][e] * ex2(run_m[n][e] - base) + ex2(z[n][e] - base) + ex2(z[n][2 + e] - base);
          run_m[n][e] = m;
        }
    }
  }
  // the CTA's maximum of each row
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = fmaxf(top[n][e], run_m[n][e]);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (g == 0) sm.warp[warp][8 * n + 2 * c + e] = m;
    }
  __syncthreads();
  if (t < 8 * NT) {
    float m = sm.warp[0][t];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm.warp[w][t]);
    sm.m[t] = m;
  }
  __syncthreads();

  // 2. weights relative to it, and their sums
  const int here = max(0, min(size, kept * kPage) - t0 * kPage);  // positions in shared memory
  float sum[8 * NT];
#pragma unroll
  for (int r = 0; r < 8 * NT; ++r) sum[r] = 0.f;
  for (int x = t; x < here; x += kThreads) {
    float* at = s_scores + x * RS;
#pragma unroll
    for (int r = 0; r < 8 * NT; r += 2) {
      if (r >= RS) break;
      float2 y = *reinterpret_cast<float2*>(at + r);
      const float m0 = sm.m[r], m1 = sm.m[r + 1];
      y.x = ex2(y.x - (m0 == -INFINITY ? 0.f : m0));
      y.y = ex2(y.y - (m1 == -INFINITY ? 0.f : m1));
      *reinterpret_cast<float2*>(at + r) = y;
      sum[r] += y.x;
      sum[r + 1] += y.y;
    }
  }
  // (the positions with a running maximum: lanes of the same c hold the same rows)
  float over[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float m = sm.m[8 * n + 2 * c + e], base = m == -INFINITY ? 0.f : m;
      float l = run_l[n][e] == 0.f ? 0.f : run_l[n][e] * ex2(run_m[n][e] - base);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      over[n][e] = l;
    }
#pragma unroll
  for (int r = 0; r < 8 * NT; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
    if (lane == (r % 8) / 2) sm.warp[warp][r] = sum[r] + over[r / 8][r % 2];
  }
  __syncthreads();
  if (t < 8 * NT) {
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l += sm.warp[w][t];
    sm.l[t] = l;
  }

  // 3. the cluster's
  cluster_sync_all();
  if (t < 8 * NT) {
    float m = -INFINITY, l = 0.f;
    for (int x = 0; x < S; ++x) {
      const float m2 = ld_peer(&sm.m[t], x), l2 = ld_peer(&sm.l[t], x);
      const float top2 = fmaxf(m, m2), base = top2 == -INFINITY ? 0.f : top2;
      l = l * ex2(m - base) + l2 * ex2(m2 - base);
      m = top2;
    }
    const bool live = t < R;
    const float base = m == -INFINITY ? 0.f : m;
    sm.factor[t] = live ? ex2(sm.m[t] - base) / l : 0.f;
    sm.lse[t] = live ? base + log2f(l) : INFINITY;
  }
  cluster_sync_all();  // the peers keep their shared memory until all have read it
  auto put = [&](int u, int64_t cell, float w) {
    float* to = p.m.mass + cell;
    *to = u < prefix && p.m.decay != 0.f ? fmaf(p.m.decay, *to, w) : w;
  };
  // The first row that sees position u: a row without weights (NaN) does not reach what it does not see
  auto first_row = [&](int u) { return max(0, u - prefix) * G; };
  for (int x = t; x < here; x += kThreads) {
    const int u = t0 * kPage + x, first = first_row(u);
    const int64_t cell = ((int64_t)table[u / kPage] * a.h_kv + head) * kPage + u % kPage;
    float w = 0.f;
    const float* at = s_scores + x * RS;
#pragma unroll
    for (int r = 0; r < 8 * NT; ++r)
      if (r >= first && r < R) w = fmaf(at[r], sm.factor[r], w);
    put(u, cell, w);
  }
#pragma unroll 1
  for (int tile = kept; inside(tile); ++tile) {
    const int b = table[tile];
    const Keys<D, E> k = load(tile, b);
    float z[NT][4];
    scores(k, tile, z);
    float w[2] = {0.f, 0.f};
    const int u0 = tile * kPage + warp * 16 + g, first[2] = {first_row(u0), first_row(u0 + 8)};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 8 * n + 2 * c + (e & 1);
        w[e >> 1] += r >= first[e >> 1] && r < R ? ex2(z[n][e] - sm.lse[r]) : 0.f;
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] += __shfl_xor_sync(0xffffffffu, w[h], 1);
      w[h] += __shfl_xor_sync(0xffffffffu, w[h], 2);
      const int at = warp * 16 + g + 8 * h, u = tile * kPage + at;
      if (c == 0 && u < size) put(u, ((int64_t)b * a.h_kv + head) * kPage + at, w[h]);
    }
  }
}

template <int D, int E, int NT>
cudaError_t launch(const MassArgs& m, int num_sms, cudaStream_t s) {
  MassRowsArgs p = {};
  p.m = m;
  p.rows = (m.s.max_chunk * m.s.group + 1) / 2 * 2;
  // A part of 4 pages or more of the widest cache that the table has room for, for each CTA of a cluster (the lengths are
  // known to the device only).  16 bf16 caches of 2 to 32 Ki positions (8 kv heads) take 94 us in clusters of 8, 119 of 4,
  // 238 of 2, 403 of 1; 4 caches of 4000 positions 11.7, 12.4, 16.7 and 25.  It costs many short caches, whose CTAs have
  // few pages or none: 32 of 64 to 2400 positions take 25 us in the clusters of 4 that their own width of 19 pages asks
  // for, 44 in those of 8 that a table of 512 does, and would take 20 in clusters of 2.  One cache of 131,072 positions
  // has 8 CTAs per kv head and no more: 240 us with one kv head of 16 q-heads, 208 with 4 of 4, where the kernels for
  // chunks take 54 and 100.
  int S = 1;
  while (S < kMaxCluster && m.s.max_blocks >= 8 * S) S *= 2;
  const int64_t most = ((int64_t)(m.s.max_blocks + S - 1) / S) * kPage;
  const int64_t room = kRoom / (4 * p.rows) / kPage * kPage;
  p.room = (int32_t)(most < room ? most : room);
  const int smem = p.room * p.rows * 4;
  auto kern = mass_rows_kernel<D, E, NT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRoom);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(m.s.n * m.s.h_kv * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
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
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_mass_rows(const MassArgs& m, int num_sms, cudaStream_t s) {
  const bool two = m.s.max_chunk * m.s.group > 8, q8 = m.s.pool_elem == 1;
  auto f = m.s.d == 64 ? (q8 ? (two ? launch<64, 1, 2> : launch<64, 1, 1>) : (two ? launch<64, 2, 2> : launch<64, 2, 1>))
                       : (q8 ? (two ? launch<128, 1, 2> : launch<128, 1, 1>) : (two ? launch<128, 2, 2> : launch<128, 2, 1>));
  return f(m, num_sms, s);
}

}  // namespace kev
