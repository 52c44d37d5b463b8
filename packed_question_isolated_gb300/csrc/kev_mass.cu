// Attention mass of fp32 q on the CUDA cores: true fp32 products and sums, cache fp32 or e4m3.  Bound by the multiply-adds
// and the shared-memory loads beside them: 8 chunks of 128 to 1024 tokens behind up to 8192 positions (28/4 heads) take 7.4
// ms, where the products, twice, are 1.9 at the CUDA cores' nominal 74 TFLOP/s (in bf16 on the tensor cores 0.21).  A decode
// step of 32 questions over 64 to 2400 positions (32/8 heads) takes 172 us (bf16 23): its row tiles of 64 hold the G rows of
// one question, so one warp of eight multiplies, and K is read by both passes.
//
// mass_rows_kernel   the rows' log sums: 64 (token, q-head) rows, 8 a warp, against 32 keys at a time; a lane owns a key
//                    and keeps a running maximum and sum of its own for each row, joined at the end.
// mass_join_kernel   rows whose key tiles were cut: the pieces' sums joined.
// mass_keys_kernel   the positions' sums: 128 keys, one per thread and half of the rows, against 32 rows at a time; the
//                    key's scores are the thread's own, so the sum over rows needs no exchange.
#include <cuda_fp8.h>

#include "kev_mass.cuh"

namespace kev {
namespace {

constexpr int kThreads = 256, kRows = 64, kSub = 32, kWarpRows = 8;
constexpr int kKeyRows = 32;  // rows at a time of the second pass

// 4 elements of a cached key
template <int D>
__device__ __forceinline__ float4 load_key(const SpanArgs& a, int64_t cell, int e) {
  if (a.pool_elem == 4) return *reinterpret_cast<const float4*>(static_cast<const float*>(a.pool_k) + cell * D + e);
  const uint32_t c = *reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(a.pool_k) + cell * D + e);
  const float s = a.scale_k[cell];
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"((uint16_t)(c >> (8 * j))));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&half2));
    f[j] = y.x * s;
    f[j + 1] = y.y * s;
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}
template <int D>
__device__ __forceinline__ float4 load_query(const SpanArgs& a, int64_t row, int e) {
  return *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + row * D + e);
}

__device__ __forceinline__ void join_sums(float& m, float& l, float m2, float l2) {
  const float top = fmaxf(m, m2);
  const float base = top == -INFINITY ? 0.f : top;
  l = l * exp2f(m - base) + l2 * exp2f(m2 - base);
  m = top;
}

template <int D>
struct RowsSmem {
  float q[kRows][D];
  float k[kSub][D + 4];  // padded: lanes read 32 different rows
};

template <int D>
__global__ void __launch_bounds__(kThreads) mass_rows_kernel(const __grid_constant__ MassArgs p) {
  extern __shared__ __align__(16) unsigned char raw[];
  RowsSmem<D>& sm = *reinterpret_cast<RowsSmem<D>*>(raw);
  const SpanArgs& a = p.s;
  pdl_wait();
  pdl_trigger();
  if (reinterpret_cast<const SpanHeader*>(a.ws)->status != ST_OK) return;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (blockIdx.x == 0 && t == 0) *reinterpret_cast<int32_t*>(a.ws + p.ticket) = 0;
  const float sl2 = a.scale * 1.4426950408889634f;
  float* lse = reinterpret_cast<float*>(a.ws + p.lse);
  for (SpanWalk walk(a, blockIdx.x); walk.live(); walk.next()) {
    const SpanItem& w = walk.item;
    const int head = walk.head, p0 = w.p0, p1 = p0 + w.tokens - 1, rows = w.tokens * a.group;
    const int32_t* table = a.table + (int64_t)w.question * a.max_blocks;
    __syncthreads();  // the shared tiles are free
    for (int x = t; x < kRows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), e = x % (D / 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) y = load_query<D>(a, (int64_t)(w.row0 + r / a.group) * a.h_q + head * a.group + r % a.group, e);
      *reinterpret_cast<float4*>(&sm.q[r][e]) = y;
    }
    float m[kWarpRows], l[kWarpRows];
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    for (int j = walk.j0; j < walk.j1; ++j)
      for (int s0 = 0; s0 < kSpanKeys; s0 += kSub) {
        const int u0 = j * kSpanKeys + s0;
        if (u0 > p1) break;
        const int64_t cell = ((int64_t)table[j] * a.h_kv + head) * kPage + s0;
        __syncthreads();
        for (int x = t; x < kSub * (D / 4); x += kThreads) {
          const int r = x / (D / 4), e = x % (D / 4) * 4;
          *reinterpret_cast<float4*>(&sm.k[r][e]) =
              u0 + r <= p1 ? load_key<D>(a, cell + r, e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        if (warp * kWarpRows >= rows) continue;
        float s[kWarpRows] = {};
#pragma unroll 4
        for (int e = 0; e < D; e += 4) {
          const float4 k = *reinterpret_cast<const float4*>(&sm.k[lane][e]);
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) {
            const float4 x = *reinterpret_cast<const float4*>(&sm.q[warp * kWarpRows + r][e]);
            s[r] = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, s[r]))));
          }
        }
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          if (u0 + lane > p0 + (warp * kWarpRows + r) / a.group) continue;
          const float z = s[r] * sl2;
          if (z > m[r]) {
            l[r] *= exp2f(m[r] - z);
            m[r] = z;
          }
          l[r] += m[r] == -INFINITY && z == z ? 0.f : exp2f(z - m[r]);
        }
      }
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1)
        join_sums(m[r], l[r], __shfl_xor_sync(0xffffffffu, m[r], x), __shfl_xor_sync(0xffffffffu, l[r], x));
      const int row = warp * kWarpRows + r;
      if (row >= rows || lane) continue;
      if (walk.whole())
        lse[(int64_t)(w.row0 + row / a.group) * a.h_q + head * a.group + row % a.group] = m[r] + log2f(l[r]);
      else
        reinterpret_cast<float2*>(a.ws + a.layout.part_ml)[walk.slot(blockIdx.x) * a.layout.rows + row] = make_float2(m[r], l[r]);
    }
  }
}

// Rows of the units that the plan lists: their pieces' sums joined, a thread per row.
__global__ void __launch_bounds__(256) mass_join_kernel(const __grid_constant__ MassArgs p) {
  const SpanArgs& a = p.s;
  pdl_wait();
  pdl_trigger();
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  if (h->status != ST_OK) return;
  const SpanCut* cuts = reinterpret_cast<const SpanCut*>(a.ws + a.line.cuts);
  const int32_t* joins = reinterpret_cast<const int32_t*>(a.ws + a.line.joins);
  const float2* ml = reinterpret_cast<const float2*>(a.ws + a.layout.part_ml);
  float* lse = reinterpret_cast<float*>(a.ws + p.lse);
  const int todo = h->n_joins * a.layout.rows;
  for (int x = blockIdx.x * 256 + threadIdx.x; x < todo; x += gridDim.x * 256) {
    const SpanCut& cut = cuts[joins[x / a.layout.rows]];
    const int row = x % a.layout.rows, rr = row % a.tile_rows, token = row / a.tile_rows * a.tile_tokens + rr / a.group;
    if (rr >= a.tile_tokens * a.group || token >= cut.record.tokens) continue;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < cut.parts; ++i) {  // slot 1 of the part the unit begins in, slot 0 of the later ones
      const float2 y = ml[(2 * (int64_t)(cut.first + i) + (i == 0)) * a.layout.rows + row];
      join_sums(m, l, y.x, y.y);
    }
    lse[(int64_t)(cut.record.row0 + token) * a.h_q + cut.head * a.group + rr % a.group] = m + log2f(l);
  }
}

template <int D>
struct KeysSmem {
  float k[kSpanKeys][D + 4];
  float q[kKeyRows][D];
  float lse[kKeyRows];
  float half[kSpanKeys];
};

template <int D>
__global__ void __launch_bounds__(kThreads) mass_keys_kernel(const __grid_constant__ MassArgs p) {
  extern __shared__ __align__(16) unsigned char raw[];
  KeysSmem<D>& sm = *reinterpret_cast<KeysSmem<D>*>(raw);
  int32_t* before = reinterpret_cast<int32_t*>(raw + sizeof(KeysSmem<D>));
  __shared__ int s_unit;
  const SpanArgs& a = p.s;
  pdl_wait();
  pdl_trigger();
  if (reinterpret_cast<const SpanHeader*>(a.ws)->status != ST_OK) return;
  mass_tiles_before(a, before);
  const int t = threadIdx.x, key = t % kSpanKeys, half = t / kSpanKeys;
  const float sl2 = a.scale * 1.4426950408889634f;
  const float* lse = reinterpret_cast<const float*>(a.ws + p.lse);
  const int64_t units = (int64_t)before[a.n] * a.h_kv;
  const int per = kKeyRows / a.group;  // tokens at a time
  for (;;) {
    __syncthreads();
    if (t == 0) s_unit = atomicAdd(reinterpret_cast<int32_t*>(a.ws + p.ticket), 1);
    __syncthreads();
    if (s_unit >= units) return;
    const int x = s_unit / a.h_kv, head = s_unit % a.h_kv, i = mass_question(before, a.n, x), j = x - before[i];
    const kev_interval iv = a.intervals[i];
    const int prefix = a.prefix[i], L = iv.end - iv.begin, u0 = j * kSpanKeys, u = u0 + key;
    const int64_t cell0 = ((int64_t)a.table[(int64_t)i * a.max_blocks + j] * a.h_kv + head) * kPage;
    const int size = prefix + L;  // cached positions
    for (int y = t; y < kSpanKeys * (D / 4); y += kThreads) {
      const int r = y / (D / 4), e = y % (D / 4) * 4;
      *reinterpret_cast<float4*>(&sm.k[r][e]) = u0 + r < size ? load_key<D>(a, cell0 + r, e) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float sum = 0.f;
    for (int t0 = max(0, u0 - prefix); t0 < L; t0 += per) {
      const int rows = min(per, L - t0) * a.group;
      __syncthreads();
      for (int y = t; y < kKeyRows * (D / 4); y += kThreads) {
        const int r = y / (D / 4), e = y % (D / 4) * 4;
        if (r < rows)
          *reinterpret_cast<float4*>(&sm.q[r][e]) =
              load_query<D>(a, (int64_t)(iv.begin + t0 + r / a.group) * a.h_q + head * a.group + r % a.group, e);
      }
      if (t < rows) sm.lse[t] = lse[(int64_t)(iv.begin + t0 + t / a.group) * a.h_q + head * a.group + t % a.group];
      __syncthreads();
      constexpr int kMine = kKeyRows / 2;
      float s[kMine] = {};
#pragma unroll 2
      for (int e = 0; e < D; e += 4) {
        const float4 k = *reinterpret_cast<const float4*>(&sm.k[key][e]);
#pragma unroll
        for (int r = 0; r < kMine; ++r) {
          const float4 y = *reinterpret_cast<const float4*>(&sm.q[half * kMine + r][e]);
          s[r] = fmaf(y.x, k.x, fmaf(y.y, k.y, fmaf(y.z, k.z, fmaf(y.w, k.w, s[r]))));
        }
      }
      float part = 0.f;
#pragma unroll
      for (int r = 0; r < kMine; ++r) {
        const int row = half * kMine + r;
        if (row < rows && u <= prefix + t0 + row / a.group) part += exp2f(s[r] * sl2 - sm.lse[row]);
      }
      sum += part;
    }
    if (half) sm.half[key] = sum;
    __syncthreads();
    if (!half && u < size) {
      sum += sm.half[key];
      float* to = p.mass + cell0 + key;
      *to = u < prefix && p.decay != 0.f ? fmaf(p.decay, *to, sum) : sum;
    }
  }
}

template <int D>
cudaError_t launch_simt(const MassArgs& m, int num_sms, cudaStream_t s) {
  const int rows_smem = sizeof(RowsSmem<D>), keys_smem = sizeof(KeysSmem<D>) + 4 * (m.s.n + 1);
  cudaError_t e = cudaFuncSetAttribute(mass_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, rows_smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(mass_keys_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(KeysSmem<D>) + 4 * (kMaxQuestions + 1));
  if (e == cudaSuccess) e = launch_pdl(mass_rows_kernel<D>, dim3(m.s.ctas), dim3(kThreads), rows_smem, s, m);
  if (e == cudaSuccess) e = launch_pdl(mass_join_kernel, dim3(num_sms), dim3(256), 0, s, m);
  if (e == cudaSuccess) e = launch_pdl(mass_keys_kernel<D>, dim3(2 * num_sms), dim3(kThreads), keys_smem, s, m);
  return e;
}

}  // namespace

cudaError_t launch_mass_simt(const MassArgs& m, int num_sms, cudaStream_t s) {
  return m.s.d == 64 ? launch_simt<64>(m, num_sms, s) : launch_simt<128>(m, num_sms, s);
}

}  // namespace kev
