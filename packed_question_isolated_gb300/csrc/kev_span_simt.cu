// Span attention on the CUDA cores: fp32 q, k, v (true fp32 products, no TF32), cache fp32 or e4m3.
//
// out = softmax(scale q K^T + M) V over the visible positions, one pass: running maximum m and sum
// l of each row (log2 units), the accumulator rescaled when m moves, divided by l at the end.
//
// A CTA of 8 warps holds 64 rows -- floor(64 / G) tokens times the group's q-heads -- as 8 rows
// per warp, and walks its part of the work line in sub-tiles of 32 keys staged in shared memory as
// fp32.  Scores: a lane owns a key, so the row of K is its own and the 8 q values are broadcasts
// (32 multiply-adds per 9 vector loads); products with V: a lane owns 4 dims per 128, so V is a
// conflict-free vector load and P a broadcast (32 multiply-adds per 3).  Bound by the multiply-add
// rate and the shared-memory loads beside it: 8 prompts of 256 to 2048 tokens, 28 heads, under a window of
// 512 take 2.06 ms (20 TFLOP/s).
#include "kev_span.cuh"

namespace kev {
namespace {

constexpr int kThreads = 256, kRows = 64, kSub = 32, kWarpRows = 8;

template <int D> struct Smem {
  float q[kRows][D];
  float k[kSub][D + 4];  // padded: lanes read 32 different rows
  float v[kSub][D];
  float p[kThreads / 32][kSub][kWarpRows];
};

// 4 elements of row u of question i, kv head g
template <int D>
__device__ __forceinline__ float4 load4(const SpanArgs& a, bool is_v, int i, int begin, int g, int u, int e) {
  if (a.pool_elem == 0) {
    const int64_t at = ((int64_t)(begin + u) * a.h_kv + g) * D + e;
    return *reinterpret_cast<const float4*>(static_cast<const float*>(is_v ? a.v : a.k) + at);
  }
  const int64_t cell =
      ((int64_t)a.table[(int64_t)i * a.max_blocks + u / kPage] * a.h_kv + g) * kPage + u % kPage;
  if (a.pool_elem == 4)
    return *reinterpret_cast<const float4*>(static_cast<const float*>(is_v ? a.pool_v : a.pool_k) + cell * D + e);
  const uint32_t c = *reinterpret_cast<const uint32_t*>(static_cast<const unsigned char*>(is_v ? a.pool_v : a.pool_k) +
                                                        cell * D + e);
  const float s = (is_v ? a.scale_v : a.scale_k)[cell];
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // e4m3 placed in fp32: 4 exponent and 3 mantissa bits, times 2^120 for the difference of the
    // biases (exact, subnormals too); code 0x7f is the NaN
    const uint32_t b = (c >> (8 * j)) & 0xffu;
    const float x = __uint_as_float((b & 0x7fu) << 20 | (b & 0x80u) << 24) * 1.329227995784916e36f;
    f[j] = ((b & 0x7fu) == 0x7fu ? __uint_as_float(0x7fffffffu) : x) * s;
  }
  return make_float4(f[0], f[1], f[2], f[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2) span_simt_kernel(SpanArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  constexpr int kDims = D / 32;  // dims of a lane: D / 128 groups of 4, or 2 of 64
  constexpr int kV = D == 64 ? 2 : 4;
  pdl_wait();
  pdl_trigger();
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  if (h->status != ST_OK) return;
  span_zero_gaps(a, kThreads);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const float sl2 = a.scale * 1.4426950408889634f;

  for (SpanWalk walk(a, blockIdx.x); walk.live(); walk.next()) {
    const SpanItem& w = walk.item;
    const int head = walk.head, p0 = w.p0, p1 = p0 + w.tokens - 1;
    const SpanTiles tiles(p0, p1, a.window, a.sinks);
    const int rows = w.tokens * a.group;
    __syncthreads();  // the shared tiles are free
    for (int x = t; x < kRows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), e = x % (D / 4) * 4;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        y = *reinterpret_cast<const float4*>(
            static_cast<const float*>(a.q) +
            ((int64_t)(w.row0 + r / a.group) * a.h_q + head * a.group + r % a.group) * D + e);
      *reinterpret_cast<float4*>(&sm.q[r][e]) = y;
    }
    int pos[kWarpRows];
    float m[kWarpRows], l[kWarpRows], o[kWarpRows][kDims];
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      pos[r] = p0 + (warp * kWarpRows + r) / a.group;
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kDims; ++e) o[r][e] = 0.f;
    }
    for (int j = walk.j0; j < walk.j1; ++j)
      for (int s0 = 0; s0 < kSpanKeys; s0 += kSub) {
        const int u0 = tiles.at(j) * kSpanKeys + s0;
        if (u0 > p1) break;
        __syncthreads();
        for (int x = t; x < 2 * kSub * (D / 4); x += kThreads) {
          const bool is_v = x >= kSub * (D / 4);
          const int y = is_v ? x - kSub * (D / 4) : x;
          const int r = y / (D / 4), e = y % (D / 4) * 4;
          const float4 f = u0 + r <= p1 ? load4<D>(a, is_v, w.question, w.row0 - p0, head, u0 + r, e)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(is_v ? &sm.v[r][e] : &sm.k[r][e]) = f;
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
        unsigned seen = 0;  // bit r: this lane's key is visible to row r
#pragma unroll
        for (int r = 0; r < kWarpRows; ++r) {
          const bool v = span_sees(pos[r], u0 + lane, a.window, a.sinks);
          seen |= (unsigned)v << r;
          const float z = v ? s[r] * sl2 : -INFINITY;
          float top = z;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float mn = fmaxf(m[r], top);
          const float base = mn == -INFINITY ? 0.f : mn;  // nothing visible yet
          const float alpha = exp2f(m[r] - base);
          const float p = v ? exp2f(z - base) : 0.f;
          m[r] = mn;
          l[r] = l[r] * alpha + p;
#pragma unroll
          for (int e = 0; e < kDims; ++e) o[r][e] *= alpha;
          sm.p[warp][lane][r] = p;
        }
        // a masked key's V may hold anything: its product is left out, not multiplied by zero
        const bool edge = __any_sync(0xffffffffu, seen != (1u << kWarpRows) - 1);
        __syncwarp();
        auto product = [&](int u, unsigned vis) {
          const float4 pa = *reinterpret_cast<const float4*>(&sm.p[warp][u][0]);
          const float4 pb = *reinterpret_cast<const float4*>(&sm.p[warp][u][4]);
          const float p[kWarpRows] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
          float v[kDims];
#pragma unroll
          for (int e = 0; e < kDims; ++e) v[e] = sm.v[u][lane * kV + e];
#pragma unroll
          for (int r = 0; r < kWarpRows; ++r) {
            if (!(vis >> r & 1)) continue;
#pragma unroll
            for (int e = 0; e < kDims; ++e) o[r][e] = fmaf(p[r], v[e], o[r][e]);
          }
        };
        if (edge) {
#pragma unroll 1
          for (int u = 0; u < kSub; ++u) product(u, __shfl_sync(0xffffffffu, seen, u));
        } else {
#pragma unroll 4
          for (int u = 0; u < kSub; ++u) product(u, 0xffu);
        }
        __syncwarp();
      }
#pragma unroll
    for (int r = 0; r < kWarpRows; ++r) {
      float sum = l[r];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      const int row = warp * kWarpRows + r;
      if (row >= rows) continue;
      if (walk.whole()) {
        const float inv = 1.f / sum;
        const int64_t at =
            ((int64_t)(w.row0 + row / a.group) * a.h_q + head * a.group + row % a.group) * D + lane * kV;
#pragma unroll
        for (int e = 0; e < kDims; ++e) static_cast<float*>(a.out)[at + e] = o[r][e] * inv;
      } else {
        const int64_t slot = walk.slot(blockIdx.x);
        const int dim = lane * kV;
        float* dst = reinterpret_cast<float*>(a.ws + a.layout.part_o) + span_part(a, slot, dim / 8, row) + dim % 8;
        if (lane == 0) reinterpret_cast<float2*>(a.ws + a.layout.part_ml)[slot * a.layout.rows + row] = make_float2(m[r], sum);
#pragma unroll
        for (int e = 0; e < kDims; ++e) dst[e] = o[r][e];
      }
    }
  }
}

// Joins the pieces of the units that the plan lists: a thread per row and 8 dims, weights exp2(m_i - max m).
template <typename T, int D>
__global__ void __launch_bounds__(256) span_merge_kernel(SpanArgs a) {
  pdl_wait();
  pdl_trigger();
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  if (h->status != ST_OK) return;
  const SpanCut* cuts = reinterpret_cast<const SpanCut*>(a.ws + a.line.cuts);
  const int32_t* joins = reinterpret_cast<const int32_t*>(a.ws + a.line.joins);
  const float2* ml = reinterpret_cast<const float2*>(a.ws + a.layout.part_ml);
  const float* po = reinterpret_cast<const float*>(a.ws + a.layout.part_o);
  const int per = a.layout.rows * (D / 8);
  const int64_t todo = (int64_t)h->n_joins * per;
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < todo; x += (int64_t)gridDim.x * blockDim.x) {
    const SpanCut& cut = cuts[joins[x / per]];
    const int row = (int)(x % per) % a.layout.rows, c = (int)(x % per) / a.layout.rows;
    const int rr = row % a.tile_rows, token = row / a.tile_rows * a.tile_tokens + rr / a.group;
    if (rr >= a.tile_tokens * a.group || token >= cut.record.tokens) continue;
    // piece i: slot 1 of the part the unit begins in, slot 0 of the later ones
    auto slot = [&](int i) { return 2 * (int64_t)(cut.first + i) + (i == 0); };
    float top = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < cut.parts; ++i) top = fmaxf(top, ml[slot(i) * a.layout.rows + row].x);
    const float base = top == -INFINITY ? 0.f : top;
    float l = 0.f, o[8] = {};
#pragma unroll 4
    for (int i = 0; i < cut.parts; ++i) {
      const float2 p = ml[slot(i) * a.layout.rows + row];
      const float4* src = reinterpret_cast<const float4*>(po + span_part(a, slot(i), c, row));
      const float4 u = src[0], v = src[1];
      const float wgt = exp2f(p.x - base), y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      l = fmaf(p.y, wgt, l);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(y[e], wgt, o[e]);
    }
    const float inv = 1.f / l;
    T* dst = static_cast<T*>(a.out) +
             ((int64_t)(cut.record.row0 + token) * a.h_q + cut.head * a.group + rr % a.group) * D + c * 8;
    if (sizeof(T) == 2) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        y[e] = *reinterpret_cast<const uint32_t*>(&z);
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
      reinterpret_cast<float4*>(dst)[0] = make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
      reinterpret_cast<float4*>(dst)[1] = make_float4(o[4] * inv, o[5] * inv, o[6] * inv, o[7] * inv);
    }
  }
}

template <int D>
cudaError_t launch_simt(const SpanArgs& a, cudaStream_t s) {
  const int smem = sizeof(Smem<D>);
  const cudaError_t e = cudaFuncSetAttribute(span_simt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(span_simt_kernel<D>, dim3(a.ctas), dim3(kThreads), smem, s, a);
}

}  // namespace

cudaError_t launch_span_simt(const SpanArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_simt<64>(a, s) : launch_simt<128>(a, s);
}

cudaError_t launch_span_merge(const SpanArgs& a, int num_sms, cudaStream_t s) {
  auto kern = a.elem == 2 ? (a.d == 64 ? span_merge_kernel<__nv_bfloat16, 64> : span_merge_kernel<__nv_bfloat16, 128>)
                          : (a.d == 64 ? span_merge_kernel<float, 64> : span_merge_kernel<float, 128>);
  return launch_pdl(kern, dim3(4 * num_sms), dim3(256), 0, s, a);
}

}  // namespace kev
