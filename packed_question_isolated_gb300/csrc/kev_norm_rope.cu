// Norms of the new tokens' query and key heads, the rotation to their positions, and the cache write, in one
// pass over the projection's rows.
//
// Per head row x of q or k: y = x / sqrt(mean_e x_e^2 + eps) * w (fp32 throughout), then the rotate-half form of
// kev_rope.cu at the token's position p: (a, b) = (y_j, y_{j + d/2}) becomes (a cos - b sin, b cos + a sin) with the
// table's cos and sin of p theta^(-2j/d).  Rounded once: to the type of q for q_out, k_out and a cache of that type;
// to e4m3 codes straight from fp32 (scale max |y| / 448 of the unrounded row) for an e4m3 cache, so that quantisation
// is a cached key's only rounding.  v rows go to the cache as kev_paged_write puts them.
//
// A position is not the cached row's index: a question whose cache had rows evicted counts on from the tokens that
// it has seen.  So the first position of each question's new tokens is an argument of its own.
//
// Bound by memory: every row is read once and written once.  A head row belongs to a group of 4 to 16 lanes; a lane holds
// 16 bytes of the row's first half and the 16 bytes that they pair with, so the rotation needs no exchange and the sum of
// squares 2 to 4 shuffles.  A warp takes a token's head rows (q, k, v in order), kSteps of them per group in flight; the
// token's cos and sin, the same for all of them, stay in registers.  Measured: the prompts of 32 questions (64 to 4096
// tokens, 32/8 heads of 128 in bf16, into a bf16 cache) 127 us with the checks, 122 without (5.6 TB/s, 83 % of the
// measured copy rate); into an e4m3 cache 141 (4.5 TB/s of its fewer bytes: scales and codes are arithmetic that bf16 rows
// do not have); in fp32 211, into an e4m3 cache 204; one token of each of 32 questions into an e4m3 cache 6.8 us on the
// GPU, a chain of dependent loads (intervals, table, angles) behind the checks, where the call takes the host 10.
#include <cuda_fp8.h>

#include "kev_span.cuh"

namespace kev {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // rows of a group of lanes in flight

// 16 bytes as floats and back
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
template <int E>
__device__ __forceinline__ uint4 pack(const float (&f)[16 / E]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (E == 2) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      u[i] = __float_as_uint(f[i]);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
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
// N quotients as codes
template <int N>
__device__ __forceinline__ void put_codes(unsigned char* to, const float (&f)[N]) {
  uint32_t c[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) c[j] = e4m3x2(f[4 * j], f[4 * j + 1]) | e4m3x2(f[4 * j + 2], f[4 * j + 3]) << 16;
  if constexpr (N == 8) *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
  else *reinterpret_cast<uint32_t*>(to) = c[0];
}

struct Place {
  int token, pos;  // packed row; position of the rotation
  int64_t block;   // pool block and row of it (no cache: 0)
  int row;
};

// The head rows [r0, r1) of one token (H_q of q, H_kv of k, with a cache H_kv of v) by a warp.
template <int E, int D, bool Q8>
__device__ __forceinline__ void norm_rope_rows(const NormRopeArgs& p, const Place& at, int r0, int r1) {
  constexpr int EV = 16 / E, kLanes = D / 2 / EV, kRows = 32 / kLanes;
  const SpanArgs& a = p.s;
  const int lane = threadIdx.x & 31, c = lane % kLanes, g = lane / kLanes;
  float2 cs[EV];
  const float4* table = reinterpret_cast<const float4*>(p.table + (int64_t)at.pos * (D / 2) + c * EV);
#pragma unroll
  for (int e = 0; e < EV; e += 2) {
    const float4 t = __ldg(table + e / 2);
    cs[e] = make_float2(t.x, t.y);
    cs[e + 1] = make_float2(t.z, t.w);
  }
  const int64_t cell0 = at.block * a.h_kv * kPage + at.row;  // head h of the kv heads: + h * kPage
#pragma unroll 1
  for (int first = r0; first < r1; first += kRows * kSteps) {
    uint4 wa[kSteps], wb[kSteps];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int r = first + s * kRows + g;
      wa[s] = wb[s] = make_uint4(0u, 0u, 0u, 0u);
      if (r < r1) {
        const char* base;
        int64_t stride;
        int h = r;
        if (r < a.h_q) {
          base = static_cast<const char*>(a.q);
          stride = p.q_stride;
        } else if (r < a.h_q + a.h_kv) {
          base = static_cast<const char*>(a.k);
          stride = p.k_stride;
          h -= a.h_q;
        } else {
          base = static_cast<const char*>(a.v);
          stride = p.v_stride;
          h -= a.h_q + a.h_kv;
        }
        const uint4* row = reinterpret_cast<const uint4*>(base + (at.token * stride + (int64_t)h * D) * E);
        wa[s] = row[c];
        wb[s] = row[kLanes + c];
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int r = first + s * kRows + g;
      if (first + s * kRows >= r1) break;
      const bool is_q = r < a.h_q, turn = r < a.h_q + a.h_kv;
      float x[EV], y[EV];
      unpack<E>(wa[s], x);
      unpack<E>(wb[s], y);
      if (first + s * kRows < a.h_q + a.h_kv) {  // some row of this step is one of q or k
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < EV; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const uint4* weight = static_cast<const uint4*>(is_q ? p.q_weight : p.k_weight);
        if (turn) {
          if (weight) {
            const float inv = rsqrtf(fmaf(sum, 1.f / D, p.eps));
            float u[EV], v[EV];
            unpack<E>(__ldg(weight + c), u);
            unpack<E>(__ldg(weight + kLanes + c), v);
#pragma unroll
            for (int e = 0; e < EV; ++e) {
              x[e] *= inv * u[e];
              y[e] *= inv * v[e];
            }
          }
#pragma unroll
          for (int e = 0; e < EV; ++e) {
            const float b = y[e];
            y[e] = fmaf(b, cs[e].x, x[e] * cs[e].y);
            x[e] = fmaf(x[e], cs[e].x, -(b * cs[e].y));
          }
        }
      }
      if (is_q) {
        uint4* to = static_cast<uint4*>(p.q_out) + ((int64_t)at.token * a.h_q + r) * (2 * kLanes);
        to[c] = pack<E>(x);
        to[kLanes + c] = pack<E>(y);
      }
      if (first + (s + 1) * kRows <= a.h_q) continue;  // every row of this step is one of q
      const bool is_k = !is_q && turn, live = !is_q && r < r1;
      const int h = r - a.h_q - (is_k ? 0 : a.h_kv);
      if (is_k && live && p.k_out) {
        uint4* to = static_cast<uint4*>(p.k_out) + ((int64_t)at.token * a.h_kv + h) * (2 * kLanes);
        to[c] = pack<E>(x);
        to[kLanes + c] = pack<E>(y);
      }
      if (a.pool_elem == 0) continue;
      const int64_t cell = cell0 + (int64_t)h * kPage;
      if (!Q8) {
        if (live) {
          uint4* to = static_cast<uint4*>(is_k ? a.pool_k : a.pool_v) + cell * (2 * kLanes);
          to[c] = is_k ? pack<E>(x) : wa[s];  // v: the bits as they are
          to[kLanes + c] = is_k ? pack<E>(y) : wb[s];
        }
      } else {
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < EV; ++e) top = nan_max(top, nan_max(fabsf(x[e]), fabsf(y[e])));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float scale = span_scale(top);
        span_quotients(x, scale);
        span_quotients(y, scale);
        if (live) {
          unsigned char* to = static_cast<unsigned char*>(is_k ? a.pool_k : a.pool_v) + cell * D + c * EV;
          put_codes(to, x);
          put_codes(to + D / 2, y);
          if (c == 0) (is_k ? a.scale_k : a.scale_v)[cell] = scale;
        }
      }
    }
  }
}

// Row steps of a token (kRows rows each) that a warp takes at a time
template <int E, int D>
constexpr int rows_of_part() { return 32 / (D / 2 / (16 / E)) * kSteps; }

__device__ __forceinline__ Place place_of(const NormRopeArgs& p, int i, int begin, int prefix, int j) {
  const SpanArgs& a = p.s;
  const int u = prefix + j;
  return {begin + j, (a.positions ? a.positions[i] : prefix) + j,
          a.pool_elem ? (int64_t)a.table[(int64_t)i * a.max_blocks + u / kPage] : 0, u % kPage};
}

// Behind the plan: warp w takes part w % parts of token w / parts, and goes on by the whole grid.
template <int E, int D, bool Q8>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeArgs p) {
  extern __shared__ int32_t s_cu[];
  const SpanArgs& a = p.s;
  pdl_wait();
  pdl_trigger();
  const SpanHeader* hdr = reinterpret_cast<const SpanHeader*>(a.ws);
  if (hdr->status != ST_OK) return;
  const int32_t* cu = reinterpret_cast<const int32_t*>(a.ws + a.layout.cu);
  for (int i = threadIdx.x; i < a.n; i += kThreads) s_cu[i] = cu[i];
  __syncthreads();
  const int rows = a.h_q + (a.pool_elem ? 2 : 1) * a.h_kv;
  const int n_new = hdr->n_new, warps = gridDim.x * (kThreads / 32);
  auto place = [&](int x) {
    int lo = 0, hi = a.n - 1;  // the last i with cu[i] <= x (empty questions share their successor's value)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cu[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    return place_of(p, lo, a.intervals[lo].begin, a.prefix ? a.prefix[lo] : 0, x - s_cu[lo]);
  };
  int x = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  Place next = x < n_new ? place(x) : Place{};
  for (; x < n_new; x += warps) {
    const Place at = next;  // looked up one token ahead
    if (x + warps < n_new) next = place(x + warps);
    norm_rope_rows<E, D, Q8>(p, at, 0, rows);
  }
}

// Small calls: checks and rows in one kernel; a warp takes kSteps rows a group of lanes of one token.
template <int E, int D, bool Q8>
__global__ void __launch_bounds__(kSpanSmall) norm_rope_small_kernel(const __grid_constant__ NormRopeArgs p) {
  extern __shared__ unsigned used[];  // a bit per block
  __shared__ SpanSmall sm;
  const SpanArgs& a = p.s;
  span_small_clear(a, sm, used);
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (!span_small_check(a, sm, used)) return;
  const int rows = a.h_q + (a.pool_elem ? 2 : 1) * a.h_kv;
  constexpr int kPart = rows_of_part<E, D>();
  const int parts = (rows + kPart - 1) / kPart;
  const int y = blockIdx.x * (kSpanSmall / 32) + threadIdx.x / 32, x = y / parts, part = y % parts;
  const int i = x < a.T ? sm.owner[x] : -1;
  if (i < 0) return;
  const Place at = place_of(p, i, sm.iv[i].x, sm.prefix[i], x - sm.iv[i].x);
  norm_rope_rows<E, D, Q8>(p, at, part * kPart, min(rows, (part + 1) * kPart));
}

template <int E, int D, bool Q8>
cudaError_t launch(const NormRopeArgs& p, bool checked, int num_sms, cudaStream_t s) {
  const SpanArgs& a = p.s;
  if (checked) {
    const int64_t ctas = ((int64_t)a.T + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(norm_rope_kernel<E, D, Q8>, dim3((unsigned)(ctas < 8 * num_sms ? ctas : 8 * num_sms)), dim3(kThreads),
                      sizeof(int32_t) * (size_t)a.n, s, p);
  }
  const int rows = a.h_q + (a.pool_elem ? 2 : 1) * a.h_kv, part = rows_of_part<E, D>();
  const int64_t warps = (int64_t)a.T * ((rows + part - 1) / part);
  const int64_t ctas = a.T > 0 ? (warps + kSpanSmall / 32 - 1) / (kSpanSmall / 32) : 1;  // without tokens the checks are left
  return launch_pdl(norm_rope_small_kernel<E, D, Q8>, dim3((unsigned)ctas), dim3(kSpanSmall),
                    a.pool_elem ? sizeof(int32_t) * (((size_t)a.n_blocks + 31) / 32) : 0, s, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& p, bool checked, int num_sms, cudaStream_t s) {
  if (checked && p.s.T <= 0) return cudaSuccess;
  const bool q8 = p.s.pool_elem == 1;
  auto f = p.s.elem == 2 ? (p.s.d == 64 ? (q8 ? launch<2, 64, true> : launch<2, 64, false>)
                                        : (q8 ? launch<2, 128, true> : launch<2, 128, false>))
                         : (p.s.d == 64 ? (q8 ? launch<4, 64, true> : launch<4, 64, false>)
                                        : (q8 ? launch<4, 128, true> : launch<4, 128, false>));
  return f(p, checked, num_sms, s);
}

}  // namespace kev
