// Writing new K/V rows into a paged cache in the cache's own type, and reading cached rows back.
//
// An e4m3 cache holds, for each position and kv head, the row x (d elements) as codes
// c_e = rn_e4m3(x_e / s) and one fp32 scale s = max_e |x_e| / 448 (448: the largest e4m3 value), so
// a row's largest element is stored exactly up to fp32 rounding and every other one within half
// an e4m3 step of its size (relative 2^-4, or 2^-10 s below the normal range; 448 times the rounding
// of s beside that, which counts where s is subnormal).  A row of zeros has s = 0 and codes 0; a row
// that holds a NaN or an infinity has a NaN for its scale and reads back as NaN throughout.  Reading
// gives c_e * s, rounded once to the output type.  Both quotients are the correctly rounded ones: the
// codes do not depend on the kernel's shape.
//
// Bound by memory: 2 T H_kv (d elem + d + 4) bytes each way for an e4m3 cache.  A warp takes one
// token's K and V rows of all kv heads: one search for the token's question (in shared memory) and
// one page look-up, then 16-byte loads with up to 8 in flight per lane (8 heads of 128 bf16: exactly
// 8).  Measured: 97k tokens of 8 heads read back in 102 us (5.9 TB/s, 87 % of the measured copy rate);
// 27k tokens written in 42.6 us (4.0 TB/s: neither fewer instructions nor more bytes in flight moved it; the
// writes land 128 bytes at a time, 16 KB apart).
#include <cuda_fp8.h>

#include "kev_span.cuh"

namespace kev {
namespace {

constexpr int kThreads = 256;
constexpr int kSmallThreads = 512, kSmall = 512;  // of the one kernel for small calls: threads, tokens and questions

// The prefix sums of the questions' lengths into shared memory, by the whole CTA.
__device__ __forceinline__ const int32_t* share_cu(const SpanArgs& a) {
  extern __shared__ int32_t s_cu[];
  const int32_t* cu = reinterpret_cast<const int32_t*>(a.ws + a.layout.cu);
  for (int i = threadIdx.x; i < a.n; i += kThreads) s_cu[i] = cu[i];
  __syncthreads();
  return s_cu;
}

// the question of new token x: the last i with cu[i] <= x (empty questions share their successor's value)
__device__ __forceinline__ int question_of(const int32_t* cu, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Place {
  int token;      // packed row
  int64_t block;  // pool block, row of it
  int row;
};
__device__ __forceinline__ Place place_of(const SpanArgs& a, const int32_t* cu, int x) {
  const int i = question_of(cu, a.n, x);
  const int j = x - cu[i];
  const int p = (a.prefix ? a.prefix[i] : 0) + j;
  return {a.intervals[i].begin + j, a.table[(int64_t)i * a.max_blocks + p / kPage], p % kPage};
}

// max |x| that keeps NaN
__device__ __forceinline__ float nan_max(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int E> struct Vec;  // 16 bytes of a row as floats
template <> struct Vec<4> {
  static constexpr int n = 4;
  static __device__ void get(uint4 w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
  static __device__ float top(uint4 w) {  // the largest magnitude, or NaN
    return nan_max(nan_max(fabsf(__uint_as_float(w.x)), fabsf(__uint_as_float(w.y))),
                   nan_max(fabsf(__uint_as_float(w.z)), fabsf(__uint_as_float(w.w))));
  }
  static __device__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};
template <> struct Vec<2> {
  static constexpr int n = 8;
  static __device__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ float top(uint4 w) {  // two elements at a time
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = max2(max2(w.x & kAbs, w.y & kAbs), max2(w.z & kAbs, w.w & kAbs));
    return nan_max(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ void get(uint4 w, float (&f)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ uint4 put(const float (&f)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// two e4m3 codes, the first in the low byte
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// A warp's copy of one token's rows of all kv heads into the cache: K and V, or with kOne (or `split`) only
// side `side` of them.
template <int E, int D, bool Q8, bool kOne>
__device__ __forceinline__ void write_token(const SpanArgs& a, const Place& at, bool split, int side) {
  using V = Vec<E>;
  constexpr int kLanes = D / V::n;       // lanes of a row: 8, 16 or 32
  constexpr int kRows = 32 / kLanes;     // rows a warp handles at once
  constexpr int kFlight = 4;             // of those in flight
  constexpr int kSides = kOne ? 1 : 2;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, r0 = lane / kLanes;
  // this lane's places at head r0: heads r0 + kRows e lie at fixed distances from them
  const int64_t from = ((int64_t)at.token * a.h_kv + r0) * kLanes + sub;
  const int64_t cell0 = (at.block * a.h_kv + r0) * kPage + at.row;
  for (int g0 = 0; g0 < a.h_kv; g0 += kRows * kFlight) {
    const int heads = a.h_kv - g0 - r0;  // e * kRows < heads: a head of this lane's
    uint4 w[kSides][kFlight];
#pragma unroll
    for (int i = 0; i < kSides; ++i) {
      const int v = kOne ? side : i;
      if (split && v != side) continue;
      const uint4* src = static_cast<const uint4*>(v ? a.v : a.k) + from + g0 * kLanes;
#pragma unroll
      for (int e = 0; e < kFlight; ++e)
        w[i][e] = e * kRows < heads ? src[e * kRows * kLanes] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < kSides; ++i) {
      const int v = kOne ? side : i;
      if (split && v != side) continue;
      const int64_t cell = cell0 + (int64_t)g0 * kPage;
      unsigned char* dst = static_cast<unsigned char*>(v ? a.pool_v : a.pool_k) + cell * (D * (Q8 ? 1 : E)) + sub * (Q8 ? V::n : 16);
      float* dst_scale = Q8 ? (v ? a.scale_v : a.scale_k) + cell : nullptr;
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        unsigned char* at_e = dst + e * kRows * kPage * D * (Q8 ? 1 : E);
        if (!Q8) {
          if (e * kRows < heads) *reinterpret_cast<uint4*>(at_e) = w[i][e];
        } else {
          float f[V::n], top = V::top(w[i][e]);
          V::get(w[i][e], f);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = nan_max(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float scale = span_scale(top);
          span_quotients(f, scale);
          uint32_t c[V::n / 4];
#pragma unroll
          for (int j = 0; j < V::n / 4; ++j) c[j] = e4m3x2(f[4 * j], f[4 * j + 1]) | e4m3x2(f[4 * j + 2], f[4 * j + 3]) << 16;
          if (e * kRows < heads) {
            if (V::n == 8) *reinterpret_cast<uint2*>(at_e) = make_uint2(c[0], c[V::n / 4 - 1]);
            else *reinterpret_cast<uint32_t*>(at_e) = c[0];
            if (sub == 0) dst_scale[e * kRows * kPage] = scale;
          }
        }
      }
    }
  }
}

// and back
template <int E, int D, bool Q8, bool kOne>
__device__ __forceinline__ void read_token(const SpanArgs& a, void* k_out, void* v_out, const Place& at, bool split, int side) {
  using V = Vec<E>;
  constexpr int kLanes = D / V::n, kRows = 32 / kLanes, kFlight = 4, kSides = kOne ? 1 : 2;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, r0 = lane / kLanes;
  const int64_t cell0 = at.block * a.h_kv * kPage + at.row;
  for (int g0 = 0; g0 < a.h_kv; g0 += kRows * kFlight) {
    uint4 w[kSides][kFlight];
    float s[kSides][kFlight];
#pragma unroll
    for (int i = 0; i < kSides; ++i)
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        const int v = kOne ? side : i;
        if (split && v != side) continue;
        const int g = g0 + e * kRows + r0;
        const int64_t cell = cell0 + (int64_t)g * kPage;
        if (g >= a.h_kv) continue;
        if (Q8) {
          const unsigned char* src = static_cast<const unsigned char*>(v ? a.pool_v : a.pool_k) + cell * D + sub * V::n;
          if (V::n == 8) {
            const uint2 c = *reinterpret_cast<const uint2*>(src);
            w[i][e] = make_uint4(c.x, c.y, 0u, 0u);
          } else {
            w[i][e].x = *reinterpret_cast<const uint32_t*>(src);
          }
          s[i][e] = (v ? a.scale_v : a.scale_k)[cell];
        } else {
          w[i][e] = static_cast<const uint4*>(v ? a.pool_v : a.pool_k)[cell * kLanes + sub];
        }
      }
#pragma unroll
    for (int i = 0; i < kSides; ++i)
#pragma unroll
      for (int e = 0; e < kFlight; ++e) {
        const int v = kOne ? side : i;
        if (split && v != side) continue;
        const int g = g0 + e * kRows + r0;
        if (g >= a.h_kv) continue;
        uint4* dst = static_cast<uint4*>(v ? v_out : k_out) + ((int64_t)at.token * a.h_kv + g) * kLanes + sub;
        if (Q8) {
          const uint32_t c[2] = {w[i][e].x, w[i][e].y};
          float f[V::n];
#pragma unroll
          for (int j = 0; j < V::n; j += 2) {
            uint32_t half2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"((uint16_t)(c[j / 4] >> (j % 4 * 8))));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&half2));
            f[j] = y.x * s[i][e];
            f[j + 1] = y.y * s[i][e];
          }
          *dst = V::put(f);
        } else {
          *dst = w[i][e];
        }
      }
  }
}

template <int E, int D, bool Q8, bool kRead>
__global__ void __launch_bounds__(kThreads) span_copy_kernel(SpanArgs a, void* k_out, void* v_out) {
  pdl_wait();
  pdl_trigger();
  const SpanHeader* h = reinterpret_cast<const SpanHeader*>(a.ws);
  if (h->status != ST_OK) return;
  const int32_t* cu = share_cu(a);
  const int warps = gridDim.x * (kThreads / 32);
  const int n_new = h->n_new;
  // few tokens: a warp for each of K and V
  const int split = 2 * (int64_t)n_new <= warps;
  int x = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int side = x & 1;
  if (split) x >>= 1;
  Place next = x < n_new ? place_of(a, cu, x) : Place{};
  for (; x < n_new; x += warps) {
    const Place at = next;  // looked up one token ahead
    if (x + warps < n_new) next = place_of(a, cu, x + warps);
    if (kRead) read_token<E, D, Q8, false>(a, k_out, v_out, at, split, side);
    else write_token<E, D, Q8, false>(a, at, split, side);
  }
}

// The checks of the plan (kev_span_plan.cu) and the copy in one kernel, for small calls: every CTA makes all
// the checks for itself, in shared memory, and comes to the same verdict, so none has to wait for another.
// Overlapping intervals show as a token that is marked twice; the mark is also the token's question.  A warp
// copies one token's K or V.  Measured on the GPU (the call takes the host 7.2 us) for one token of each of 32
// questions 3.6 us, with two kernels 7.0; at the ends of what it takes, a chunk of 512 tokens 4.9 against 7.3 and
// 512 questions of one token 9.0 against 15.6.
template <int E, int D, bool Q8, bool kRead>
__global__ void __launch_bounds__(kSmallThreads) span_small_copy_kernel(SpanArgs a, void* k_out, void* v_out) {
  extern __shared__ unsigned small_smem[];
  unsigned* used = small_smem;  // a bit per block
  const int words = (a.n_blocks + 31) / 32, t = threadIdx.x, warp = t / 32, lane = t & 31;
  __shared__ int2 s_iv[kSmall];
  __shared__ int s_prefix[kSmall], s_owner[kSmall], s_err;
  if (t == 0) s_err = 0;
  for (int i = t; i < words; i += kSmallThreads) used[i] = 0u;
  for (int i = t; i < a.T; i += kSmallThreads) s_owner[i] = -1;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto error = [&](int rank) { atomicMax(&s_err, 8 - rank); };  // ranks as in the plan
  for (int i = t; i < a.n; i += kSmallThreads) {
    const kev_interval v = a.intervals[i];
    const int first = a.prefix[i];
    s_iv[i] = make_int2(v.begin, v.end);
    s_prefix[i] = first;
    if (v.begin < 0 || v.end < v.begin || v.end > a.T) {
      error(0);
    } else if (v.end > v.begin) {
      if (first < 0) error(1);
      else if ((int64_t)first + (v.end - v.begin) > (int64_t)a.max_blocks * kPage) error(2);
    }
  }
  __syncthreads();
  const bool clean = s_err == 0, inside = s_err != 8;  // inside: every interval at least
  __syncthreads();
  if (clean) {
    for (int i = t; i < a.n; i += kSmallThreads) {  // pages; a block's bit may be set once
      const int L = s_iv[i].y - s_iv[i].x;
      if (L <= 0) continue;
      for (int e = s_prefix[i] / kPage; e <= (s_prefix[i] + L - 1) / kPage; ++e) {
        const int b = a.table[(int64_t)i * a.max_blocks + e];
        const unsigned bit = 1u << (b & 31);
        if (b < 0 || b >= a.n_blocks || atomicOr(&used[b >> 5], bit) & bit) error(3);
      }
    }
  }
  if (inside) {
    for (int i = warp; i < a.n; i += kSmallThreads / 32)
      for (int x = s_iv[i].x + lane; x < s_iv[i].y; x += 32)
        if (atomicExch(&s_owner[x], i) >= 0) error(0);
  }
  __syncthreads();
  if (blockIdx.x == 0 && t == 0 && a.dev_status) {
    const int rank = 8 - s_err;
    *a.dev_status = s_err == 0 ? ST_OK : rank == 0 ? ST_INTERVALS : rank == 1 ? ST_PREFIX : rank == 2 ? ST_OVERFLOW : ST_SLOT;
  }
  if (s_err) return;
  const int y = blockIdx.x * (kSmallThreads / 32) + warp, x = y >> 1;
  const int i = x < a.T ? s_owner[x] : -1;
  if (i < 0) return;
  const int p = s_prefix[i] + x - s_iv[i].x;
  const Place at = {x, a.table[(int64_t)i * a.max_blocks + p / kPage], p % kPage};
  if (kRead) read_token<E, D, Q8, true>(a, k_out, v_out, at, true, y & 1);
  else write_token<E, D, Q8, true>(a, at, true, y & 1);
}

int grid_of(const SpanArgs& a, int num_sms) {  // two warps per token, 8 CTAs of 8 warps per SM at most
  const int64_t ctas = (2 * (int64_t)a.T + kThreads / 32 - 1) / (kThreads / 32);
  return (int)(ctas < 8 * num_sms ? ctas : 8 * num_sms);
}

template <int E, int D, bool Q8, bool kRead>
cudaError_t launch(const SpanArgs& a, void* k_out, void* v_out, bool checked, int num_sms, cudaStream_t s) {
  if (checked) return launch_pdl(span_copy_kernel<E, D, Q8, kRead>, dim3(grid_of(a, num_sms)), dim3(kThreads),
                                 sizeof(int32_t) * (size_t)a.n, s, a, k_out, v_out);
  const int per = kSmallThreads / 64;  // tokens of a CTA; without any the checks are left
  return launch_pdl(span_small_copy_kernel<E, D, Q8, kRead>, dim3(a.T > 0 ? (a.T + per - 1) / per : 1), dim3(kSmallThreads),
                    sizeof(int32_t) * (((size_t)a.n_blocks + 31) / 32), s, a, k_out, v_out);
}
template <bool kRead>
cudaError_t launch_copy(const SpanArgs& a, void* k_out, void* v_out, bool checked, int num_sms, cudaStream_t s) {
  const bool q8 = a.pool_elem == 1;
  auto f = a.elem == 2 ? (a.d == 64 ? (q8 ? launch<2, 64, true, kRead> : launch<2, 64, false, kRead>)
                                    : (q8 ? launch<2, 128, true, kRead> : launch<2, 128, false, kRead>))
                       : (a.d == 64 ? (q8 ? launch<4, 64, true, kRead> : launch<4, 64, false, kRead>)
                                    : (q8 ? launch<4, 128, true, kRead> : launch<4, 128, false, kRead>));
  return f(a, k_out, v_out, checked, num_sms, s);
}

}  // namespace

// What the small kernel's shared memory holds without asking for more: 512 tokens and questions (every CTA
// checks them all) and 2^18 blocks.
bool span_small_copy(const SpanArgs& a) { return a.T <= kSmall && a.n <= kSmall && a.n_blocks <= 1 << 18; }

cudaError_t launch_span_write(const SpanArgs& a, bool checked, int num_sms, cudaStream_t s) {
  return a.T <= 0 && checked ? cudaSuccess : launch_copy<false>(a, nullptr, nullptr, checked, num_sms, s);
}

cudaError_t launch_span_read(const SpanArgs& a, void* k_out, void* v_out, bool checked, int num_sms, cudaStream_t s) {
  return a.T <= 0 && checked ? cudaSuccess : launch_copy<true>(a, k_out, v_out, checked, num_sms, s);
}

}  // namespace kev
