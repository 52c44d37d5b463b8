// Eviction from a paged cache: which positions stay, and the move of their rows to the front.
//
// evict_check_kernel   every check of device data, before anything is written: CTA 0 looks at lengths and block tables
//                      (a bit map of the blocks in use: two questions on one block is the shared-state bug of the
//                      KV-cache isolation article, hnwysp.cn, §2.3 -- of the questions that are cut: the table row of one
//                      that is not may be stale, so a block that it shares with one that is cut is not found), all CTAs at
//                      the kept lists.  Each leaves a verdict of its own, and the kernel behind it takes the first error of
//                      them all.
//
// select_kernel        a CTA per (question, kv head).  The kept positions are the protected ones (the first and the last
//                      few) and of the others those of the `want` largest masses: the want-th largest value is found by
//                      radix, 11 bits of the ordered key at a time, from counts in shared memory; everything above it
//                      stays, and of the equal ones those of the lowest positions.  One more pass writes them in order:
//                      a warp takes a contiguous run of positions and knows from a scan over the warps where it writes.
//
// compact_kernel       row kept[j] to row j, j ascending, in place.  kept[j] >= j, so a row is overwritten only after
//                      the move that needs it in every order that reads a chunk of rows before it or any later chunk is
//                      written.  A chunk is 64 rows of one question and head, in K, V, the scales and the mass: a CTA
//                      takes the next chunk by a ticket (lower chunks of the same list have lower tickets, so they have
//                      begun), reads its rows into registers, says so, waits until every lower chunk of its list has
//                      been read, and writes.  Nobody waits before it has read, so the waits end; they are bounded all
//                      the same (a call that gave up has moved some chunks and not others).  Every row is read once and
//                      written once.
//
// Measured: 16 caches of 2 to 32 Ki positions cut to 4096 (8 kv heads of 128) selected in 31 us, most of it the largest
// list's: 32 Ki masses in 1024 threads, three counts of them; moved in 85 (bf16, 6.1 TB/s, 90 % of the measured copy rate
// with the checks; fp32 163).  32 caches of 200 to 2400 positions cut to 1024 selected in 13 us and moved, e4m3, in 21.
// Measured and left in the selection: four copies of the counts with 256 threads (17 us against 13), eight masses on their
// way (38 against 31).
#include "kev_internal.cuh"

namespace kev {
namespace {

constexpr int kCheckThreads = 512, kCheckRun = 4 * kCheckThreads;  // entries of a kept list that a CTA looks at at a time
constexpr int kCompactThreads = 256;

__device__ __forceinline__ int32_t* words_of(const EvictArgs& a) { return reinterpret_cast<int32_t*>(a.ws); }

// the first error of all verdicts (8 - rank each: 0 none, 3 kept, 5 slot, 6 overflow), by a whole CTA of >= 32 threads
__device__ __forceinline__ int verdict_of(const EvictArgs& a, int* shared) {
  if (threadIdx.x < 32) {
    int e = 0;
    for (int i = threadIdx.x; i < a.check_ctas; i += 32) e = max(e, words_of(a)[kEvictVerdicts + i]);
    e = __reduce_max_sync(0xffffffffu, e);
    if (threadIdx.x == 0) *shared = e;
  }
  __syncthreads();
  return *shared;
}
__device__ __forceinline__ int code_of(int e) { return e == 0 ? ST_OK : e == 6 ? ST_OVERFLOW : e == 5 ? ST_SLOT : ST_KEPT; }

__global__ void __launch_bounds__(kCheckThreads) evict_check_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ unsigned used[];  // CTA 0 of a compaction: a bit per block
  __shared__ int s_err;
  const int t = threadIdx.x, warp = t / 32, lane = t & 31;
  const bool compact = a.cells != 0;
  if (t == 0) s_err = 0;
  if (compact && blockIdx.x == 0)
    for (int i = t; i < (a.n_blocks + 31) / 32; i += kCheckThreads) used[i] = 0u;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto error = [&](int e) { atomicMax(&s_err, e); };
  auto takes_part = [&](int i) { return compact ? a.kept_lens_in[i] != a.lens[i] : !a.active || a.active[i]; };
  if (blockIdx.x == 0) {
    if (t == 0 && a.dev_status) *a.dev_status = ST_OK;  // the kernel behind reports what it finds
    for (int i = t; i < a.n; i += kCheckThreads) {
      if (!takes_part(i)) continue;
      const int n = a.lens[i];
      if (n < 0 || (int64_t)n > (int64_t)a.max_blocks * kPage) error(6);
    }
    __syncthreads();
    if (s_err == 0) {
      for (int i = warp; i < a.n; i += kCheckThreads / 32) {
        if (!takes_part(i)) continue;
        const int pages = (a.lens[i] + kPage - 1) / kPage;
        for (int e = lane; e < pages; e += 32) {
          const int b = a.table[(int64_t)i * a.max_blocks + e];
          if (b < 0 || b >= a.n_blocks) {
            error(5);
          } else if (compact) {
            const unsigned bit = 1u << (b & 31);
            if (atomicOr(&used[b >> 5], bit) & bit) error(5);
          }
        }
      }
    }
  }
  if (compact) {
    // kept lists: strictly ascending inside [0, lens[i])
    const int segments = (a.keep + kCheckRun - 1) / kCheckRun, units = a.n * a.h_kv * segments;
    for (int x = blockIdx.x; x < units; x += gridDim.x) {
      const int list = x / segments, j0 = x % segments * kCheckRun, i = list / a.h_kv;
      const int n = a.lens[i], m = a.kept_lens_in[i];
      if (n == m) continue;
      if (m < 0 || m > a.keep || m > n) {
        error(3);
        continue;
      }
      const int32_t* kept = a.kept_in + (int64_t)list * a.keep;
#pragma unroll
      for (int e = 0; e < kCheckRun / kCheckThreads; ++e) {
        const int j = j0 + e * kCheckThreads + t;
        if (j >= m) break;
        const int u = kept[j];
        if (u < 0 || u >= n || (j > 0 && kept[j - 1] >= u)) error(3);
      }
    }
    const int64_t step = (int64_t)gridDim.x * kCheckThreads;
    int32_t* flags = words_of(a) + a.flags;
    for (int64_t x = (int64_t)blockIdx.x * kCheckThreads + t; x < a.n_flags; x += step) flags[x] = 0;
    if (blockIdx.x == 0 && t < kEvictVerdicts) words_of(a)[t] = 0;  // ticket, abort
  }
  __syncthreads();
  if (t == 0) words_of(a)[kEvictVerdicts + blockIdx.x] = s_err;
}

// Whole numbers in the order of the floats; every NaN above all, -0 and 0 the same.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kWarps = kThreads / 32, kBins = 2048, kCopies = kThreads == 1024 ? 4 : 1;
  extern __shared__ uint32_t s_keys[];  // [a.smem_keys] ordered masses, as far as they fit
  __shared__ int s_bins[kCopies][kBins];  // lanes that differ mod kCopies count apart: masses share few exponents
  __shared__ int s_warp[kWarps][2];
  __shared__ int s_word[3];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  pdl_wait();
  pdl_trigger();
  const int err = verdict_of(a, s_word);
  const int i = blockIdx.x / a.h_kv, g = blockIdx.x % a.h_kv;
  if (blockIdx.x == 0 && t == 0 && a.dev_status && err) *a.dev_status = code_of(err);
  if (err || i >= a.n) return;
  const int n = a.lens[i];
  const bool live = !a.active || a.active[i];
  if (g == 0 && t == 0) a.kept_lens[i] = live ? min(n, a.keep) : n;
  if (!live) return;
  int32_t* out = a.kept + ((int64_t)i * a.h_kv + g) * a.keep;
  if (n <= a.keep) {
    for (int u = t; u < n; u += kThreads) out[u] = u;
    return;
  }
  const int32_t* row = a.table + (int64_t)i * a.max_blocks;
  const int lo = a.first, hi = n - a.last;       // the positions to choose from (lo <= hi: first + last <= keep < n)
  const int want = a.keep - a.first - a.last;    // and how many of them
  auto load = [&](int u) { return order_of(__ldg(a.mass + ((int64_t)__ldg(row + u / kPage) * a.h_kv + g) * kPage + u % kPage)); };
  for (int u = lo + t; u < hi && u < a.smem_keys; u += kThreads) s_keys[u] = load(u);
  auto key = [&](int u) { return u < a.smem_keys ? s_keys[u] : load(u); };

  // the want-th largest key v: digits of 11, 11 and 10 bits
  uint32_t v = 0, mask = 0;
  int left = want;  // still to be found among the keys that agree with v in the bits of the mask
  if (want > 0) {
#pragma unroll 1
    for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
      const int bins = shift == 0 ? 1024 : 2048;
      for (int b = t; b < kCopies * kBins; b += kThreads) s_bins[0][b] = 0;
      __syncthreads();
      for (int u = lo + t; u < hi; u += kThreads) {
        const uint32_t k = key(u);
        if ((k & mask) == v) atomicAdd(&s_bins[lane % kCopies][k >> shift & (bins - 1)], 1);
      }
      __syncthreads();
      // counts from the top: a thread has `per` neighbouring bins
      const int per = bins / kThreads;
      int mine = 0;
      for (int b = 0; b < per; ++b) {
        const int at = bins - 1 - (t * per + b);
        int n_at = 0;
#pragma unroll
        for (int x = 0; x < kCopies; ++x) n_at += s_bins[x][at];
        mine += s_bins[0][at] = n_at;
      }
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[warp][0] = incl;
      __syncthreads();
      int before = incl - mine;
      for (int w = 0; w < warp; ++w) before += s_warp[w][0];
      if (before < left && before + mine >= left) {  // one thread
        int at = before, b = 0;
        while (at + s_bins[0][bins - 1 - (t * per + b)] < left) at += s_bins[0][bins - 1 - (t * per + b++)];
        s_word[1] = bins - 1 - (t * per + b);
        s_word[2] = at;
      }
      __syncthreads();
      v |= (uint32_t)s_word[1] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      left -= s_word[2];
      __syncthreads();
    }
  }
  // v is the want-th largest, `left` of the keys equal to it stay.  Warp w writes those of positions [u0, u1).
  const int per = (n + kThreads - 1) / kThreads * 32;
  const int u0 = min(n, warp * per), u1 = min(n, u0 + per);
  auto kind = [&](int u) {  // 2 stays, 1 equal, 0 goes
    if (u < lo || u >= hi) return 2;
    if (want == 0) return 0;
    const uint32_t k = key(u);
    return k > v ? 2 : k == v ? 1 : 0;
  };
  __syncthreads();  // (the keys, where nothing was searched)
  int above = 0, equal = 0;
  for (int u = u0 + lane; u < u1; u += 32) {
    const int k = kind(u);
    above += k == 2;
    equal += k == 1;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    s_warp[warp][0] = above;
    s_warp[warp][1] = equal;
  }
  __syncthreads();
  above = equal = 0;
  for (int w = 0; w < warp; ++w) {
    above += s_warp[w][0];
    equal += s_warp[w][1];
  }
  for (int b = u0; b < u1; b += 32) {
    const int u = b + lane;
    const int k = u < u1 ? kind(u) : 0;
    const unsigned is2 = __ballot_sync(0xffffffffu, k == 2), is1 = __ballot_sync(0xffffffffu, k == 1), below = (1u << lane) - 1;
    const int a2 = above + __popc(is2 & below), a1 = equal + __popc(is1 & below);
    if (k == 2 || (k == 1 && a1 < left)) out[a2 + min(a1, left)] = u;
    above += __popc(is2);
    equal += __popc(is1);
  }
}

__device__ __forceinline__ int32_t ld_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// kRow: bytes of a cached row of one head
template <int kRow>
__global__ void __launch_bounds__(kCompactThreads) compact_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kVecs = kRow / 16;                                  // of a row
  constexpr int kMine = kEvictChunk * kVecs / kCompactThreads;      // of K, and of V, a thread moves
  constexpr int kRows = kCompactThreads / kVecs;                    // rows side by side
  static_assert(kMine >= 1, "a chunk fills the CTA");
  __shared__ int64_t s_src[kEvictChunk];  // cell of each row of the chunk, -1: it stays where it is
  __shared__ int s_word, s_moves, s_ticket;
  const int t = threadIdx.x;
  int32_t* words = words_of(a);
  int32_t* flags = words + a.flags;
  volatile int32_t* abort_word = words + kEvictAbort;
  pdl_wait();
  pdl_trigger();
  const int err = verdict_of(a, &s_word);
  if (blockIdx.x == 0 && t == 0 && a.dev_status && err) *a.dev_status = code_of(err);
  if (err) return;
  // true once *word is set; false when the call has given up
  auto wait = [&](const int32_t* word) {
    const long long began = clock64();
    while (ld_acquire(word) == 0) {
      if (*abort_word) return false;
      if (clock64() - began > a.wait_budget) {
        *abort_word = 1;
        if (a.dev_status) *a.dev_status = ST_TIMEOUT;
        return false;
      }
    }
    return true;
  };
  // test hook: the first chunk of a list does not say that it has been read, and those that wait for it give up
  auto says_so = [&](int c) { return c > 0 || !a.test_stall; };
  const int lists = a.n * a.h_kv, chunks = a.chunks;
  const int sub = t % kVecs, r0 = t / kVecs;
  for (;;) {
    __syncthreads();  // the last chunk's shared words are free
    if (t == 0) {
      s_ticket = atomicAdd(words + kEvictTicket, 1);
      s_moves = 0;
    }
    __syncthreads();
    const int64_t ticket = s_ticket;
    if (ticket >= (int64_t)lists * chunks) return;
    const int c = (int)(ticket / lists), list = (int)(ticket % lists), i = list / a.h_kv, g = list % a.h_kv;
    const int n = a.lens[i], m = a.kept_lens_in[i], j0 = c * kEvictChunk;
    if (n == m || j0 >= m) continue;
    const int32_t* row = a.table + (int64_t)i * a.max_blocks;
    float sk = 0.f, sv = 0.f, sm = 0.f;
    int64_t src = -1;
    if (t < kEvictChunk) {
      const int j = j0 + t;
      const int u = j < m ? a.kept_in[(int64_t)list * a.keep + j] : j;
      if (u != j) {
        src = ((int64_t)row[u / kPage] * a.h_kv + g) * kPage + u % kPage;
        s_moves = 1;
        if (a.scale_k) {
          sk = a.scale_k[src];
          sv = a.scale_v[src];
        }
        if (a.mass_io) sm = a.mass_io[src];
      }
      s_src[t] = src;
    }
    __syncthreads();
    int32_t* mine = flags + (int64_t)list * chunks;
    if (s_moves) {  // else the chunk stays as it is: all that is read there is in no chunk's way
      uint4 k[kMine], v[kMine];
#pragma unroll
      for (int e = 0; e < kMine; ++e) {
        const int64_t from = s_src[e * kRows + r0];
        if (from >= 0) {
          k[e] = static_cast<const uint4*>(a.k)[from * kVecs + sub];
          v[e] = static_cast<const uint4*>(a.v)[from * kVecs + sub];
        }
      }
      __threadfence();  // this thread's reads are done
      __syncthreads();
      if (t == 0 && says_so(c)) st_release(mine + c, 1);
      bool ok = true;
      for (int x = t; ok && x < c; x += kCompactThreads) ok = wait(mine + x);
      if (__syncthreads_or(!ok)) return;
      const int64_t to = ((int64_t)row[j0 / kPage] * a.h_kv + g) * kPage + j0 % kPage;
#pragma unroll
      for (int e = 0; e < kMine; ++e) {
        const int r = e * kRows + r0;
        if (s_src[r] >= 0) {
          static_cast<uint4*>(a.k)[(to + r) * kVecs + sub] = k[e];
          static_cast<uint4*>(a.v)[(to + r) * kVecs + sub] = v[e];
        }
      }
      if (src >= 0) {
        if (a.scale_k) {
          a.scale_k[to + t] = sk;
          a.scale_v[to + t] = sv;
        }
        if (a.mass_io) a.mass_io[to + t] = sm;
      }
    } else if (t == 0 && says_so(c)) {
      st_release(mine + c, 1);
    }
  }
}

// The check kernel: as many CTAs as the kept lists fill.
cudaError_t launch_check(EvictArgs& a, int num_sms, cudaStream_t s) {
  int64_t ctas = a.cells ? (int64_t)a.n * a.h_kv * ((a.keep + kCheckRun - 1) / kCheckRun) : 1;
  ctas = ctas < 1 ? 1 : ctas < 2 * num_sms ? ctas : 2 * num_sms;
  a.check_ctas = (int32_t)(ctas < kEvictCheckCtas ? ctas : kEvictCheckCtas);
  const size_t smem = a.cells ? ((size_t)a.n_blocks + 31) / 32 * 4 : 0;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(evict_check_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (1 << 20) / 8);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(evict_check_kernel, dim3(a.check_ctas), dim3(kCheckThreads), smem, s, a);
}

}  // namespace

cudaError_t launch_select(const EvictArgs& call, int num_sms, cudaStream_t s) {
  EvictArgs a = call;
  cudaError_t e = launch_check(a, num_sms, s);
  if (e != cudaSuccess) return e;
  const int64_t cap = (int64_t)a.max_blocks * kPage;
  constexpr int kMost = 48 * 1024;  // keys: 192 KB
  a.smem_keys = (int32_t)(cap < kMost ? cap : kMost);
  // The lists' lengths are known to the device only, so the table's width decides.  1024 threads are for long lists, and for
  // few: 32 lists of 16,000 positions (8 kv heads) take 39 us with them and 43 with 256, 4 of them 21 and 39.  They cost
  // short lists in a wide table: 32 of 8000 take 28 us and 26, of 2000 18 and 13.5, of 500 16 and 9.4.
  const bool wide = cap > 4096;
  auto kern = wide ? select_kernel<1024> : select_kernel<256>;
  const size_t smem = 4 * (size_t)a.smem_keys;
  if (smem > 12 * 1024) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMost);
    if (e != cudaSuccess) return e;
  }
  const int64_t units = (int64_t)a.n * a.h_kv;
  return launch_pdl(kern, dim3((unsigned)(units > 0 ? units : 1)), dim3(wide ? 1024 : 256), smem, s, a);
}

cudaError_t launch_compact(const EvictArgs& call, int num_sms, cudaStream_t s) {
  EvictArgs a = call;
  a.wait_budget = wait_budget_cycles();
  a.test_stall = test_stall_requested();
  const cudaError_t e = launch_check(a, num_sms, s);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.n * a.h_kv * a.chunks;
  const int64_t most = 8 * (int64_t)num_sms;
  const dim3 grid((unsigned)(units < 1 ? 1 : units < most ? units : most));
  auto kern = a.cells == 64 ? compact_kernel<64> : a.cells == 128 ? compact_kernel<128> : a.cells == 256 ? compact_kernel<256>
                                                                                                      : compact_kernel<512>;
  return launch_pdl(kern, grid, dim3(kCompactThreads), 0, s, a);
}

}  // namespace kev
