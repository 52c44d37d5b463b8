// Host side of the span operators of include/kev.h: argument checks and launches.
#include <math.h>

#include <atomic>

#include "kev_span.cuh"

using namespace kev;

namespace {

// kernel launches of the most recent successful call of each
std::atomic<int32_t> g_chunk_launches{2}, g_write_launches{2}, g_read_launches{2};

bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

kev_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KEV_OK : KEV_ERR_CUDA; }

int sms_of_current_device() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

kev_status check_span_shape(const kev_attn_shape* s) {
  if (!s || s->h_q <= 0 || s->h_kv <= 0) return KEV_ERR_INVALID_ARG;
  if (s->h_q % s->h_kv || s->h_q / s->h_kv > 16) return KEV_ERR_UNSUPPORTED;
  if (s->dtype != KEV_BF16 && s->dtype != KEV_FP32) return KEV_ERR_UNSUPPORTED;
  if (s->d_h != 64 && s->d_h != 128) return KEV_ERR_UNSUPPORTED;
  if (!(s->scale >= 0.f) || isinf(s->scale)) return KEV_ERR_INVALID_ARG;
  return KEV_OK;
}

// The arguments every span call shares, checked and laid out.
kev_status span_common(SpanArgs* a, int32_t T, const kev_interval* intervals, int32_t n, const kev_attn_shape* shape,
                       void* ws, size_t ws_bytes, int32_t* dev_status) {
  const kev_status st = check_span_shape(shape);
  if (st != KEV_OK) return st;
  if (T < 0 || n < 0) return KEV_ERR_INVALID_ARG;
  if (n > kMaxQuestions) return KEV_ERR_UNSUPPORTED;
  if (n > 0 && (!intervals || !aligned(intervals, 8))) return KEV_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || !aligned(dev_status, 4)) return KEV_ERR_INVALID_ARG;
  *a = SpanArgs{};
  a->intervals = intervals;
  a->n = n;
  a->T = T;
  a->h_q = shape->h_q;
  a->h_kv = shape->h_kv;
  a->group = shape->h_q / shape->h_kv;
  a->d = shape->d_h;
  a->elem = shape->dtype == KEV_BF16 ? 2 : 4;
  a->scale = shape->scale == 0.f ? 1.0f / sqrtf((float)shape->d_h) : shape->scale;
  a->max_chunk = T;
  a->ws = static_cast<char*>(ws);
  a->layout = span_layout(n, T, a->group, a->d);
  a->dev_status = dev_status;
  return ws_bytes < a->layout.total ? KEV_ERR_INVALID_ARG : KEV_OK;
}

kev_status span_cache(SpanArgs* a, const kev_attn_shape* shape, const int32_t* prefix_lens, const kev_paged_cache* c) {
  if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return KEV_ERR_INVALID_ARG;
  if (c->n_blocks <= 0 || c->max_blocks <= 0 || !c->block_table || !aligned(c->block_table, 4)) return KEV_ERR_INVALID_ARG;
  if (c->dtype != KEV_E4M3 && c->dtype != shape->dtype) return KEV_ERR_UNSUPPORTED;
  if (c->dtype == KEV_E4M3 && (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)))
    return KEV_ERR_INVALID_ARG;
  if (c->n_blocks > kSpanMaxBlocks || (int64_t)c->max_blocks * kPage > (1 << 30) ||
      (int64_t)c->n_blocks * a->h_kv * kPage > 0x7fffffffll)  // cached rows: coordinates of tensor copies
    return KEV_ERR_UNSUPPORTED;
  if (a->n > 0 && (!prefix_lens || !aligned(prefix_lens, 4))) return KEV_ERR_INVALID_ARG;
  a->prefix = prefix_lens;
  a->pool_k = c->k;
  a->pool_v = c->v;
  a->scale_k = c->k_scale;
  a->scale_v = c->v_scale;
  a->table = c->block_table;
  a->max_blocks = c->max_blocks;
  a->n_blocks = c->n_blocks;
  a->pool_elem = c->dtype == KEV_E4M3 ? 1 : c->dtype == KEV_BF16 ? 2 : 4;
  return KEV_OK;
}

// The launch of a kernel with row tiles of `rows` rows, `tiles` of them an item, on `ctas` CTAs.
SpanArgs span_line(const SpanArgs& call, int line, int rows, int tiles, int ctas) {
  SpanArgs a = call;
  a.line = call.layout.line[line];
  a.min_tokens = 1;
  a.max_tokens = call.max_chunk;
  a.tile_rows = rows;
  a.tile_tokens = rows / a.group;
  a.item_tiles = tiles;
  a.ctas = ctas < kSpanMaxCtas ? ctas : kSpanMaxCtas;
  return a;
}

// Every cached row meets at most 8 or 16 rows, which the register kernel takes at memory speed; it
// joins its own pieces.
SpanArgs span_few_rows(const SpanArgs& call, int line, int rows, int sms) {
  SpanArgs a = span_line(call, line, rows, 1, span_rows_ctas(call.d, rows) * sms);
  // Measured: e4m3 decode of 32 questions 29.2 us with 2, 32.1 with 1; bf16 pages at d = 128 take longer
  // each: 64 questions 44.7 us with 1, 46.3 with 2 (16 rows: 85.6 with 2, 90.1 with 1)
  a.unit_cost = call.pool_elem == 2 && call.d == 128 && rows == 8 ? 1 : 2;
  a.join_from = kSpanMaxCtas + 1;
  return a;
}

// Windows are at most 2^30 long (a longer one sees everything: positions end there), and sinks as many.
kev_status span_mask(SpanArgs* a, int32_t window, int32_t sinks) {
  if (window < 0 || sinks < 0) return KEV_ERR_INVALID_ARG;
  a->window = window > (1 << 30) ? 0 : window;
  a->sinks = sinks > (1 << 30) ? 1 << 30 : sinks;
  return KEV_OK;
}

// Do the T rows at out and those of `heads` heads at `in` share bytes?  (Units read q, k and v while others write out.)
bool overlap(const SpanArgs& a, const void* in, int heads) {
  const uint64_t row = (uint64_t)a.d * a.elem * a.T, o = (uint64_t)(uintptr_t)a.out, i = (uint64_t)(uintptr_t)in;
  return in && o < i + row * heads && i < o + row * a.h_q;
}
bool out_overlaps(const SpanArgs& a) { return overlap(a, a.q, a.h_q) || overlap(a, a.k, a.h_kv) || overlap(a, a.v, a.h_kv); }

// Launches the attention; *launches: how many kernels.
kev_status span_attend(const SpanArgs& call, bool write, int32_t* launches, cudaStream_t s) {
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  cudaError_t e;
  if (call.T <= 0) {  // no tokens (every question dropped): the checks alone; a tile of max_chunk = 0 rows holds no token
    *launches = 1;
    return from_cuda(launch_span_plan(call, 0, nullptr, nullptr, s));
  }
  *launches = 3 + write;
  if (call.elem == 4) {
    SpanArgs a = span_line(call, 0, 64, 1, 2 * sms);
    a.join_from = 2;
    e = launch_span_plan(call, 1, &a, nullptr, s);
    if (e == cudaSuccess && write) e = launch_span_write(a, true, sms, s);
    if (e == cudaSuccess) e = launch_span_simt(a, s);
    if (e == cudaSuccess) e = launch_span_merge(a, sms, s);
    return from_cuda(e);
  }
  const int64_t rows = (int64_t)call.max_chunk * call.group;
  if (call.pool_elem && rows <= 16) {  // few rows per question, and the caller said so
    const SpanArgs a = span_few_rows(call, 0, rows <= 8 ? 8 : 16, sms);
    *launches = 2;
    e = launch_span_plan(call, 1, &a, nullptr, s);
    if (e == cudaSuccess) e = launch_span_rows(a, write, s);
    return from_cuda(e);
  }
  SpanArgs a = span_line(call, 0, 128, 2, sms);
  // measured: a unit of two row tiles costs 1.8 us a key tile and 3.3 us beside them (loading q, the
  // masks of its first and last tiles, the epilogue)
  a.unit_cost = 2;
  a.join_from = 3;
  // Over an e4m3 cache, where an average question fills no row tile, most have one token or two: these go
  // to the kernel for few rows, the others to the tensor cores.  Measured on 4 chunks of 256 to 512 tokens
  // beside 60 single ones: 132 us, in one kernel 171 (the tensor-core kernel's conversion costs a page
  // as much for 4 rows as for 256); over a bf16 cache it is the other way round, 122 against 111.
  const bool split = call.pool_elem == 1 && (int64_t)call.T * call.group <= 128 * (int64_t)call.n;
  if (split) {
    ++*launches;
    SpanArgs b = span_few_rows(call, 1, call.group <= 8 ? 8 : 16, sms);
    b.max_tokens = b.tile_tokens;
    a.min_tokens = b.max_tokens + 1;
    e = launch_span_plan(call, 2, &a, &b, s);
    if (e == cudaSuccess && write) e = launch_span_write(call, true, sms, s);
    if (e == cudaSuccess) e = launch_span_rows(b, false, s);
  } else {
    e = launch_span_plan(call, 1, &a, nullptr, s);
    if (e == cudaSuccess && write) e = launch_span_write(call, true, sms, s);
  }
  if (e == cudaSuccess) e = launch_span_tc(a, s);
  if (e == cudaSuccess) e = launch_span_merge(a, sms, s);
  return from_cuda(e);
}

}  // namespace

int32_t kev::chunk_launches() { return g_chunk_launches.load(); }
int32_t kev::paged_write_launches() { return g_write_launches.load(); }
int32_t kev::paged_read_launches() { return g_read_launches.load(); }

extern "C" {

size_t kev_paged_workspace_size(int32_t n_questions, int32_t total_tokens, const kev_attn_shape* shape) {
  if (check_span_shape(shape) != KEV_OK || n_questions < 0 || n_questions > kMaxQuestions || total_tokens < 0) return 0;
  return span_layout(n_questions, total_tokens, shape->h_q / shape->h_kv, shape->d_h).total;
}

kev_status kev_paged_write(const void* k, const void* v, int32_t total_tokens, const kev_interval* intervals,
                           int32_t n_questions, const int32_t* prefix_lens, const kev_paged_cache* cache,
                           const kev_attn_shape* shape, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           kev_stream_t stream) {
  SpanArgs a;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st == KEV_OK) st = span_cache(&a, shape, prefix_lens, cache);
  if (st != KEV_OK) return st;
  if (total_tokens > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return KEV_ERR_INVALID_ARG;
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  a.k = k;
  a.v = v;
  const bool small = span_small_copy(a);
  cudaError_t e = small ? cudaSuccess : launch_span_plan(a, 0, nullptr, nullptr, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_span_write(a, !small, sms, (cudaStream_t)stream);
  if (e == cudaSuccess) g_write_launches = small ? 1 : 2;
  return from_cuda(e);
}

kev_status kev_paged_read(void* k, void* v, int32_t total_tokens, const kev_interval* intervals, int32_t n_questions,
                          const int32_t* prefix_lens, const kev_paged_cache* cache, const kev_attn_shape* shape,
                          void* workspace, size_t workspace_bytes, int32_t* dev_status, kev_stream_t stream) {
  SpanArgs a;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st == KEV_OK) st = span_cache(&a, shape, prefix_lens, cache);
  if (st != KEV_OK) return st;
  if (total_tokens > 0 && (!k || !v || !aligned(k, 16) || !aligned(v, 16))) return KEV_ERR_INVALID_ARG;
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  const bool small = span_small_copy(a);
  cudaError_t e = small ? cudaSuccess : launch_span_plan(a, 0, nullptr, nullptr, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_span_read(a, k, v, !small, sms, (cudaStream_t)stream);
  if (e == cudaSuccess) g_read_launches = small ? 1 : 2;
  return from_cuda(e);
}

kev_status kev_chunk_attn_paged(const void* q, const void* k, const void* v, int32_t total_tokens,
                                const kev_interval* intervals, int32_t n_questions, const int32_t* prefix_lens,
                                int32_t max_chunk, const kev_paged_cache* cache, int32_t window, int32_t sinks, void* out,
                                const kev_attn_shape* shape, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, kev_stream_t stream) {
  SpanArgs a;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st == KEV_OK) st = span_cache(&a, shape, prefix_lens, cache);
  if (st != KEV_OK) return st;
  if (max_chunk < 0) return KEV_ERR_INVALID_ARG;
  st = span_mask(&a, window, sinks);
  if (st != KEV_OK) return st;
  if ((k == nullptr) != (v == nullptr) || !aligned(k, 16) || !aligned(v, 16)) return KEV_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !out || !aligned(q, 16) || !aligned(out, 16))) return KEV_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  if (out_overlaps(a)) return KEV_ERR_INVALID_ARG;
  if (max_chunk > 0 && max_chunk < a.max_chunk) a.max_chunk = max_chunk;
  int32_t launches;
  st = span_attend(a, k != nullptr, &launches, (cudaStream_t)stream);
  if (st == KEV_OK) g_chunk_launches = launches;
  return st;
}

kev_status kev_prefill_attn_window(const void* q, const void* k, const void* v, int32_t total_tokens,
                                   const kev_interval* intervals, int32_t n_questions, int32_t window, int32_t sinks,
                                   void* out, const kev_attn_shape* shape, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_status, kev_stream_t stream) {
  SpanArgs a;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st != KEV_OK) return st;
  st = span_mask(&a, window, sinks);
  if (st != KEV_OK) return st;
  if (total_tokens > 0 && (!q || !k || !v || !out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)))
    return KEV_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.out = out;
  if (out_overlaps(a)) return KEV_ERR_INVALID_ARG;
  int32_t launches;
  return span_attend(a, false, &launches, (cudaStream_t)stream);
}

}  // extern "C"
