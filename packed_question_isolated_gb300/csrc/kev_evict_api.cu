// Host side of the operators around the span attention: norms with rotation and cache write, attention mass, eviction.
#include <atomic>

#include "kev_mass.cuh"
#include "kev_span_host.cuh"

using namespace kev;

namespace {

// kernel launches of the most recent successful call of each
std::atomic<int32_t> g_norm_rope_launches{2}, g_mass_launches{4};

// Attention mass: the span workspace, and behind it the rows' log sums, a ticket and the second pass's parts.
size_t mass_layout(const SpanLayout& l, int32_t T, int32_t h_q, MassArgs* m) {
  m->lse = l.total;
  m->ticket = align_up(m->lse + sizeof(float) * (size_t)T * h_q, 256);
  m->cuts = m->ticket + 256;
  return m->cuts + align_up(mass_cuts_bytes(), 256);
}

kev_status mass_attend(const MassArgs& call, int32_t* launches, cudaStream_t s) {
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  if (call.s.T <= 0 || call.s.n <= 0) {  // no tokens, or none in a question: the checks alone
    *launches = 1;
    return from_cuda(launch_span_plan(call.s, 0, nullptr, nullptr, s));
  }
  MassArgs m = call;
  const bool bf16 = call.s.elem == 2;
  m.s = bf16 ? span_line(call.s, 0, 128, 2, sms) : span_line(call.s, 0, 64, 1, 2 * sms);
  m.s.unit_cost = bf16 ? 1 : 0;
  m.s.join_from = 2;
  // Few rows per question, and the caller said so; a grid has a cluster of up to 8 CTAs for every question and kv head.  Rows
  // that fill 16 gain least: 4 tokens (G = 4) of each of 32 caches of 64 to 2400 positions take 41 us, and 40 with the kernels
  // for chunks (e4m3 41 and 50), of each of 16 caches of 2 to 32 Ki 211 and 238 (181 and 324); one token of each 25 and 40 (26
  // and 50), 94 and 237 (79 and 327).
  const bool lists_fit = (int64_t)call.s.n * call.s.h_kv < 1 << 28;
  if (bf16 && lists_fit && (int64_t)call.s.max_chunk * call.s.group <= 16) {
    *launches = 2;
    cudaError_t e = launch_span_plan(call.s, 0, nullptr, nullptr, s, true);
    if (e == cudaSuccess) e = launch_mass_rows(m, sms, s);
    return from_cuda(e);
  }
  *launches = 4;
  cudaError_t e = launch_span_plan(call.s, 1, &m.s, nullptr, s);
  if (e == cudaSuccess) e = bf16 ? launch_mass_tc(m, sms, s) : launch_mass_simt(m, sms, s);
  return from_cuda(e);
}

// Eviction: the arguments of both calls, checked and laid out.
size_t evict_bytes(int32_t n, int32_t keep, int32_t h_kv) {
  const int64_t chunks = ((int64_t)keep + kEvictChunk - 1) / kEvictChunk;
  return align_up(4 * ((size_t)(kEvictVerdicts + kEvictCheckCtas) + (size_t)n * h_kv * chunks), 256);
}
// Positions end at 2^30 and cached rows at 2^31, so longer lists and more heads are of no use; tickets are counted in 32 bits
bool evict_sizes_fit(int32_t n, int32_t keep, int32_t h_kv) {
  return keep <= 1 << 30 && h_kv <= 1 << 24 && ((int64_t)keep + kEvictChunk - 1) / kEvictChunk * n * h_kv <= 1 << 30;
}
kev_status evict_common(EvictArgs* a, const int32_t* lens, int32_t n, const int32_t* table, int32_t max_blocks, int32_t n_blocks,
                        int32_t keep, const kev_attn_shape* shape, void* ws, size_t ws_bytes, int32_t* dev_status) {
  if (!shape || shape->h_kv <= 0) return KEV_ERR_INVALID_ARG;  // the rest of it: the move, whose rows it describes
  if (n < 0 || keep <= 0 || max_blocks <= 0 || n_blocks <= 0) return KEV_ERR_INVALID_ARG;
  if (n > kMaxQuestions || n_blocks > kSpanMaxBlocks || (int64_t)max_blocks * kPage > (1 << 30) ||
      (int64_t)n_blocks * shape->h_kv * kPage > 0x7fffffffll || !evict_sizes_fit(n, keep, shape->h_kv))
    return KEV_ERR_UNSUPPORTED;
  if (!table || !aligned(table, 4) || (n > 0 && (!lens || !aligned(lens, 4)))) return KEV_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256) || ws_bytes < evict_bytes(n, keep, shape->h_kv) || !aligned(dev_status, 4))
    return KEV_ERR_INVALID_ARG;
  *a = EvictArgs{};
  a->lens = lens;
  a->n = n;
  a->h_kv = shape->h_kv;
  a->table = table;
  a->max_blocks = max_blocks;
  a->n_blocks = n_blocks;
  a->keep = keep;
  a->chunks = (keep + kEvictChunk - 1) / kEvictChunk;
  a->flags = kEvictVerdicts + kEvictCheckCtas;
  a->n_flags = (int64_t)n * shape->h_kv * a->chunks;
  a->ws = static_cast<char*>(ws);
  a->dev_status = dev_status;
  return KEV_OK;
}

}  // namespace

int32_t kev::norm_rope_launches() { return g_norm_rope_launches.load(); }
int32_t kev::mass_launches() { return g_mass_launches.load(); }

extern "C" {

kev_status kev_norm_rope_paged(const void* q, const void* k, const void* v, int32_t q_stride, int32_t k_stride,
                               int32_t v_stride, void* q_out, void* k_out, int32_t total_tokens,
                               const kev_interval* intervals, int32_t n_questions, const int32_t* prefix_lens,
                               const int32_t* positions, const void* q_weight, const void* k_weight, float eps,
                               const void* rope_table, int32_t max_pos, const kev_paged_cache* cache,
                               const kev_attn_shape* shape, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                               kev_stream_t stream) {
  NormRopeArgs p = {};
  SpanArgs& a = p.s;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st != KEV_OK) return st;
  if (cache) {
    st = span_cache(&a, shape, prefix_lens, cache);
    if (st != KEV_OK) return st;
  } else {
    if (!aligned(prefix_lens, 4)) return KEV_ERR_INVALID_ARG;
    a.prefix = prefix_lens;
  }
  if (!aligned(positions, 4) || !rope_table || !aligned(rope_table, 16) || max_pos <= 0) return KEV_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16)) return KEV_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && !(eps > 0.f && !isinf(eps))) return KEV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)a.h_q * a.d, kv_row = (int64_t)a.h_kv * a.d;
  // a stride of 0: rows without anything between them
  p.q_stride = q_stride ? q_stride : q_row;
  p.k_stride = k_stride ? k_stride : kv_row;
  p.v_stride = v_stride ? v_stride : kv_row;
  if (p.q_stride < q_row || p.k_stride < kv_row || p.v_stride < kv_row) return KEV_ERR_INVALID_ARG;
  if ((p.q_stride * a.elem) % 16 || (p.k_stride * a.elem) % 16 || (p.v_stride * a.elem) % 16) return KEV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return KEV_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !k || !q_out || (cache ? !v : !k_out))) return KEV_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    // outputs over inputs: only q_out over q and k_out over k row for row, which their own threads read first
    const int64_t T = total_tokens;
    auto bytes = [&](int64_t stride, int64_t row) { return (uint64_t)(((T - 1) * stride + row) * a.elem); };
    auto meet = [](const void* x, uint64_t nx, const void* y, uint64_t ny) {
      const uint64_t i = (uint64_t)(uintptr_t)x, j = (uint64_t)(uintptr_t)y;
      return x && y && i < j + ny && j < i + nx;
    };
    const uint64_t nq = bytes(p.q_stride, q_row), nk = bytes(p.k_stride, kv_row), nv = bytes(p.v_stride, kv_row);
    const uint64_t mq = bytes(q_row, q_row), mk = bytes(kv_row, kv_row);
    const bool over_q = q_out == q && p.q_stride == q_row, over_k = k_out == k && p.k_stride == kv_row;
    if ((!over_q && meet(q_out, mq, q, nq)) || meet(q_out, mq, k, nk) || (cache && meet(q_out, mq, v, nv)) ||
        (!over_k && meet(k_out, mk, k, nk)) || meet(k_out, mk, q, nq) || (cache && meet(k_out, mk, v, nv)) ||
        meet(q_out, mq, k_out, mk))
      return KEV_ERR_INVALID_ARG;
  }
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.max_pos = max_pos;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.table = static_cast<const float2*>(rope_table);
  const bool small = span_small_copy(a);
  cudaError_t e = small ? cudaSuccess : launch_span_plan(a, 0, nullptr, nullptr, (cudaStream_t)stream);
  if (e == cudaSuccess) e = launch_norm_rope(p, !small, sms, (cudaStream_t)stream);
  if (e == cudaSuccess) g_norm_rope_launches = small ? 1 : 2;
  return from_cuda(e);
}

size_t kev_attn_mass_workspace_size(int32_t n_questions, int32_t total_tokens, const kev_attn_shape* shape) {
  if (check_span_shape(shape) != KEV_OK || n_questions < 0 || n_questions > kMaxQuestions || total_tokens < 0) return 0;
  MassArgs m;
  return mass_layout(span_layout(n_questions, total_tokens, shape->h_q / shape->h_kv, shape->d_h), total_tokens, shape->h_q, &m);
}

kev_status kev_attn_mass_paged(const void* q, int32_t total_tokens, const kev_interval* intervals, int32_t n_questions,
                               const int32_t* prefix_lens, int32_t max_chunk, const kev_paged_cache* cache, float decay,
                               float* mass, const kev_attn_shape* shape, void* workspace, size_t workspace_bytes,
                               int32_t* dev_status, kev_stream_t stream) {
  MassArgs m = {};
  SpanArgs& a = m.s;
  kev_status st = span_common(&a, total_tokens, intervals, n_questions, shape, workspace, workspace_bytes, dev_status);
  if (st == KEV_OK) st = span_cache(&a, shape, prefix_lens, cache);
  if (st != KEV_OK) return st;
  if (workspace_bytes < mass_layout(a.layout, total_tokens, a.h_q, &m)) return KEV_ERR_INVALID_ARG;
  if (max_chunk < 0 || !(decay >= 0.f) || isinf(decay) || !mass || !aligned(mass, 16)) return KEV_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!q || !aligned(q, 16))) return KEV_ERR_INVALID_ARG;
  a.q = q;
  if (max_chunk > 0 && max_chunk < a.max_chunk) a.max_chunk = max_chunk;
  m.mass = mass;
  m.decay = decay;
  int32_t launches;
  st = mass_attend(m, &launches, (cudaStream_t)stream);
  if (st == KEV_OK) g_mass_launches = launches;
  return st;
}

size_t kev_evict_workspace_size(int32_t n_questions, int32_t keep, const kev_attn_shape* shape) {
  if (!shape || shape->h_kv <= 0 || n_questions < 0 || n_questions > kMaxQuestions || keep <= 0 ||
      !evict_sizes_fit(n_questions, keep, shape->h_kv))
    return 0;
  return evict_bytes(n_questions, keep, shape->h_kv);
}

kev_status kev_select_paged(const float* mass, const int32_t* lens, const uint8_t* active, int32_t n_questions,
                            const int32_t* block_table, int32_t max_blocks, int32_t n_blocks, int32_t keep, int32_t first,
                            int32_t last, int32_t* kept, int32_t* kept_lens, const kev_attn_shape* shape, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, kev_stream_t stream) {
  EvictArgs a;
  const kev_status st = evict_common(&a, lens, n_questions, block_table, max_blocks, n_blocks, keep, shape, workspace,
                                     workspace_bytes, dev_status);
  if (st != KEV_OK) return st;
  if (first < 0 || last < 0 || (int64_t)first + last > keep || !mass || !aligned(mass, 16)) return KEV_ERR_INVALID_ARG;
  if (n_questions > 0 && (!kept || !aligned(kept, 4) || !kept_lens || !aligned(kept_lens, 4) || kept_lens == lens))
    return KEV_ERR_INVALID_ARG;
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  a.mass = mass;
  a.active = active;
  a.first = first;
  a.last = last;
  a.kept = kept;
  a.kept_lens = kept_lens;
  return from_cuda(launch_select(a, sms, (cudaStream_t)stream));
}

kev_status kev_compact_paged(const int32_t* kept, int32_t keep, const int32_t* lens, const int32_t* kept_lens,
                             int32_t n_questions, const kev_paged_cache* cache, float* mass, const kev_attn_shape* shape,
                             void* workspace, size_t workspace_bytes, int32_t* dev_status, kev_stream_t stream) {
  EvictArgs a;
  if (!cache) return KEV_ERR_INVALID_ARG;
  kev_status st = check_span_shape(shape);
  if (st == KEV_OK)
    st = evict_common(&a, lens, n_questions, cache->block_table, cache->max_blocks, cache->n_blocks, keep, shape, workspace,
                      workspace_bytes, dev_status);
  if (st != KEV_OK) return st;
  SpanArgs c = {};  // the cache's own checks
  c.h_kv = shape->h_kv;
  st = span_cache(&c, shape, nullptr, cache);
  if (st != KEV_OK) return st;
  if (!aligned(mass, 16)) return KEV_ERR_INVALID_ARG;
  if (n_questions > 0 && (!kept || !aligned(kept, 4) || !kept_lens || !aligned(kept_lens, 4))) return KEV_ERR_INVALID_ARG;
  const int sms = sms_of_current_device();
  if (sms <= 0) return KEV_ERR_CUDA;
  a.kept_in = kept;
  a.kept_lens_in = kept_lens;
  a.k = c.pool_k;
  a.v = c.pool_v;
  a.scale_k = c.pool_elem == 1 ? c.scale_k : nullptr;
  a.scale_v = c.pool_elem == 1 ? c.scale_v : nullptr;
  a.mass_io = mass;
  a.cells = shape->d_h * c.pool_elem;
  return from_cuda(launch_compact(a, sms, (cudaStream_t)stream));
}

}  // extern "C"
