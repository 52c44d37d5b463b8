// Host side that the span operators of include/kev.h and those beside them share: argument checks.
#pragma once

#include <math.h>

#include "kev_span.cuh"

namespace kev {

inline bool aligned(const void* p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

inline kev_status from_cuda(cudaError_t e) { return e == cudaSuccess ? KEV_OK : KEV_ERR_CUDA; }

inline int sms_of_current_device() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return sms;
}

inline kev_status check_span_shape(const kev_attn_shape* s) {
  if (!s || s->h_q <= 0 || s->h_kv <= 0) return KEV_ERR_INVALID_ARG;
  if (s->h_q % s->h_kv || s->h_q / s->h_kv > 16) return KEV_ERR_UNSUPPORTED;
  if (s->dtype != KEV_BF16 && s->dtype != KEV_FP32) return KEV_ERR_UNSUPPORTED;
  if (s->d_h != 64 && s->d_h != 128) return KEV_ERR_UNSUPPORTED;
  if (!(s->scale >= 0.f) || isinf(s->scale)) return KEV_ERR_INVALID_ARG;
  return KEV_OK;
}

// The arguments every span call shares, checked and laid out.
inline kev_status span_common(SpanArgs* a, int32_t T, const kev_interval* intervals, int32_t n, const kev_attn_shape* shape,
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

inline kev_status span_cache(SpanArgs* a, const kev_attn_shape* shape, const int32_t* prefix_lens, const kev_paged_cache* c) {
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
inline SpanArgs span_line(const SpanArgs& call, int line, int rows, int tiles, int ctas) {
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

}  // namespace kev
