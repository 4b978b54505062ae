// C ABI of the 8-bit cache (include/rq_q8.h): argument validation, then the launchers.
#include <cmath>

#include "rq_checks.h"
#include "rq_kernels.h"
#include "rq_q8.cuh"

namespace {

using rq::from_cuda;

rq_status check_shape(const rq_q8_shape* s) {
  if (!s) return RQ_ERR_INVALID_ARG;
  if (s->batch <= 0 || s->n_q_heads <= 0 || s->n_kv_heads <= 0 || s->capacity <= 0 || s->n_loops <= 0)
    return RQ_ERR_INVALID_ARG;
  if (s->n_q_heads % s->n_kv_heads != 0 || s->capacity % 64 != 0) return RQ_ERR_INVALID_ARG;
  if (s->head_dim != 64 && s->head_dim != 128) return RQ_ERR_UNSUPPORTED;
  if (s->format != RQ_Q8_E4M3 && s->format != RQ_Q8_INT8) return RQ_ERR_UNSUPPORTED;
  if (s->n_loops > RQ_MAX_LOOPS) return RQ_ERR_UNSUPPORTED;
  if (s->batch > 65535 || s->n_kv_heads > 65535 || s->capacity > (1 << 30)) return RQ_ERR_UNSUPPORTED;
  if (!(s->softmax_scale >= 0.f) || std::isinf(s->softmax_scale)) return RQ_ERR_INVALID_ARG;
  return RQ_OK;
}

rq_status check_cache(const rq_q8_shape* s, const rq_q8_cache* c, const rq_paging* pg, bool paged) {
  if (!c || !c->codes || !c->scales) return RQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->codes) & 127) != 0 || (reinterpret_cast<uintptr_t>(c->scales) & 15) != 0)
    return RQ_ERR_INVALID_ARG;
  if (!paged) return RQ_OK;
  if (!pg || !pg->block_table || pg->max_pages <= 0 || pg->n_pages <= 0) return RQ_ERR_INVALID_ARG;
  if (int64_t(s->capacity) != int64_t(64) * pg->max_pages) return RQ_ERR_INVALID_ARG;
  if (int64_t(pg->n_pages) * s->n_kv_heads * 64 > (int64_t(1) << 40)) return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

rq_status check_rope(const rq_q8_shape* s, const rq_rope* r, rq::Q8Rope& out) {
  out = {};
  if (!r) return RQ_OK;
  if (!r->table || (reinterpret_cast<uintptr_t>(r->table) & 15) != 0 || r->n_pos <= 0) return RQ_ERR_INVALID_ARG;
  if (r->rot_dim <= 0 || r->rot_dim > s->head_dim || (r->interleaved != 0 && r->interleaved != 1))
    return RQ_ERR_INVALID_ARG;
  if (r->rot_dim % 16 != 0) return RQ_ERR_UNSUPPORTED;
  out = {r->table, r->positions, r->n_pos, r->rot_dim, r->interleaved};
  return RQ_OK;
}

rq_status append_common(const rq_q8_shape* s, const rq_q8_cache* cache, const rq_paging* paging, bool paged,
                        const uint16_t* kv_new, const int64_t strides[5], int32_t loop_begin,
                        int32_t loop_count, const int32_t* n_lens, int32_t n_new, const int32_t* ctx_lens,
                        const rq_rope* rope, void* stream) {
  rq_status st = check_shape(s);
  if (st != RQ_OK) return st;
  if ((st = check_cache(s, cache, paging, paged)) != RQ_OK) return st;
  if (!strides || !ctx_lens || n_new < 0 || (n_new > 0 && !kv_new)) return RQ_ERR_INVALID_ARG;
  if (loop_begin < 0 || loop_count < 1 || loop_begin > s->n_loops - loop_count) return RQ_ERR_INVALID_ARG;
  const int64_t extents[5] = {s->batch, n_new, 2, loop_count, s->n_kv_heads};
  if (!rq::strides_ok(strides, extents, 5)) return RQ_ERR_INVALID_ARG;
  rq::Q8Rope r;
  if ((st = check_rope(s, rope, r)) != RQ_OK) return st;
  const int64_t blocks = (int64_t(n_new < s->capacity ? n_new : s->capacity) + 30) / 16;
  if (int64_t(s->batch) * s->n_kv_heads > ((int64_t(1) << 31) - 1) / (blocks * loop_count * 2)) return RQ_ERR_UNSUPPORTED;   // (grid.x)
  if (n_new == 0) return RQ_OK;
  try {
    return from_cuda(rq::launch_q8_append(*s, *cache, paging, kv_new, strides, loop_begin, loop_count,
                                          n_lens, n_new, ctx_lens, r, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return RQ_ERR_INTERNAL;
  }
}

rq_status check_sizes(const rq_q8_shape* s, int32_t n_new, int32_t max_ctx, int32_t window, int32_t n_sink) {
  if (n_new < 0 || max_ctx < 0 || max_ctx > s->capacity || window < 0 || n_sink < 0) return RQ_ERR_INVALID_ARG;
  const int64_t heads = s->n_q_heads / s->n_kv_heads, rows = heads * n_new;
  if (rows > (1 << 22)) return RQ_ERR_UNSUPPORTED;
  if (int64_t(s->batch) * s->n_kv_heads * ((rows + 31) / 32) > (int64_t(1) << 40) / (s->capacity / 64 + 1))
    return RQ_ERR_UNSUPPORTED;
  if (int64_t(s->batch) * s->n_q_heads * (n_new > 0 ? n_new : 1) > (int64_t(1) << 31)) return RQ_ERR_UNSUPPORTED;
  return RQ_OK;
}

rq_status attention_common(const rq_q8_shape* s, const rq_q8_cache* cache, const rq_paging* paging, bool paged,
                           const uint16_t* q, const int64_t q_strides[3], int32_t loop, const int32_t* n_lens,
                           int32_t n_new, const int32_t* ctx_lens, int32_t max_ctx, int32_t window,
                           int32_t n_sink, const rq_rope* rope, uint16_t* out, void* ws, size_t ws_bytes,
                           void* stream) {
  rq_status st = check_shape(s);
  if (st != RQ_OK) return st;
  if ((st = check_cache(s, cache, paging, paged)) != RQ_OK) return st;
  if (!q_strides || !ctx_lens || (n_new != 0 && (!q || !out))) return RQ_ERR_INVALID_ARG;
  if (loop < 0 || loop >= s->n_loops) return RQ_ERR_INVALID_ARG;
  if ((st = check_sizes(s, n_new, max_ctx, window, n_sink)) != RQ_OK) return st;
  const int64_t extents[3] = {s->batch, n_new, s->n_q_heads};
  if (!rq::strides_ok(q_strides, extents, 3)) return RQ_ERR_INVALID_ARG;
  const int32_t most = 1 << 30;                             // (as many slots as there can be)
  rq::Q8Call c = {q, {q_strides[0], q_strides[1], q_strides[2]}, loop, n_lens, n_new, ctx_lens, max_ctx,
                  window < most ? window : most, n_sink < most ? n_sink : most, {}, out};
  if ((st = check_rope(s, rope, c.rope)) != RQ_OK) return st;
  if (n_new == 0) return RQ_OK;
  if (!ws || ws_bytes < rq::q8_workspace_bytes(*s, n_new, max_ctx, window, n_sink)) return RQ_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return RQ_ERR_WORKSPACE;
  // rows are read while others are written
  const uintptr_t o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t o1 = o0 + size_t(s->batch) * n_new * s->n_q_heads * s->head_dim * 2;
  if (rq::overlaps(q, q_strides, extents, 3, s->head_dim, o0, o1)) return RQ_ERR_INVALID_ARG;
  try {
    return from_cuda(rq::launch_q8_attention(*s, *cache, paging, c, ws, static_cast<cudaStream_t>(stream)));
  } catch (...) {
    return RQ_ERR_INTERNAL;
  }
}

}  // namespace

extern "C" {

size_t rq_q8_cache_bytes(const rq_q8_shape* s) {
  if (check_shape(s) != RQ_OK) return 0;
  return size_t(s->batch) * s->n_kv_heads * size_t(s->capacity) * s->n_loops * 2 * s->head_dim;
}

size_t rq_q8_paged_cache_bytes(const rq_q8_shape* s, int32_t n_pages) {
  if (check_shape(s) != RQ_OK || n_pages <= 0) return 0;
  return size_t(n_pages) * s->n_kv_heads * 64 * s->n_loops * 2 * s->head_dim;
}

rq_status rq_q8_append(const rq_q8_shape* shape, const rq_q8_cache* cache, const uint16_t* kv_new,
                       const int64_t strides[5], int32_t loop_begin, int32_t loop_count,
                       const int32_t* n_lens, int32_t n_new, const int32_t* ctx_lens,
                       const rq_rope* rope, void* stream) {
  return append_common(shape, cache, nullptr, false, kv_new, strides, loop_begin, loop_count, n_lens, n_new,
                       ctx_lens, rope, stream);
}

rq_status rq_paged_q8_append(const rq_q8_shape* shape, const rq_q8_cache* cache,
                             const rq_paging* paging, const uint16_t* kv_new,
                             const int64_t strides[5], int32_t loop_begin, int32_t loop_count,
                             const int32_t* n_lens, int32_t n_new, const int32_t* ctx_lens,
                             const rq_rope* rope, void* stream) {
  return append_common(shape, cache, paging, true, kv_new, strides, loop_begin, loop_count, n_lens, n_new,
                       ctx_lens, rope, stream);
}

size_t rq_q8_workspace_bytes(const rq_q8_shape* s, int32_t n_new, int32_t max_ctx, int32_t window,
                             int32_t n_sink) {
  if (check_shape(s) != RQ_OK || check_sizes(s, n_new, max_ctx, window, n_sink) != RQ_OK) return 0;
  return n_new == 0 ? size_t(rq::kWsHeaderBytes) : rq::q8_workspace_bytes(*s, n_new, max_ctx, window, n_sink);
}

rq_status rq_q8_attention(const rq_q8_shape* shape, const rq_q8_cache* cache, const uint16_t* q,
                          const int64_t q_strides[3], int32_t loop, const int32_t* n_lens,
                          int32_t n_new, const int32_t* ctx_lens, int32_t max_ctx, int32_t window,
                          int32_t n_sink, const rq_rope* rope, uint16_t* out, void* ws,
                          size_t ws_bytes, void* stream) {
  return attention_common(shape, cache, nullptr, false, q, q_strides, loop, n_lens, n_new, ctx_lens, max_ctx,
                          window, n_sink, rope, out, ws, ws_bytes, stream);
}

rq_status rq_paged_q8_attention(const rq_q8_shape* shape, const rq_q8_cache* cache,
                                const rq_paging* paging, const uint16_t* q,
                                const int64_t q_strides[3], int32_t loop, const int32_t* n_lens,
                                int32_t n_new, const int32_t* ctx_lens, int32_t max_ctx,
                                int32_t window, int32_t n_sink, const rq_rope* rope, uint16_t* out,
                                void* ws, size_t ws_bytes, void* stream) {
  return attention_common(shape, cache, paging, true, q, q_strides, loop, n_lens, n_new, ctx_lens, max_ctx,
                          window, n_sink, rope, out, ws, ws_bytes, stream);
}

}  // extern "C"
