/*
 * librq -- a cache held in 8 bits: appending (the position rotation on the way), and attention of
 * one or several new tokens over it, with or without a sliding window.
 *
 * The packed cache of rq.h needs a reference loop.  What has none -- the layers before and after
 * the looped block, a loop whose residual resists 2 or 4 bits -- keeps its keys and values here, at
 * 8 bits a value.  (An interface choice: the method's pages describe the packed cache only.)
 *
 * Conventions are those of rq.h: caller-owned device memory, all work on `stream` of the current
 * device, arguments checked before anything is enqueued, no allocation, no synchronisation.
 *
 * Layout (one layer; kv = 0 for K, 1 for V; d = head_dim).  Tiles of 64 slots, one record per
 * (sequence, kv-head, tile), [B][Hkv][capacity/64], or paged [n_pages][Hkv] (rq_paging):
 *   codes   bytes [record][n_loops][2][64][d]; row t of a tile keeps its 16-byte chunk c at chunk
 *           position c ^ (t & 7) (d = 128) or c ^ ((t >> 1) & 3) (d = 64): rows then lie in
 *           distinct shared-memory banks as they are copied
 *   scales  fp32 [record][n_loops][2][4]: one for every block of 16 slots, a power of two 2^e
 * A value is code * scale, a code e4m3 (RQ_Q8_E4M3) or a two's-complement integer in -127..127
 * (RQ_Q8_INT8).  e is the least exponent with amax <= M 2^e, M = 448 or 127, at least -100; amax is
 * the largest magnitude of the block's rows, rounded to bf16 (a code saturates at M).
 * A block that takes a row that is not finite gets the scale NaN: outputs of every new token that
 * sees any slot of the block are NaN, until the block is begun anew.
 */
#ifndef RQ_Q8_H_
#define RQ_Q8_H_

#include "rq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RQ_Q8_E4M3 = 0, RQ_Q8_INT8 = 1 } rq_q8_format;

typedef struct {
  int32_t batch;        /* B                                                            */
  int32_t n_q_heads;    /* Hq, a multiple of n_kv_heads (query head h reads kv-head      */
  int32_t n_kv_heads;   /*     h / (Hq / Hkv))                                           */
  int32_t head_dim;     /* d: 64 or 128                                                 */
  int32_t n_loops;      /* 1..16, each with keys and values of its own                  */
  int32_t capacity;     /* slots per sequence; a multiple of 64                         */
  int32_t format;       /* rq_q8_format                                                 */
  float softmax_scale;  /* 0 => 1/sqrt(d)                                               */
} rq_q8_shape;

typedef struct {
  uint8_t* codes;       /* 128-byte aligned                                             */
  float* scales;        /* 16-byte aligned                                              */
} rq_q8_cache;

/* Position rotation of the first rot_dim channels of a row at position p: the pair (x, y) of angle
 * a becomes (x cos a - y sin a, y cos a + x sin a) in fp32, products and sums rounded one by one.
 * Angle i turns channels (i, i + rot_dim/2), or (2i, 2i + 1) if interleaved. */
typedef struct {
  const float* table;         /* device fp32 [n_pos][rot_dim/2][2]: cos, sin; 16-byte aligned  */
  const int32_t* positions;   /* device int32 [B][n_new]: position of new token j; or NULL: its */
                              /* slot, ctx_lens[b] + j                                         */
  int32_t n_pos;              /* a position outside [0, n_pos) is never looked up: the row counts */
                              /* as not finite (append), the token's outputs are NaN (attention) */
  int32_t rot_dim;            /* a multiple of 16, at most d                                   */
  int32_t interleaved;        /* 0 or 1                                                        */
} rq_rope;

/* Bytes of the codes of one layer's cache: batch * n_kv_heads * capacity * n_loops * 2 * d (paged:
 * n_pages * 64 for batch * capacity), 0 for an invalid shape.  The scales take 1 / (4 d) of that as
 * fp32 numbers. */
size_t rq_q8_cache_bytes(const rq_q8_shape* shape);
size_t rq_q8_paged_cache_bytes(const rq_q8_shape* shape, int32_t n_pages);

/* Appends new tokens: token j of sequence b goes to slot ctx_lens[b] + j of loops loop_begin ..
 * + loop_count - 1, its K rotated if `rope` is given.
 *   kv_new     bf16, element (b, j, kv, l, h, i) at b*strides[0] + j*strides[1] + kv*strides[2] +
 *              l*strides[3] + h*strides[4] + i (elements, non-negative), l from loop_begin on
 *   n_lens     device int32 [B]: new tokens of each sequence, 0..n_new (a padded batch), or NULL
 *   n_new      >= 0 (0: nothing enqueued)
 *   ctx_lens   device int32 [B]: tokens cached before; not changed (rq_advance_ctx)
 *   rope       host struct, or NULL
 * Tokens at or behind the capacity are dropped; a sequence whose ctx_len is negative or whose n_len
 * lies outside 0..n_new, and a token whose block-table entry lies outside [0, n_pages), write
 * nothing.  Slots behind the last new token are left as they were.
 * A block of 16 slots that holds older rows keeps its scale if the new rows fit; else the scale
 * grows and the older rows' codes are divided by the same power of two, rounded to nearest even
 * (e4m3: exact but for the smallest codes).  Pages that take new tokens must belong to one sequence
 * only.  The same call repeated leaves the same bits. */
rq_status rq_q8_append(const rq_q8_shape* shape, const rq_q8_cache* cache, const uint16_t* kv_new,
                       const int64_t strides[5], int32_t loop_begin, int32_t loop_count,
                       const int32_t* n_lens, int32_t n_new, const int32_t* ctx_lens,
                       const rq_rope* rope, void* stream);
rq_status rq_paged_q8_append(const rq_q8_shape* shape, const rq_q8_cache* cache,
                             const rq_paging* paging, const uint16_t* kv_new,
                             const int64_t strides[5], int32_t loop_begin, int32_t loop_count,
                             const int32_t* n_lens, int32_t n_new, const int32_t* ctx_lens,
                             const rq_rope* rope, void* stream);

/* Attention of n_new tokens per sequence over one loop of the cache, which holds them already:
 * token j of sequence b is slot i = ctx_lens[b] + j and attends over the slots t <= i; with
 * window > 0 over those with t > i - window or t < n_sink.  n_new = 1 is the decode step.
 *   q          bf16, element (b, j, hq, i) at b*q_strides[0] + j*q_strides[1] + hq*q_strides[2] + i
 *              (elements, non-negative), rotated on the way if `rope` is given
 *   n_lens     device int32 [B]: new tokens of each sequence, 0..n_new, or NULL: n_new each
 *   n_new      >= 0 (0: nothing enqueued)
 *   ctx_lens   device int32 [B]: slots before the new tokens (as the append before was given)
 *   max_ctx    host upper bound of ctx_lens, 0..capacity
 *   window     0: every slot up to the token's own; n_sink >= 0, of no meaning without a window
 *   out        bf16 [B][n_new][Hq][d]; rows behind a sequence's last token are left as they were;
 *              it must not overlap q's span (RQ_ERR_INVALID_ARG)
 *   ws         256-byte aligned, at least rq_q8_workspace_bytes(...) bytes for the call's n_new, max_ctx,
 *              window and n_sink, or for a larger n_new or max_ctx.  Its first uint32 is the call's error
 *              word: nonzero after a ctx_len outside [0, max_ctx], an n_len outside [0, n_new] (taken
 *              as n_new), ctx_len + n_len beyond the capacity, a bad block-table entry of a tile that is
 *              seen, or a pipeline wait that gave up; outputs of the sequences (of a bad page: of the
 *              tokens that see it) concerned are NaN.  Calls that share a workspace must not overlap on
 *              the GPU.  Up to 32 rows a kv-head (n_new * Hq / Hkv) it takes some MB; from 33 on it holds
 *              fp16 operands, the queries' and twice the bytes of the loop's codes that are seen, for as many
 *              sequences at a time as 2 GB hold, for one at least (a million slots of 8 heads of 128: 4.3 GB)
 * Only tiles that some new token sees are read; block-table entries of others may be anything, so
 * pages that fell out of the window may be given away.
 * Sizes: n_new * (Hq / Hkv) <= 2^22, B * Hkv * ceil(n_new * (Hq / Hkv) / 32) * (capacity / 64 + 1) <= 2^40,
 * B * Hq * n_new <= 2^31 (RQ_ERR_UNSUPPORTED).
 * Precision: codes enter the products exactly; q . k, its product with softmax_scale, statistics and
 * accumulators are fp32.  A rotated query's element is rounded once to fp16 (2^-11 of itself); of any
 * query, elements below 2^-31 of their row's largest to 2^-39 of that, and rows below 2^-96 to 2^-135.  A
 * softmax weight times its block's V scale is rounded once to fp16: 2^-11 of itself, or 2^-24 of the largest
 * such product that the row sees.  What a row does not see takes no bits from it.  No atomics on results:
 * the same call gives the same bits. */
size_t rq_q8_workspace_bytes(const rq_q8_shape* shape, int32_t n_new, int32_t max_ctx,
                             int32_t window, int32_t n_sink);
rq_status rq_q8_attention(const rq_q8_shape* shape, const rq_q8_cache* cache, const uint16_t* q,
                          const int64_t q_strides[3], int32_t loop, const int32_t* n_lens,
                          int32_t n_new, const int32_t* ctx_lens, int32_t max_ctx, int32_t window,
                          int32_t n_sink, const rq_rope* rope, uint16_t* out, void* ws,
                          size_t ws_bytes, void* stream);
rq_status rq_paged_q8_attention(const rq_q8_shape* shape, const rq_q8_cache* cache,
                                const rq_paging* paging, const uint16_t* q,
                                const int64_t q_strides[3], int32_t loop, const int32_t* n_lens,
                                int32_t n_new, const int32_t* ctx_lens, int32_t max_ctx,
                                int32_t window, int32_t n_sink, const rq_rope* rope, uint16_t* out,
                                void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RQ_Q8_H_ */
