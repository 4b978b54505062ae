// Chunk attention (rq_chunk_attention): host side, and the kernels of calls with few rows.
//
// A row is one (new token j, query head g) of a kv-head: row = j * heads + g.  Few rows take the
// decode kernel's chunk variants (rq_decode_mma.cuh): the cache is streamed once per block of 8
// rows, and the combine below merges the splits and adds the chunk's own tokens, causally.
#include "rq_common.cuh"
#include "rq_kernels.h"
#include "rq_launch.cuh"

namespace rq {
namespace {

constexpr float kStateMax = 65504.f;   // largest fp16: the states' range

struct TailArgs {
  const uint16_t* q;
  const uint16_t* kv_new;    // K rows of the call's loop; V rows at + kv_v
  int64_t qs0, qs1, qs2, ks0, ks1, kv_v, ks_h;
  const int32_t* n_lens;
  const int32_t* ctx_lens;
  const int8_t* vsigns;      // null: final loop (no residual part)
  const float* part;
  const unsigned* err;
  uint16_t* out;
  float* scores;             // [B][H][window * heads][score_stride], or null
  float* lse;                // [B][H][window * heads], log2 units
  float* weights;
  int64_t score_stride;
  int B, H, heads, n_new, n_splits, window, cap, max_ctx;
  int vec;                   // states, queries and outputs may be read and written 8 bytes at a time
  float scale_log2;
};

template <int P>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[P]) {
  if constexpr (P == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x, x[1] = v.y;
  }
}

// P consecutive bf16 values, two per word.
template <int P>
__device__ __forceinline__ void load_words(const uint16_t* p, bool vec, uint32_t (&w)[P / 2]) {
  if (vec) {
    if constexpr (P == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) w[i] = uint32_t(p[2 * i]) | uint32_t(p[2 * i + 1]) << 16;
  }
}

// One warp per row: merge the split partials, then the chunk's tokens 0..j, eight at a time (their
// loads and sums in flight together; online softmax), undo the rotation, store bf16.  Rows whose
// weights are asked for also store the chunk tokens' scores and their log2-sum-exp.  Bound by
// latency (2,048 rows of 7 splits and up to 8 tokens: 10 us; one token at a time 14).
template <int D>
__global__ void __launch_bounds__(128) chunk_combine_kernel(const __grid_constant__ TailArgs a) {
  grid_wait();
  grid_next();
  constexpr int P = D / 32;
  constexpr int rec = 4 + 2 * D;
  const int lane = threadIdx.x & 31;
  const int rows = a.n_new * a.heads;
  const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (wid >= int64_t(a.B) * a.H * rows) return;
  const int row = int(wid % rows), h = int(wid / rows % a.H), b = int(wid / rows / a.H);
  const int j = row / a.heads, g = row % a.heads;
  int n_len = a.n_lens ? a.n_lens[b] : a.n_new;
  bool bad = *a.err != 0u;
  if (n_len < 0 || n_len > a.n_new) {   // (the error word is set: every row of the sequence)
    n_len = a.n_new;
    bad = true;
  }
  if (j >= n_len) return;
  uint16_t* o = a.out + ((int64_t(b) * a.n_new + j) * a.H * a.heads + h * a.heads + g) * D + lane * P;
  const int first = max(0, n_len - a.window) * a.heads;
  const int64_t wrow = (int64_t(b) * a.H + h) * a.window * a.heads + row - first;
  const bool voted = a.scores && row >= first;
  float M = -INFINITY, ell = 0.f, ar[P], ae[P];
#pragma unroll
  for (int i = 0; i < P; ++i) ar[i] = ae[i] = 0.f;
  if (!bad) {
    // splits in groups of 32: a lane loads one split's (m, l), the warp their accumulators
    const float* part = a.part + wid * a.n_splits * rec;
    for (int s0 = 0; s0 < a.n_splits; s0 += 32) {
      const int ns = min(32, a.n_splits - s0);
      const float2 ml = lane < ns ? *reinterpret_cast<const float2*>(part + int64_t(s0 + lane) * rec)
                                  : make_float2(-INFINITY, 0.f);
      const float m = fmaxf(M, warp_max(ml.x)), f0 = M == -INFINITY ? 0.f : exp2f(M - m);
      const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
      ell = fmaf(ell, f0, warp_sum(f == 0.f ? 0.f : f * ml.y));
#pragma unroll
      for (int i = 0; i < P; ++i) {
        ar[i] *= f0;
        ae[i] *= f0;
      }
      M = m;
#pragma unroll 4
      for (int s = 0; s < ns; ++s) {
        const float fs = __shfl_sync(RQ_FULL_MASK, f, s);
        float x[P], y[P];
        const float* ps = part + int64_t(s0 + s) * rec + 4 + lane * P;
        load_floats<P>(ps, x);
        load_floats<P>(ps + D, y);
#pragma unroll
        for (int i = 0; i < P; ++i) {   // (an empty split's accumulators may hold anything)
          ar[i] = fs == 0.f ? ar[i] : fmaf(fs, x[i], ar[i]);
          ae[i] = fs == 0.f ? ae[i] : fmaf(fs, y[i], ae[i]);
        }
      }
    }
    float qv[P];
    uint32_t qw[P / 2];
    load_words<P>(a.q + b * a.qs0 + j * a.qs1 + (int64_t(h) * a.heads + g) * a.qs2 + lane * P, a.vec, qw);
#pragma unroll
    for (int i = 0; i < P; ++i) qv[i] = __uint_as_float(i & 1 ? qw[i / 2] & 0xffff0000u : qw[i / 2] << 16) * a.scale_log2;
    const uint16_t* const own = a.kv_new + b * a.ks0 + h * a.ks_h + lane * P;
    constexpr int U = 8;
    for (int t0 = 0; t0 <= j; t0 += U) {
      uint32_t k[U][P / 2], v[U][P / 2];
#pragma unroll
      for (int u = 0; u < U; ++u) {   // (behind the row's own token: that one again, weight 0)
        const uint16_t* const kp = own + int64_t(min(t0 + u, j)) * a.ks1;
        load_words<P>(kp, a.vec, k[u]);
        load_words<P>(kp + a.kv_v, a.vec, v[u]);
      }
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float x = __uint_as_float(i & 1 ? k[u][i / 2] & 0xffff0000u : k[u][i / 2] << 16);
          const float y = __uint_as_float(i & 1 ? v[u][i / 2] & 0xffff0000u : v[u][i / 2] << 16);
          bad |= !(fabsf(x) <= kStateMax) || !(fabsf(y) <= kStateMax);
          s[u] = fmaf(qv[i], x, s[u]);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(RQ_FULL_MASK, s[u], o);
      if (voted && lane == 0) {
        float* const to = a.scores + wrow * a.score_stride + a.ctx_lens[b] + t0;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (t0 + u <= j) to[u] = s[u];
      }
      float m = M;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = t0 + u <= j ? s[u] : -INFINITY;
        m = fmaxf(m, s[u]);
      }
      const float f0 = exp2f(M - m);   // (m is finite: the row's own token has a finite score)
      ell *= f0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        ar[i] *= f0;
        ae[i] *= f0;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = exp2f(s[u] - m);
        ell += f;
#pragma unroll
        for (int i = 0; i < P; ++i)
          ar[i] = fmaf(f, __uint_as_float(i & 1 ? v[u][i / 2] & 0xffff0000u : v[u][i / 2] << 16), ar[i]);
      }
      M = m;
    }
    bad = __any_sync(RQ_FULL_MASK, bad);
  }
  if (a.vsigns) {
    warp_fwht<P>(ae, lane);
    const float inv_sqrt_d = (D == 128) ? 0.08838834764831845f : 0.125f;
    const int8_t* sg = a.vsigns + int64_t(h) * D + lane * P;
#pragma unroll
    for (int i = 0; i < P; ++i) ar[i] = fmaf(ae[i] * inv_sqrt_d, float(sg[i]), ar[i]);
  }
  const float nan = __int_as_float(0x7fc00000);
  const float inv = bad ? nan : 1.f / ell;
  uint32_t w[P / 2];
#pragma unroll
  for (int i = 0; i < P / 2; ++i)
    w[i] = uint32_t(float_to_bf16_bits(ar[2 * i] * inv)) | uint32_t(float_to_bf16_bits(ar[2 * i + 1] * inv)) << 16;
  if (a.vec) {
    if constexpr (P == 4)
      *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(o) = w[0];
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
  if (voted && lane == 0) a.lse[wrow] = bad ? nan : M + log2f(ell);
}

// Four slots per thread: the weights of the window's rows, in row order.  A score per slot and row is
// read, a weight read and written; with one row bound by latency (256 x 4,097 slots: 12.6 MB in 6 us,
// launch included).
__global__ void __launch_bounds__(128) chunk_weights_kernel(const __grid_constant__ TailArgs a) {
  grid_wait();
  const int t0 = (blockIdx.x * 128 + threadIdx.x) * 4, h = blockIdx.y, b = blockIdx.z;
  const int n_len = a.n_lens ? a.n_lens[b] : a.n_new, ctx = a.ctx_lens[b];
  if (n_len < 0 || n_len > a.n_new || ctx < 0 || ctx > a.max_ctx) return;   // (flagged)
  const int end = min(ctx + n_len, a.cap);
  if (t0 >= end) return;
  const int first = max(0, n_len - a.window);
  const int64_t base = (int64_t(b) * a.H + h) * a.window * a.heads;
  const int n = (n_len - first) * a.heads;
  const float* const scores = a.scores + base * a.score_stride + t0;
  const float* const lse = a.lse + base;
  float* const out = a.weights + (int64_t(b) * a.H + h) * a.cap + t0;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  if (t0 + 4 <= ctx) {                // cached slots: every row
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
      const float4 s = *reinterpret_cast<const float4*>(scores + r * a.score_stride);
      const float z = lse[r];
      w[0] += exp2f(s.x - z);
      w[1] += exp2f(s.y - z);
      w[2] += exp2f(s.z - z);
      w[3] += exp2f(s.w - z);
    }
  } else {
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i;
      if (t >= end) break;
      const int from = t < ctx ? 0 : max(0, t - ctx - first) * a.heads;   // chunk token t - ctx: rows j >= it
      for (int r = from; r < n; ++r) w[i] += exp2f(scores[r * a.score_stride + i] - lse[r]);
    }
  }
  if (t0 + 4 <= end && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
    float4 v = *reinterpret_cast<const float4*>(out);
    v.x += w[0];
    v.y += w[1];
    v.z += w[2];
    v.w += w[3];
    *reinterpret_cast<float4*>(out) = v;
  } else {
    for (int i = 0; i < 4 && t0 + i < end; ++i) out[i] += w[i];
  }
}

// Workspace of a call with few rows: header, partial records, then (with weights) the scores and
// log2-sum-exps of the window's rows.
struct RowsLayout {
  SplitPlan plan;
  size_t part, scores, lse, total;
  int64_t score_stride;
};

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// The best plan within `budget`, else one split.
RowsLayout rows_layout(const rq_shape& s, int loop, int n_new, int max_ctx, int window, size_t budget) {
  RowsLayout l;
  const int heads = s.n_q_heads / s.n_kv_heads;
  l.plan = plan_splits_chunk(s, loop, heads * n_new, max_ctx);
  l.score_stride = (int64_t(max_ctx) + n_new + 31) / 32 * 32;
  const size_t units = size_t(s.batch) * s.n_kv_heads;
  const int tiles = max_ctx > 0 ? (max_ctx + kTile - 1) / kTile : 1;
  for (;;) {
    size_t o = kWsHeaderBytes;
    l.part = o;
    o = round256(o + units * heads * n_new * l.plan.n_splits * partial_floats(s) * sizeof(float));
    l.scores = o;
    o = round256(o + units * heads * window * size_t(l.score_stride) * sizeof(float));
    l.lse = o;
    o = round256(o + units * heads * window * sizeof(float));
    l.total = o;
    if (o <= budget || l.plan.n_splits == 1) return l;
    const int per = (tiles + l.plan.n_splits - 2) / (l.plan.n_splits - 1);
    l.plan.tokens_per_split = per * kTile;
    l.plan.n_splits = (tiles + per - 1) / per;
  }
}

}  // namespace

// How a call runs (times in us, 2-bit loop, 128 channels, L2 flushed; B x Hkv after ctx):
// - kStream: the cache once per 8 rows.  Up to 8 rows (8 x 8 after 16384: 112 us against 130 fused;
//   16 rows 206 against 132).  With weights up to 32 rows, because its scores carry 21 bits and tiles
//   need a second pass for that (32 rows 448 us against 728; 64 rows 857 against 729).
// - kFused: up to 128 rows without weights, the codes converted in shared memory once for all rows
//   (32 rows 136 us, 128 rows 185 us against 390 with tiles).  Its combine walks a row's chunk tokens
//   (about 0.35 us each), so beyond 32 of them the context must be worth it: 64 tokens after 2048
//   46 us against 52 (1 x 16), after 512 118 against 95 (16 x 16); 128 after 8192 263 against 369.
// - kTiles: K and V rebuilt once, for everything else.
ChunkPath chunk_path(const rq_shape& s, int n_new, int max_ctx, int window) {
  const int64_t rows = int64_t(s.n_q_heads / s.n_kv_heads) * n_new;
  if (rows <= (window > 0 ? 32 : 8)) return ChunkPath::kStream;
  if (window == 0 && rows <= 128 && (n_new <= 32 || n_new * 32 <= max_ctx)) return ChunkPath::kFused;
  return ChunkPath::kTiles;
}

namespace {

size_t path_bytes(ChunkPath path, const rq_shape& s, int loop, int n_new, int max_ctx, int window, size_t budget) {
  if (path == ChunkPath::kTiles) return chunk_tc_workspace_bytes(s, n_new, max_ctx, window, budget);
  if (path == ChunkPath::kFused) return chunk_fused_workspace_bytes(s, loop, n_new, max_ctx, budget);
  return rows_layout(s, loop, n_new, max_ctx, window, budget).total;
}

}  // namespace

// The way a call with this much workspace runs.  Less than its best plan takes means fewer splits or
// smaller groups, then another way that fits.  A call never needs more than chunk_workspace_bytes gives
// one with more new tokens, more context or a longer window: each way's least need grows with the sizes,
// each way that the larger call may take is open to the smaller one too (kTiles and kStream take any
// rows), and where a smaller one can only stream, the larger one's size counts that.
ChunkPath chunk_path_within(const rq_shape& s, int loop, int n_new, int max_ctx, int window, size_t budget) {
  const int64_t rows = int64_t(s.n_q_heads / s.n_kv_heads) * n_new;
  const ChunkPath best = chunk_path(s, n_new, max_ctx, window);
  if (path_bytes(best, s, loop, n_new, max_ctx, window, budget) <= budget) return best;
  if (window > 0 || rows <= 8 || rows > 128) return ChunkPath::kNone;
  for (ChunkPath other : {ChunkPath::kFused, ChunkPath::kTiles, ChunkPath::kStream}) {
    if (other == ChunkPath::kStream && rows > 32) break;
    if (path_bytes(other, s, loop, n_new, max_ctx, window, budget) <= budget) return other;
  }
  return ChunkPath::kNone;
}

size_t chunk_workspace_bytes(const rq_shape& s, int loop, int n_new, int max_ctx, int window) {
  const ChunkPath path = chunk_path(s, n_new, max_ctx, window);
  size_t most = path_bytes(path, s, loop, n_new, max_ctx, window, SIZE_MAX);
  // shorter contexts that take the other way of up to 128 rows
  if (path == ChunkPath::kFused && n_new > 32) {
    const size_t x = path_bytes(ChunkPath::kTiles, s, loop, n_new, n_new * 32 - 1, window, SIZE_MAX);
    most = x > most ? x : most;
  }
  // fewer tokens, which stream the cache
  const int heads = s.n_q_heads / s.n_kv_heads, few = (window > 0 ? 32 : 8) / heads;
  if (path != ChunkPath::kStream && few > 0) {
    const int n = n_new < few ? n_new : few;
    const size_t x = path_bytes(ChunkPath::kStream, s, loop, n, max_ctx, window < n ? window : n, 0);
    most = x > most ? x : most;
  }
  return most;
}

cudaError_t launch_chunk(const rq_shape& s, const rq_cache& cache, const rq_paging* paging,
                         const ChunkCall& c, ChunkPath path, void* ws, size_t ws_bytes, cudaStream_t stream) {
  char* const w = static_cast<char*>(ws);
  unsigned* err = reinterpret_cast<unsigned*>(w);
  cudaError_t e;
  TailArgs a;
  RowsLayout l = {};
  if (path == ChunkPath::kFused) {
    if ((e = launch_chunk_fused(s, cache, paging, c, ws, ws_bytes, &a.part, &a.n_splits, stream)) != cudaSuccess) return e;
  } else {
    if ((e = cudaMemsetAsync(w, 0, kWsHeaderBytes, stream)) != cudaSuccess) return e;
    if (path == ChunkPath::kTiles) return launch_chunk_tc(s, cache, paging, c, ws, ws_bytes, stream);
    l = rows_layout(s, c.loop, c.n_new, c.max_ctx, c.window, ws_bytes);
    a.part = reinterpret_cast<const float*>(w + l.part);
    a.n_splits = l.plan.n_splits;
    e = launch_chunk_mma(s, cache, paging, c, l.plan, reinterpret_cast<float*>(w + l.part),
                         c.weights ? reinterpret_cast<float*>(w + l.scores) : nullptr, l.score_stride, err, stream);
    if (e != cudaSuccess) return e;
  }
  a.q = c.q;
  a.kv_new = c.kv_new + c.loop * c.kv_strides[3];
  a.qs0 = c.q_strides[0];
  a.qs1 = c.q_strides[1];
  a.qs2 = c.q_strides[2];
  a.ks0 = c.kv_strides[0];
  a.ks1 = c.kv_strides[1];
  a.kv_v = c.kv_strides[2];
  a.ks_h = c.kv_strides[4];
  a.n_lens = c.n_lens;
  a.ctx_lens = c.ctx_lens;
  a.vsigns = c.loop < s.n_loops - 1 ? cache.rot_signs[1] : nullptr;
  a.err = err;
  a.out = c.out;
  a.scores = c.weights ? reinterpret_cast<float*>(w + l.scores) : nullptr;
  a.lse = reinterpret_cast<float*>(w + l.lse);
  a.weights = c.weights;
  a.score_stride = l.score_stride;
  a.B = s.batch;
  a.H = s.n_kv_heads;
  a.heads = s.n_q_heads / s.n_kv_heads;
  a.n_new = c.n_new;
  a.window = c.window;
  a.cap = s.capacity;
  a.max_ctx = c.max_ctx;
  a.vec = ((reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.kv_new) | reinterpret_cast<uintptr_t>(a.out)) & 7) == 0 &&
          ((a.qs0 | a.qs1 | a.qs2 | a.ks0 | a.ks1 | a.kv_v | a.ks_h) & 3) == 0;
  const float scale = s.softmax_scale > 0.f ? s.softmax_scale : 1.0f / sqrtf(float(s.head_dim));
  a.scale_log2 = scale * kLog2e;
  const int64_t warps = int64_t(s.batch) * s.n_q_heads * c.n_new;
  e = launch_after(true, s.head_dim == 128 ? chunk_combine_kernel<128> : chunk_combine_kernel<64>,
                   unsigned((warps + 3) / 4), 128, 0, stream, a);
  if (e != cudaSuccess || !c.weights) return e;
  const dim3 grid((c.max_ctx + c.n_new + 511) / 512, s.n_kv_heads, s.batch);
  return launch_after(true, chunk_weights_kernel, grid, 128, 0, stream, a);
}

}  // namespace rq
