// The line of an attention call over the 8-bit cache: for each sequence, for each block of rows and
// kv-head, the key tiles that the block sees.  It is cut evenly for the CTAs that fit the GPU at once;
// a unit (sequence, block, kv-head) that cuts divide leaves partial results in the workspace.
#pragma once

#include <algorithm>
#include <cmath>

#include "rq_kernels.h"
#include "rq_launch.cuh"
#include "rq_q8.cuh"
#include "rq_tc.cuh"

namespace rq {

constexpr float kNoMax = -3.402823466e38f;   // m of a row that has seen nothing: no finite score is below it
constexpr int kNoScale = -1000;              // h of sums that hold nothing

struct Cut {           // a CTA's stretch of the line
  int64_t pos, base;    // where it begins; where the units of (sequence, block) begin
  int32_t b, block;
};

struct Parted {        // a divided unit: its rows, the CTAs that share it; no rows: there is none
  int32_t b, h, r0, rows, first, last;
};

struct Q8Line {
  Q8View v;
  Q8Call c;
  int32_t B, Hq, G, cap, qvec;
  int32_t blocks;        // blocks of rows, of n_new tokens
  float scale_log2;
  unsigned* err;         // workspace: error word, ...
  int32_t* used;         // CTAs with work
  Parted* parted;        // [CTA] the unit that begins in its stretch and goes on behind it
  int64_t* prefix;       // [B * blocks + 1] places of (sequence, block)
  Cut* cut;              // [CTA + 1]
  float4* stats;         // [2 CTA + (0: the unit began before, 1: goes on)][rows] maxima, sums, units
  float* part;           // ... their sums
  int32_t n_ctas;
  int32_t clear;         // the call's first launch
  int32_t own_cut;       // each CTA cuts for itself
  int32_t least;         // steps of a CTA
  int32_t whole;         // (own_cut) units are not divided
};

// The tiles of 64 slots that some new token of a sequence sees, as a list: 0 .. sink0 and then from
// first0 on; and what a block of ROWS rows sees of it, in steps of KEYS keys.
struct Rows {
  int ctx, n, j0, j1;      // tokens of the block's rows
  int rows;                // of the block
  int sink0, first0, tiles, end;   // the list, its length, the slot behind its last
  int oldest;              // slots before this one are seen as sinks only
  int sink, first, V, hi;  // steps 0 .. sink and from `first` on, V in all; the slot behind the block's last
  bool ok;
  __device__ __forceinline__ int step(int u) const { return u < sink ? u : first + u - sink; }     // the u-th step's place
  __device__ __forceinline__ int tile(int v) const { return v < sink0 ? v : first0 + v - sink0; }  // tile at place v
};

__device__ __forceinline__ Rows sequence_of(const Q8Line& a, int b) {
  Rows x;
  x.ctx = a.c.ctx_lens[b];
  x.n = a.c.n_lens ? a.c.n_lens[b] : a.c.n_new;
  x.ok = x.ctx >= 0 && x.ctx <= a.c.max_ctx && x.n >= 0 && x.n <= a.c.n_new && x.ctx <= a.cap - x.n;
  if (x.n < 0 || x.n > a.c.n_new) x.n = a.c.n_new;
  x.sink0 = x.first0 = x.tiles = x.end = x.oldest = 0;
  if (!x.ok || x.n == 0) return x;
  const int lo = a.c.window > 0 ? max(0, x.ctx + 1 - a.c.window) : 0;
  x.end = x.ctx + x.n;
  x.oldest = lo;
  x.first0 = lo / kQ8Tile;
  x.sink0 = min((min(a.c.n_sink, lo) + kQ8Tile - 1) / kQ8Tile, x.first0);
  x.tiles = x.sink0 + (x.end + kQ8Tile - 1) / kQ8Tile - x.first0;
  return x;
}

template <int ROWS, int KEYS>
__device__ __forceinline__ Rows rows_of(const Q8Line& a, int b, int block) {
  constexpr int K = KEYS / kQ8Tile;
  Rows x = sequence_of(a, b);
  const int r0 = block * ROWS;
  x.rows = min(ROWS, x.n * a.G - r0);
  x.sink = x.first = x.V = x.hi = 0;
  if (x.rows <= 0) return x;
  x.j0 = r0 / a.G;
  x.j1 = (r0 + x.rows - 1) / a.G;
  x.V = 1;                                                  // (bad lengths: one step, not read)
  if (!x.ok) return x;
  const int lo = a.c.window > 0 ? max(0, x.ctx + x.j0 + 1 - a.c.window) : 0, first = lo / kQ8Tile;
  x.hi = x.ctx + x.j1 + 1;
  // (sinks beyond sink0 only where the list begins at tile 0 without a gap: their places are their tiles)
  const int sinks = min((min(a.c.n_sink, lo) + kQ8Tile - 1) / kQ8Tile, first);
  x.first = (x.sink0 + first - x.first0) / K;
  x.sink = min((sinks + K - 1) / K, x.first);
  x.V = x.sink + (x.sink0 + (x.hi + kQ8Tile - 1) / kQ8Tile - x.first0 + K - 1) / K - x.first;
  return x;
}

// CTAs that share a line of N steps: `least` steps each where there are few.
__device__ __forceinline__ int ctas_used(const Q8Line& a, int64_t N) {
  return int(min((N + a.least - 1) / a.least, int64_t(a.n_ctas)));
}

// One CTA: clears the error word and what tells of divided units, cuts the line.
template <int ROWS, int KEYS, int THREADS>
__device__ __forceinline__ void cut_line(const Q8Line& a) {
  __shared__ int64_t warp_sum[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0 && a.clear) *a.err = 0u;
  for (int i = tid; i < a.n_ctas; i += THREADS) a.parted[i].rows = 0;
  const int64_t pairs = int64_t(a.B) * a.blocks;
  int64_t run = 0;
  bool bad = false;
  for (int64_t p0 = 0; p0 < pairs; p0 += THREADS) {
    int64_t units = 0;
    if (p0 + tid < pairs) {
      const Rows x = rows_of<ROWS, KEYS>(a, int((p0 + tid) / a.blocks), int((p0 + tid) % a.blocks));
      bad |= !x.ok;
      units = int64_t(x.V) * a.v.H;
    }
    int64_t sum = units;                                    // inclusive scan over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(RQ_FULL_MASK, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t before = run;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      run += warp_sum[w];
    }
    if (p0 + tid < pairs) a.prefix[p0 + tid] = before + sum - units;
    __syncthreads();
  }
  if (tid == 0) a.prefix[pairs] = run;
  bad = __syncthreads_or(bad);                              // (and the prefix is written)
  if (bad && tid == 0) *a.err = 1u;
  const int used = ctas_used(a, run);
  if (tid == 0) *a.used = used;
  for (int i = tid; i <= used; i += THREADS) {
    const int64_t pos = used ? run * i / used : 0;
    int64_t lo = 0, hi = pairs;                             // the last pair that begins at or before pos
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.prefix[mid] <= pos) lo = mid; else hi = mid;
    }
    a.cut[i] = {pos, a.prefix[lo], int(lo / a.blocks), int(lo % a.blocks)};
  }
}

// The same cut by a CTA of THREADS threads for itself, where there are at most kOwnCutPairs pairs; the
// kernel before then does not cut, and need not be waited for until the error word or
// the workspace is used.
constexpr int kOwnCutPairs = 640;

struct OwnCut {
  Cut from;
  Rows rows;             // what the first (sequence, block) sees
  int64_t to, N;         // where the stretch ends; the line's length
  int32_t used;
  int64_t warp_sum[8];
};

template <int ROWS, int KEYS, int THREADS>
__device__ __forceinline__ bool own_cut(const Q8Line& a, OwnCut& out, int me) {   // whether some length is bad
  constexpr int EACH = (kOwnCutPairs + THREADS - 1) / THREADS, WARPS = THREADS / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = a.B * a.blocks;
  int64_t run = 0;
  int64_t before[EACH];
  int units[EACH];
  bool bad = false;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    before[k] = run;
    units[k] = 0;
    if (k * THREADS >= pairs) continue;
    const int p = tid + k * THREADS;
    if (p < pairs) {
      const Rows x = rows_of<ROWS, KEYS>(a, p / a.blocks, p % a.blocks);
      bad |= !x.ok;
      units[k] = x.V;
    }
    int64_t sum = int64_t(units[k]) * a.v.H;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(RQ_FULL_MASK, sum, o);
      if (lane >= o) sum += y;
    }
    if (lane == 31) out.warp_sum[warp] = sum;
    __syncthreads();
    before[k] = run + sum - int64_t(units[k]) * a.v.H;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before[k] += out.warp_sum[w];
      run += out.warp_sum[w];
    }
    __syncthreads();
  }
  const int used = ctas_used(a, run);
  const int64_t pos = used ? run * me / used : 0, to = used ? run * (me + 1) / used : 0;
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const int p = tid + k * THREADS;
    const int64_t stop = before[k] + int64_t(units[k]) * a.v.H;
    // (whole: a cut inside a unit moves to its end)
    auto cut_at = [&](int64_t x) { return a.whole ? before[k] + (x - before[k] + units[k] - 1) / units[k] * units[k] : x; };
    if (before[k] <= pos && pos < stop) {
      out.from = {cut_at(pos), before[k], p / a.blocks, p % a.blocks};
      out.rows = rows_of<ROWS, KEYS>(a, p / a.blocks, p % a.blocks);
    }
    if (before[k] < to && to <= stop) out.to = cut_at(to);
  }
  if (tid == 0) {
    out.N = run;
    out.used = used;
  }
  return __syncthreads_or(bad);
}

// The parts of a divided unit's row, joined.  A part (m, l, h): its weights' sum l is in units of 2^m, the
// sums with the values in units of 2^(m + h).  Both are joined under the largest unit of their kind, (Mo, h)
// for the second: V's size would not fit beside a weight's.
struct Join {
  float M, sum, Mo, h;
  __device__ __forceinline__ static Join none() { return {kNoMax, 0.f, kNoMax, float(kNoScale)}; }
  // The second unit becomes (m, hn) if that is larger; what the sums before are multiplied by.
  __device__ __forceinline__ float raise(float m, float hn) {
    const float d = (m - Mo) + (hn - h);
    if (!(d > 0.f)) return 1.f;
    Mo = m;
    h = hn;
    return ex2(-d);
  }
  __device__ __forceinline__ float factor(float m, float hn) const { return ex2((m - Mo) + (hn - h)); }
  __device__ __forceinline__ float inverse() const { return sum == 0.f ? 0.f : 1.f / sum; }
  __device__ __forceinline__ float unit() const { return (Mo - M) + h; }
};

// A CTA's segments in order.  (No constructor: it may lie in shared memory, which keeps it out of the
// registers of the threads that read it.)
template <int ROWS, int KEYS>
struct Walk {
  int64_t pos, end, base;   // base: where the units of (b, block) begin
  int64_t unit;             // the unit's place on the line
  int b, block, h, kt0, T;
  Rows x;
  bool loaded, more;
  __device__ __forceinline__ void begin(const Cut& from, int64_t to) {
    pos = from.pos;
    end = to;
    base = from.base;
    b = from.b;
    block = from.block;
    loaded = false;
  }
  __device__ __forceinline__ void begin(const OwnCut& cut) {
    begin(cut.from, cut.to);
    x = cut.rows;
    loaded = true;
  }
  __device__ __forceinline__ bool next(const Q8Line& a) {
    more = advance(a);
    return more;
  }
  __device__ __forceinline__ bool advance(const Q8Line& a) {
    if (pos >= end) return false;
    for (;;) {
      if (!loaded) {
        x = rows_of<ROWS, KEYS>(a, b, block);
        loaded = true;
      }
      const int64_t stop = base + int64_t(x.V) * a.v.H;
      if (pos < stop) break;
      base = stop;
      loaded = false;
      if (x.V == 0 || ++block == a.blocks) {
        block = 0;
        if (++b == a.B) return false;                       // (not with a sound schedule)
      }
    }
    h = int((pos - base) / x.V);
    unit = base + int64_t(h) * x.V;
    kt0 = int(pos - unit);
    T = int(min(int64_t(x.V - kt0), end - pos));
    pos += T;
    return true;
  }
  // The CTAs that share the unit (cut i lies at N i / used; N: the line's length).
  __device__ __forceinline__ void sharers(int64_t N, int used, int& first, int& last) const {
    first = int(((unit + 1) * used + N - 1) / N) - 1;
    last = int(((unit + x.V) * used + N - 1) / N) - 1;
  }
};

inline Q8Line q8_line(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging, const Q8Call& c,
                      int rows) {
  Q8Line a = {};
  a.v = q8_view(s, cache, paging, c.loop);
  a.c = c;
  a.B = s.batch;
  a.Hq = s.n_q_heads;
  a.G = s.n_q_heads / s.n_kv_heads;
  a.cap = s.capacity;
  bool vec = (reinterpret_cast<uintptr_t>(c.q) & 15) == 0;
  for (int i = 0; i < 3; ++i) vec = vec && c.q_strides[i] % 8 == 0;
  a.qvec = vec;
  a.blocks = int((int64_t(c.n_new) * a.G + rows - 1) / rows);
  a.scale_log2 = (s.softmax_scale > 0.f ? s.softmax_scale : 1.0f / sqrtf(float(s.head_dim))) * kLog2e;
  return a;
}

// Places in the workspace, and its size.
struct Q8Layout {
  int n_ctas;
  size_t parted, prefix, cut, stats, part, total;
};

inline Q8Layout q8_layout(const rq_q8_shape& s, int n_new, int max_ctx, int rows, int keys, int fit) {
  Q8Layout x;
  const int64_t all = int64_t(n_new) * (s.n_q_heads / s.n_kv_heads);
  const int64_t tiles = (std::min<int64_t>(int64_t(max_ctx) + n_new, s.capacity) + keys - 1) / keys + 1;
  const int64_t most = int64_t(s.batch) * s.n_kv_heads * ((all + rows - 1) / rows) * tiles;
  x.n_ctas = int(std::min<int64_t>(most, fit));
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  x.parted = kWsHeaderBytes;
  x.prefix = x.parted + up(size_t(x.n_ctas) * sizeof(Parted));
  x.cut = x.prefix + up((size_t(s.batch) * size_t((all + rows - 1) / rows) + 1) * 8);
  x.stats = x.cut + up((size_t(x.n_ctas) + 1) * sizeof(Cut));
  x.part = x.stats + up(size_t(x.n_ctas) * 2 * rows * 16);
  x.total = x.part + up(size_t(x.n_ctas) * 2 * rows * s.head_dim * 4);
  return x;
}

inline void q8_place(Q8Line& a, const Q8Layout& x, void* ws) {
  char* const base = static_cast<char*>(ws);
  a.err = reinterpret_cast<unsigned*>(base);
  a.used = reinterpret_cast<int32_t*>(base + 4);
  a.parted = reinterpret_cast<Parted*>(base + x.parted);
  a.prefix = reinterpret_cast<int64_t*>(base + x.prefix);
  a.cut = reinterpret_cast<Cut*>(base + x.cut);
  a.stats = reinterpret_cast<float4*>(base + x.stats);
  a.part = reinterpret_cast<float*>(base + x.part);
  a.n_ctas = x.n_ctas;
  a.clear = 1;
  a.least = 1;
}

}  // namespace rq
