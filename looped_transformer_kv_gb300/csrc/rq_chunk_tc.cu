// Chunk attention of many rows on the 5th-generation tensor cores (sm_103a).
//
// Many rows share every cached token, so the loop's K and V are rebuilt once per call, in
// original channels, into the workspace as fp16 operand images (rebuild_kernel), and read from
// there by the attention kernel (attention_kernel): S = Q K^T and O += P V as tcgen05 products of
// 128 x 128 tiles, S, P and O in tensor memory.
//   K_t = a_t (s^r c^r + z^r) + R^T (s^e c^e + z^e)        (final loop: the reference alone)
// The chunk's own K and V follow the cached tokens in the same images, so a row's keys are
// 0 .. ctx + j whatever their origin; padding rows are zeros.
//
// Operands are fp16: a rebuilt element and a softmax weight are each rounded once (2^-11
// relative); the queries are exact (a row's bf16 values times a power of two, undone in the
// score's fp32 scale), and a tile with new keys carries a power of two, so that small states keep their
// bits.  Collected weights need more: their scores take K as two fp16 parts.
#include <climits>

#include "rq_common.cuh"
#include "rq_kernels.h"
#include "rq_launch.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr int kKeys = 128;                 // keys per tile (two cache records)
constexpr int kRows = 128;                 // query rows per tile
constexpr unsigned kStateMaxBits = 0x477f0000u;   // the largest bf16 up to 65504, as fp32
constexpr uint64_t kTcWaitLimitNs = 2000000000ull;

__device__ __forceinline__ uint32_t half2_sat(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct ChunkView {     // what every kernel knows of the call
  const int32_t* n_lens;
  const int32_t* ctx_lens;
  unsigned* err;
  int* first_bad;      // [B][H]: first chunk token out of range (0x7f7f7f7f: none)
  uint16_t* exps;      // [unit][tile]: exponents of K's image, and of V's << 8
  int b0, H, heads, n_new, max_ctx, window, tiles;   // tiles: key tiles per (sequence, head)
};

__device__ __forceinline__ bool lens_of(const ChunkView& v, int b, int& n, int& ctx) {
  n = v.n_lens ? v.n_lens[b] : v.n_new;
  ctx = v.ctx_lens[b];
  return n >= 0 && n <= v.n_new && ctx >= 0 && ctx <= v.max_ctx;
}

// Images carry a power of two per tile, undone in its scores' scale and between tiles of different ones
// in O: new states may lie below fp16's normal range (2^-14), so a tile that holds any takes the largest
// multiple of 16 that leaves its bound below 2^15.  A tile of which 1/2 or more is the largest has 0, as
// cached ones always have (their steps and offsets are no finer than fp16's 2^-24 themselves).
// bound: its fp32 bits.
__device__ __forceinline__ int image_exponent(unsigned bound) {
  const int x = int(bound >> 23);                        // in [2^(x - 127), 2^(x - 126))
  return min(max(141 - x, 0) & ~15, 64);                 // (O, below 2^61, times 2^64 is still an fp32)
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// Lengths and block-table entries of the whole batch, where its sequences are handled in several
// groups: what is wrong with a later one has to be known when the first group's outputs are stored.
// A thread per sequence and record.
__global__ void __launch_bounds__(256) check_kernel(const __grid_constant__ ChunkView v, const int32_t* bt, int max_pages,
                                                    int n_pages) {
  grid_next();
  const int b = blockIdx.y, rec = blockIdx.x * 256 + threadIdx.x;
  int n, ctx;
  bool bad = !lens_of(v, b, n, ctx);
  if (!bad && bt && n > 0 && rec < (ctx + kTile - 1) / kTile) {
    const int pg = bt[int64_t(b) * max_pages + rec];
    bad = pg < 0 || pg >= n_pages;
  }
  if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(v.err, 1u);
}

// --------------------------------------------------------------------------------- schedule

// Rows and key tiles of row block `block` of a (sequence, kv-head): key tiles up to the block's last
// row's own token.  A sequence with bad lengths has one tile (its outputs become NaN).
struct BlockInfo {
  int b, h, n, ctx, first, rows, tiles;   // first: the unit's first row (a window's), rows: behind it
  bool ok;
};
__device__ __forceinline__ BlockInfo block_info(const ChunkView& v, int unit, int block, bool window) {
  BlockInfo x;
  x.h = unit % v.H;
  x.b = v.b0 + unit / v.H;
  x.ok = lens_of(v, x.b, x.n, x.ctx);
  if (!x.ok) x.n = x.n < 0 || x.n > v.n_new ? v.n_new : x.n;
  x.first = window ? max(0, x.n - v.window) * v.heads : 0;
  x.rows = x.n * v.heads - x.first;
  const int r0 = block * 2 * kRows;
  const int j_last = (min(r0 + 2 * kRows, x.rows) - 1 + x.first) / v.heads;
  x.tiles = r0 >= x.rows ? 0 : x.ok ? (x.ctx + j_last + kKeys) / kKeys : 1;
  return x;
}

// The attention's work in one line: row blocks, the longest of every unit first, each block's set-up
// (as long as about five key tiles) and its key tiles in order.  The line is cut evenly for one CTA
// per SM; a cut close to a block's edge moves there, because a block that two CTAs share costs a
// merge of their results.  A shorter line is cut for fewer CTAs, yet one for each block that has rows:
// no stretch between two cuts is then shorter than a block of one tile, and every CTA that a merge
// reads from has written.
constexpr int kSetup = 5, kSnap = 7;

struct Schedule {
  int pairs, grid;         // row blocks of all units, CTAs at most
  int* at;                 // [pairs + 1] places of the pairs on the line: pair p is row block
                           // blocks - 1 - p / units of unit p % units
  int2* cut;               // [grid + 1] (place, pair) where each CTA starts
};

// key tile of a place on a pair's stretch
__device__ __forceinline__ int tile_at(int place, int from) { return max(0, place - from - kSetup); }

// One CTA of 256 threads.
__device__ __forceinline__ void write_schedule(const ChunkView& v, const Schedule& s, int units, int blocks) {
  __shared__ int sums[256], counts[256];
  const int per = (s.pairs + 255) / 256;
  const int p0 = min(s.pairs, int(threadIdx.x) * per), p1 = min(s.pairs, p0 + per);
  auto stretch = [&](int p) {
    const int tiles = block_info(v, p % units, blocks - 1 - p / units, false).tiles;
    return tiles ? tiles + kSetup : 0;
  };
  int sum = 0, count = 0;
  for (int p = p0; p < p1; ++p) {
    const int x = stretch(p);
    sum += x;
    count += x > 0 ? 1 : 0;
  }
  sums[threadIdx.x] = sum;
  counts[threadIdx.x] = count;
  __syncthreads();
  int at = 0, total = 0, live = 0;       // live: blocks that have rows
  for (int i = 0; i < 256; ++i) {
    at += i < int(threadIdx.x) ? sums[i] : 0;
    total += sums[i];
    live += counts[i];
  }
  for (int p = p0; p < p1; ++p) {
    s.at[p] = at;
    at += stretch(p);
  }
  if (threadIdx.x == 0) s.at[s.pairs] = total;
  __syncthreads();
  const int ctas = max(1, min(s.grid, max(live, total / 8)));
  for (int c = threadIdx.x; c <= s.grid; c += 256) {
    int x = c >= ctas ? total : int(int64_t(c) * total / ctas);
    int lo = 0, hi = s.pairs;              // the last pair at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s.at[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int from = s.at[lo], to = s.at[lo + 1];
    if (x < to && x > from) {
      if (x - from <= kSnap && x - from <= to - x)
        x = from;
      else if (to - x <= kSnap)
        x = to;
    }
    s.cut[c] = make_int2(x, lo);
  }
}

// ---------------------------------------------------------------------------------- rebuild

struct RebuildArgs {
  ChunkView v;
  const uint8_t* data;
  int64_t rec_bytes;
  const int32_t* bt;
  int max_pages, n_pages, cap;
  int old_tiles;                 // tiles of cached keys, at most
  int bits, sec_off;             // residual bits (0: final loop), offset of the loop's section
  const int8_t* signs[2];
  const uint16_t* kv_new;
  int64_t ks0, ks1, kv_v, ks_h;
  int vec;                       // kv_new rows allow 16-byte loads
  uint8_t *k, *klo, *val;        // images [unit][tile][...]; klo may be null
  Schedule schedule;             // the attention's; at may be null
  int units, blocks;
};

// The residual levels s c + z of one word, as fp16 pairs of neighbouring channels (rounded once;
// LO: and the rest of the fp32 value as a second fp16).
template <int BITS, bool LO>
__device__ __forceinline__ void word_levels(uint32_t w, uint32_t meta, uint32_t* hi, uint32_t* lo) {
  constexpr int HALF = 8 / BITS;                     // pairs per 16 code bits
  constexpr uint32_t MASK = BITS == 2 ? 0x00030003u : 0x000F000Fu;
  const __half2 m = *reinterpret_cast<const __half2*>(&meta);
  const __half2 s = __half2half2(__low2half(m)), z = __half2half2(__high2half(m));
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t x = e ? w >> 16 : w;
    const uint32_t y = __byte_perm(x, x << (16 - BITS), 0x7610);   // halves: codes 0.., codes 1..
#pragma unroll
    for (int i = 0; i < HALF; ++i) {
      const uint32_t c = code_pair_normal(y >> (2 * BITS * i), MASK);
      const __half2 ch = *reinterpret_cast<const __half2*>(&c);
      if constexpr (LO) {
        const float2 cf = __half22float2(ch), mf = __half22float2(m);
        const float v0 = fmaf(mf.x, cf.x, mf.y), v1 = fmaf(mf.x, cf.y, mf.y);
        const uint32_t h = half2_sat(v0, v1);
        const float2 hf = __half22float2(*reinterpret_cast<const __half2*>(&h));
        hi[e * HALF + i] = h;
        lo[e * HALF + i] = half2_sat(v0 - hf.x, v1 - hf.y);
      } else {
        const __half2 v = __hfma2(ch, s, z);
        hi[e * HALF + i] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
  }
}

// x (8 channels as 4 fp32 pairs) += a s c of 8 4-bit codes: a code at bit k of a 16-bit half is
// the exact fp32 c 2^k after subtracting 2^23, its power of two folded into the steps.
__device__ __forceinline__ void add_codes4(uint32_t w, uint64_t s01, uint64_t s23, uint64_t* x) {
  const uint64_t base = pack2(-8388608.f, -8388608.f);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t y = e ? w >> 16 : w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t c = pack2(__uint_as_float((y & (0xFu << (8 * i))) | 0x4B000000u),
                               __uint_as_float((y & (0xF0u << (8 * i))) | 0x4B000000u));
      x[2 * e + i] = fma2(add2(c, base), i ? s23 : s01, x[2 * e + i]);
    }
  }
}

template <int D, int RES, bool KLO>
struct RebuildSmem {
  static constexpr int NG = D / 32;
  static constexpr int kRef = kTile * (D + 8 * NG);                       // one record's sections
  static constexpr int kRes = RES ? kTile * (2 * (D * RES / 8) + 8 * NG + 4) : 0;
  static constexpr int kImg = kKeys * D * 2;
  // H; E, then the images going out (V's and K's low parts in a region of their own where there is
  // room)
  static constexpr int h = 0, e = RES ? 128 * D * 2 : 0, v = RES ? e : e + kImg;
  static constexpr int sec = v + kImg;
  static constexpr int az = sec + 2 * (kRef + kRes), sign = az + kKeys * NG * 8;
  static constexpr int bars = sign + 2 * D * 4, total = bars + 64 + 1024;
  static_assert(total <= 113 * 1024, "two CTAs per SM");
};

// 8 channels of a chunk token's K or V.
__device__ __forceinline__ uint4 load_states(const uint16_t* src, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(src);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = uint32_t(src[2 * k]) | (uint32_t(src[2 * k + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The values of chunk token t (those at or behind token n: zeros); one out of range (beyond 65504, or not
// a number) becomes 0 and `out` the token, so that the images stay finite while its own and later rows
// become NaN.
__device__ __forceinline__ uint32_t state_in_range(uint32_t w, int t, int& out) {
  const bool b0 = (w << 16 & 0x7fffffffu) > kStateMaxBits, b1 = (w & 0x7fff0000u) > kStateMaxBits;
  if (b0 | b1) out = min(out, t);
  return w & (b0 ? 0xffff0000u : 0xffffffffu) & (b1 ? 0x0000ffffu : 0xffffffffu);
}
__device__ __forceinline__ uint4 states_in_range(uint4 w, int t, int n, int& out) {
  if (t >= n) return make_uint4(0u, 0u, 0u, 0u);
  return make_uint4(state_in_range(w.x, t, out), state_in_range(w.y, t, out), state_in_range(w.z, t, out),
                    state_in_range(w.w, t, out));
}
// most: largest magnitudes so far, as bf16 pairs (not-a-number above infinity)
__device__ __forceinline__ void most_states(uint4 w, uint32_t& most) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(most) : "r"(x[k] & 0x7fff7fffu));
}
// fp32 bits of the warp's largest magnitude.
__device__ __forceinline__ unsigned warp_bound(uint32_t most) {
  return __reduce_max_sync(RQ_FULL_MASK, max(most << 16, most & 0xffff0000u));
}
// A pair of them times `up` as fp16 (lo: and the rest of the value).
__device__ __forceinline__ uint32_t state_pair(uint32_t w, float up, uint32_t* lo = nullptr) {
  const float v0 = __uint_as_float(w << 16) * up, v1 = __uint_as_float(w & 0xffff0000u) * up;
  const uint32_t hi = half2_sat(v0, v1);
  if (lo) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    *lo = half2_sat(v0 - f.x, v1 - f.y);
  }
  return hi;
}

// Largest magnitudes of a cached key's levels z .. z + top s over its groups, and (SUM) their norm.
template <int NG, bool SUM>
__device__ __forceinline__ float level_bound(const uint8_t* meta, float top) {
  float most = 0.f, sq = 0.f;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float2 m = __half22float2(*reinterpret_cast<const __half2*>(meta + 4 * g));
    const float x = fmaxf(fabsf(m.y), fabsf(fmaf(top, m.x, m.y)));
    most = fmaxf(most, x);
    sq = fmaf(x, x, sq);
  }
  return SUM ? sqrtf(float(kGroup) * sq) : most;
}

// A tile that holds cached and new keys: bounds of its K and V, into `bounds` (fp32 bits, 0 before).
template <int D, int RES>
__device__ __noinline__ void mixed_bounds(const RebuildArgs& a, int b, int h, int n, int ctx, int t0, int old,
                                          const uint8_t* sec0, unsigned* bounds) {
  constexpr int NG = D / 32, RROW = D * RES / 8;
  constexpr int SIDE = kTile * (D / 2 + 4 * NG), RSIDE = kTile * (RROW + 4 * NG + 2);
  constexpr int REF = kTile * (D + 8 * NG), SEC = REF + (RES ? 2 * RSIDE : 0);
  unsigned found[2] = {0u, 0u};
  if (int(threadIdx.x) < old) {
    const uint8_t* const s = sec0 + (threadIdx.x >> 6) * SEC;
    const int row = threadIdx.x & 63;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float x = level_bound<NG, false>(s + kv * SIDE + kTile * D / 2 + row * NG * 4, 15.f);
      if constexpr (RES != 0) {   // |x| <= |a| largest reference level + norm of the residual levels
        const uint8_t* const r = s + REF + kv * RSIDE + kTile * RROW;
        const float al = __half2float(*reinterpret_cast<const __half*>(r + kTile * 4 * NG + row * 2));
        x = fmaf(fabsf(al), x, level_bound<NG, true>(r + row * NG * 4, RES == 2 ? 3.f : 15.f));
      }
      found[kv] = __float_as_uint(x);
    }
  }
  uint32_t most[2] = {0u, 0u};
  int out = INT_MAX;
  constexpr int C = D / 8, U = 4;            // 16-byte chunks of a row; loads of each side in flight
  const int end = min(n, t0 + kKeys - ctx);  // the tile's new tokens: 0 .. end
  const uint16_t* const src = a.kv_new + b * a.ks0 + h * a.ks_h + 8 * (threadIdx.x % C);
#pragma unroll 1
  for (int t = threadIdx.x / C; t < end; t += U * 256 / C) {
    uint4 y[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)         // (behind the last row: that one again)
        y[u][kv] = load_states(src + int64_t(min(t + u * (256 / C), end - 1)) * a.ks1 + kv * a.kv_v, a.vec);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        most_states(states_in_range(y[u][kv], 0, 1, out), most[kv]);
  }
  __syncwarp();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const unsigned x = max(warp_bound(most[kv]), __reduce_max_sync(RQ_FULL_MASK, found[kv]));
    if ((threadIdx.x & 31) == 0) atomicMax(bounds + kv, x);
  }
}

// The chunk's own keys in the tile that holds the context's end: rows old .. 127 of the image in
// shared memory (zeros behind the last token).  PART 0: K, 1: K's low parts, 2: V.
template <int D, int PART>
__device__ __noinline__ void mixed_rows(const RebuildArgs& a, int b, int h, int n, int ctx, int t0, int old,
                                        float up, uint8_t* img) {
  int out = INT_MAX;
#pragma unroll 1
  for (int i = old * (D / 8) + threadIdx.x; i < kKeys * (D / 8); i += 256) {
    const int key = i / (D / 8), c = i % (D / 8), t = t0 + key - ctx;
    const uint16_t* src = a.kv_new + (PART == 2 ? a.kv_v : 0) + b * a.ks0 + int64_t(min(t, n - 1)) * a.ks1 + h * a.ks_h + 8 * c;
    const uint4 y = states_in_range(load_states(src, a.vec), t, n, out);
    uint32_t lo[4];
    uint32_t w[4] = {state_pair(y.x, up, lo), state_pair(y.y, up, lo + 1), state_pair(y.z, up, lo + 2),
                     state_pair(y.w, up, lo + 3)};
    if constexpr (PART < 2) {
      *reinterpret_cast<uint4*>(img + (c / 8) * (kKeys * 128) + panel_offset(key, c % 8)) =
          PART ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint16_t*>(img + (key >> 6) * (D * 128) + panel_offset(8 * c + e, (key & 63) >> 3) +
                                     (key & 7) * 2) = uint16_t(w[e / 2] >> (16 * (e & 1)));
    }
  }
  if (out != INT_MAX) atomicMin(a.v.first_bad + int64_t(b) * a.v.H + h, out);
}

// Tiles of the chunk's own keys alone: one CTA each (and one for the attention's schedule).  Rows
// are loaded 16 bytes a lane; V goes through shared memory to have channels as rows.  Bound by the
// latency of HBM (2,048 tokens of 8 heads: 7.5 us).
template <int D, bool KLO>
__global__ void __launch_bounds__(256) chunk_image_kernel(const __grid_constant__ RebuildArgs a) {
  grid_wait();
  grid_next();
  if (blockIdx.x == gridDim.x - 1) {            // the attention's schedule
    if (blockIdx.z == 0 && a.schedule.at) write_schedule(a.v, a.schedule, a.units, a.blocks);
    return;
  }
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
  constexpr int IMG = kKeys * D * 2, C = D / 8, IT = kKeys * C / 256;
  uint8_t* const img = smem;                    // K, then V
  uint8_t* const rows = smem + IMG;             // V as it came
  uint8_t* const img_lo = smem + 2 * IMG;
  const int tid = threadIdx.x, h = blockIdx.x % a.v.H, b = a.v.b0 + blockIdx.z;
  int n, ctx;
  if (!lens_of(a.v, b, n, ctx)) {
    if (tid == 0) atomicOr(a.v.err, 1u);
    return;
  }
  const int tile = (ctx + kKeys - 1) / kKeys + blockIdx.x / a.v.H, t0 = tile * kKeys - ctx;   // first token
  if (t0 >= n) return;
  const int c = tid % C;
  const uint16_t* const src = a.kv_new + b * a.ks0 + h * a.ks_h + 8 * c;
  uint4 y[IT], v[IT];
  auto load = [&](int i, uint4& yk, uint4& yv) {
    const uint16_t* p = src + int64_t(min(t0 + (tid + 256 * i) / C, n - 1)) * a.ks1;
    yk = load_states(p, a.vec);
    yv = load_states(p + a.kv_v, a.vec);
  };
  auto convert = [&](int i, const uint4& yk, const uint4& yv, float up_k, float up_v) {
    const int key = (tid + 256 * i) / C;
    uint32_t lo[4];
    const uint4 hi = make_uint4(state_pair(yk.x, up_k, lo), state_pair(yk.y, up_k, lo + 1),
                                state_pair(yk.z, up_k, lo + 2), state_pair(yk.w, up_k, lo + 3));
    const uint32_t o = (c / 8) * (kKeys * 128) + panel_offset(key, c % 8);
    *reinterpret_cast<uint4*>(img + o) = hi;
    if (KLO) *reinterpret_cast<uint4*>(img_lo + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(rows + key * (D * 2) + c * 16) =
        make_uint4(state_pair(yv.x, up_v), state_pair(yv.y, up_v), state_pair(yv.z, up_v), state_pair(yv.w, up_v));
  };
  __shared__ unsigned bounds[2][8];
  auto block_bound = [&](uint32_t most_k, uint32_t most_v, unsigned& k, unsigned& v) {
    most_k = warp_bound(most_k);
    most_v = warp_bound(most_v);
    if (tid % 32 == 0) {
      bounds[0][tid / 32] = most_k;
      bounds[1][tid / 32] = most_v;
    }
    fence_async_smem();
    __syncthreads();
    k = __reduce_max_sync(RQ_FULL_MASK, bounds[0][tid % 8]);
    v = __reduce_max_sync(RQ_FULL_MASK, bounds[1][tid % 8]);
  };
#pragma unroll
  for (int i = 0; i < IT; ++i) load(i, y[i], v[i]);
  uint32_t most_k = 0u, most_v = 0u;
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    if (t0 + (tid + 256 * i) / C >= n) y[i] = v[i] = make_uint4(0u, 0u, 0u, 0u);
    most_states(y[i], most_k);
    most_states(v[i], most_v);
    convert(i, y[i], v[i], 1.f, 1.f);
  }
  unsigned bound_k, bound_v;
  block_bound(most_k, most_v, bound_k, bound_v);
  int ek = 0, ev = 0;
  if (image_exponent(bound_k) | image_exponent(bound_v) || max(bound_k, bound_v) > kStateMaxBits) {
    // a few tiles: once more, without what is out of range and with their powers of two
    int out = INT_MAX;
    uint4 yk, yv;
    most_k = most_v = 0u;
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
      load(i, yk, yv);
      most_states(states_in_range(yk, t0 + (tid + 256 * i) / C, n, out), most_k);
      most_states(states_in_range(yv, t0 + (tid + 256 * i) / C, n, out), most_v);
    }
    if (out != INT_MAX) atomicMin(a.v.first_bad + int64_t(b) * a.v.H + h, out);
    __syncthreads();                            // (the bounds have been read)
    block_bound(most_k, most_v, bound_k, bound_v);
    ek = image_exponent(bound_k);
    ev = image_exponent(bound_v);
#pragma unroll 1
    for (int i = 0; i < IT; ++i) {
      const int t = t0 + (tid + 256 * i) / C;
      load(i, yk, yv);
      convert(i, states_in_range(yk, t, n, out), states_in_range(yv, t, n, out), power_of_two(ek), power_of_two(ev));
    }
    fence_async_smem();
    __syncthreads();
  }
  const int64_t key_tile = (int64_t(blockIdx.z) * a.v.H + h) * a.v.tiles + tile;
  if (tid == 0) a.v.exps[key_tile] = uint16_t(ek | ev << 8);
  const int64_t at = key_tile * IMG;
  if (tid == 0) {
    bulk_s2g(a.k + at, smem_u32(img), IMG);
    if (KLO) bulk_s2g(a.klo + at, smem_u32(img_lo), IMG);
    bulk_s2g_commit();
  }
  // V^T: a thread per channel and 8 keys at a time (lanes: channels)
  uint4 w[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int id = tid + 256 * i, ch = id % D, k0 = id / D * 8;
    uint32_t p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      p[k] = uint32_t(*reinterpret_cast<const uint16_t*>(rows + (k0 + 2 * k) * (D * 2) + ch * 2)) |
             (uint32_t(*reinterpret_cast<const uint16_t*>(rows + (k0 + 2 * k + 1) * (D * 2) + ch * 2)) << 16);
    w[i] = make_uint4(p[0], p[1], p[2], p[3]);
  }
  __syncthreads();                              // `rows` becomes the image
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int id = tid + 256 * i, ch = id % D, k0 = id / D * 8;
    *reinterpret_cast<uint4*>(rows + (k0 >> 6) * (D * 128) + panel_offset(ch, (k0 & 63) >> 3)) = w[i];
  }
  fence_async_smem();
  __syncthreads();
  if (tid == 0) {
    bulk_s2g(a.val + at, smem_u32(rows), IMG);
    bulk_s2g_commit();
    bulk_s2g_wait();
  }
}

// Persistent CTAs over tiles of 128 keys that hold cached ones.  The rotation is undone on the tensor cores:
//   K: D[key][channel] = E H^T,   V: D[channel][key] = H E^T     (E: residual levels, fp16;
// H: Hadamard +-1), and the epilogues add the reference, x = D sign / sqrt(d) + a (s c + z), in
// fp32, round once and write the images through shared memory: a thread per key and half the
// channels for K, per channel and half the keys for V (the V image has channels as rows).
// Bound by instructions and the barriers between its phases (140 warp instructions per token-head
// with 2-bit residuals; two CTAs per SM overlap): 14,336 tokens of 8 heads in 33 us, 2.7 TB/s of
// rows read and images written; with 4-bit residuals and low parts 12,000 of 16 heads in 69 us.
template <int D, int RES, bool KLO>
__global__ void __launch_bounds__(256, 2) rebuild_kernel(const __grid_constant__ RebuildArgs a, int n_items) {
  grid_wait();
  grid_next();
  using L = RebuildSmem<D, RES, KLO>;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  constexpr int NG = D / 32;
  constexpr int SIDE = kTile * (D / 2 + 4 * NG);         // K (or V) part of the reference section
  constexpr int RROW = D * RES / 8;
  constexpr int RSIDE = kTile * (RROW + 4 * NG + 2);
  constexpr int SEC = L::kRef + L::kRes;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  const uint32_t loaded = smem_u32(bars), kdone = loaded + 8, vdone = loaded + 16;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 3);
  float* const sign = reinterpret_cast<float*>(smem + L::sign);            // [2][D], / sqrt(d), times `up`
  unsigned* const bounds = reinterpret_cast<unsigned*>(bars + 4);          // of a tile with new keys
  float* const up = reinterpret_cast<float*>(bars + 5);                    // [2]: powers of two of the images
  float2* const az = reinterpret_cast<float2*>(smem + L::az);              // [pair][group][parity]
  const int tid = threadIdx.x, warp = tid >> 5;
  const int r = tid & 127, hh = tid >> 7;
  const uint32_t lanes = uint32_t(warp & 3) << 21;

  if (RES && warp == 0) tc_alloc(smem_u32(tslot), 256);
  if (tid == 0) {
    mbar_init(loaded, 1);
    mbar_init(kdone, 1);
    mbar_init(vdone, 1);
    fence_mbar_init();
  }
  if constexpr (RES != 0) {   // H as an image of 128 rows (D = 64: its rows twice)
    for (int i = tid; i < 128 * (D / 8); i += 256) {
      const int row = i / (D / 8), c = i % (D / 8);
      uint32_t w[4];
      const uint32_t flip = (__popc(row & (8 * c)) & 1) ? 0x80008000u : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t s0 = uint32_t(__popc(row & (2 * k)) & 1) << 15;
        const uint32_t s1 = uint32_t(__popc(row & (2 * k + 1)) & 1) << 31;
        w[k] = (0x3C003C00u | s0 | s1) ^ flip;
      }
      *reinterpret_cast<uint4*>(smem + L::h + (c / 8) * (128 * 128) + panel_offset(row, c % 8)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = RES ? *tslot : 0u;
  const bool leader = warp == 0 && elect_one();            // issues the products
  const float inv_sqrt_d = (D == 128) ? 0.08838834764831845f : 0.125f;
  int phase = 0;
  bool failed = false, loading = false;

  // record i (0, 1) of a tile; a bad page (flagged) reads as page 0
  auto record = [&](int b, int h, int tile, int i) -> const uint8_t* {
    int64_t rec;
    if (a.bt) {
      int pg = a.bt[int64_t(b) * a.max_pages + 2 * tile + i];
      if (pg < 0 || pg >= a.n_pages) {
        atomicOr(a.v.err, 1u);
        pg = 0;
      }
      rec = int64_t(pg) * a.v.H + h;
    } else {
      rec = (int64_t(b) * a.v.H + h) * (a.cap / kTile) + 2 * tile + i;
    }
    return a.data + rec * a.rec_bytes;
  };
  int bl_known = -1, n = 0, ctx = 0;
  bool lens_good = false;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    // heads first: the heads of a chunk token lie next to each other; the last tile, which may hold new
    // keys and then takes longer, before the others
    const int h = item % a.v.H, tile = a.old_tiles - 1 - item / a.v.H % a.old_tiles, bl = item / a.v.H / a.old_tiles;
    const int b = a.v.b0 + bl, unit = bl * a.v.H + h;
    if (bl != bl_known) {
      bl_known = bl;
      lens_good = lens_of(a.v, b, n, ctx);
      if (!lens_good && tid == 0) atomicOr(a.v.err, 1u);
    }
    if (!lens_good) continue;
    const int t0 = tile * kKeys;
    if (t0 >= ctx || n == 0) continue;
    const int old = min(kKeys, ctx - t0);                  // cached keys of the tile
    uint8_t* const sec0 = smem + L::sec;
    loading = true;
    if (tid == 0) {
      fence_async_smem();
      const int n_rec = old > kTile ? 2 : 1;
      mbar_arrive_expect_tx(loaded, uint32_t(n_rec) * SEC);
      for (int i = 0; i < n_rec; ++i) {
        const uint8_t* src = record(b, h, tile, i);
        const uint32_t dst = smem_u32(sec0) + i * SEC;
        bulk_g2s(dst, src, L::kRef, loaded);
        if (RES) bulk_g2s(dst + L::kRef, src + a.sec_off, L::kRes, loaded);
      }
      // the sections of the next tile of this sequence come to L2 meanwhile
      const int next = item + gridDim.x;
      if (next < n_items && next / a.v.H / a.old_tiles == bl) {
        const int nh = next % a.v.H, nt = a.old_tiles - 1 - next / a.v.H % a.old_tiles;
        for (int i = 0; i < 2 && nt * kKeys + i * kTile < ctx; ++i) {
          const uint8_t* src = record(b, nh, nt, i);
          bulk_prefetch(src, L::kRef);
          if (RES) bulk_prefetch(src + a.sec_off, L::kRes);
        }
      }
      bulk_s2g_wait_read();       // the last tile's image has left
    }
    if (tid < 2 * D) sign[tid] = float(a.signs[tid / D][int64_t(h) * D + tid % D]) * inv_sqrt_d;
    if (tid < 2) {
      bounds[tid] = 0u;
      up[tid] = 1.f;
    }
    __syncthreads();
    constexpr int LOW = KLO && RES ? 16 * NG / 2 : 1;   // fp16 pairs of low parts a thread keeps
    uint32_t e_lo[LOW];
    {
      failed = !mbar_wait_bounded(loaded, phase, kTcWaitLimitNs);
      if (old < kKeys) {
        mixed_bounds<D, RES>(a, b, h, n, ctx, t0, old, sec0, bounds);
        __syncthreads();
        if (tid < 2 * D) sign[tid] *= power_of_two(image_exponent(bounds[tid / D]));
        if (tid < 2) up[tid] = power_of_two(image_exponent(bounds[tid]));
        __syncthreads();
      }
      if (tid == 0)
        a.v.exps[int64_t(unit) * a.v.tiles + tile] =
            old < kKeys ? uint16_t(image_exponent(bounds[0]) | image_exponent(bounds[1]) << 8) : uint16_t(0);
      if constexpr (RES != 0) {   // E of K: a thread per key and half its words
        constexpr int PER = 32 / RES, CPW = PER / 8;      // codes and 16-byte chunks per word
        const int key = tid >> 1;
        const uint8_t* const res = sec0 + (key >> 6) * SEC + L::kRef;
        const int row = key & 63;
        uint32_t m[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) m[g] = *reinterpret_cast<const uint32_t*>(res + kTile * RROW + (row * NG + g) * 4);
#pragma unroll
        for (int jj = 0; jj < RES / 2; ++jj) {
          const int j = 2 * jj + (tid & 1);               // word j of every group
          uint32_t w[NG];
          if constexpr (NG == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(res + row * RROW + j * 16);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(res + row * RROW + j * 8);
            w[0] = x.x, w[1] = x.y;
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            uint32_t hi[PER / 2];
            word_levels<RES, KLO>(w[g], m[g], hi, e_lo + (jj * NG + g) * (KLO ? PER / 2 : 0));
#pragma unroll
            for (int c = 0; c < CPW; ++c)
              *reinterpret_cast<uint4*>(smem + L::e + (g / 2) * (kKeys * 128) + panel_offset(key, (g % 2) * 4 + j * CPW + c)) =
                  make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
          }
        }
        fence_async_smem();
        tc_fence_before();
      }
      // a s and a z of every (key, group) of V
      for (int i = tid; i < kKeys * NG; i += 256) {
        const int t = i / NG, g = i % NG;
        const uint8_t* s = sec0 + (t >> 6) * SEC;
        const float2 m = __half22float2(*reinterpret_cast<const __half2*>(s + SIDE + kTile * D / 2 + ((t & 63) * NG + g) * 4));
        float al = 1.f;
        if (RES)
          al = __half2float(*reinterpret_cast<const __half*>(s + L::kRef + RSIDE + kTile * (RROW + 4 * NG) + (t & 63) * 2));
        al *= up[1];
        // (the odd key's code sits 16 bits higher in its word)
        az[((t >> 1) * NG + g) * 2 + (t & 1)] = make_float2((t & 1) ? m.x * al * 0x1p-16f : m.x * al, m.y * al);
      }
    }
    if (__syncthreads_or(failed)) {
      failed = true;
      break;
    }
    if constexpr (RES != 0) {
      constexpr uint32_t idk = f16_idesc(kKeys, D), idv = f16_idesc(128, kKeys);
      const uint32_t hs = smem_u32(smem + L::h), es = smem_u32(smem + L::e);
      auto k_products = [&](bool add) {
        if (leader) {
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            tc_mma(tmem, panel_desc(es + (x / 4) * (kKeys * 128) + (x % 4) * 32),
                   panel_desc(hs + (x / 4) * (128 * 128) + (x % 4) * 32), idk, add || x > 0);
          tc_commit(kdone);
        }
      };
      k_products(false);
      if constexpr (KLO) {     // the levels' low parts, in the same place
        failed = !mbar_wait_bounded(kdone, 0, kTcWaitLimitNs);
        if (__syncthreads_or(failed)) {
          failed = true;
          break;
        }
        tc_fence_after();
        constexpr int PER = 32 / RES, CPW = PER / 8;
#pragma unroll
        for (int jj = 0; jj < RES / 2; ++jj)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int c = 0; c < CPW; ++c) {
              const uint32_t* lo = e_lo + (jj * NG + g) * (PER / 2) + 4 * c;
              const int j = 2 * jj + (tid & 1);
              *reinterpret_cast<uint4*>(smem + L::e + (g / 2) * (kKeys * 128) + panel_offset(tid >> 1, (g % 2) * 4 + j * CPW + c)) =
                  make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        k_products(true);
      }
      // E of V: a thread per pair of keys and 16 bytes of its words (4 units of both keys)
      constexpr int CHUNKS = D * RES / 64;                // 16-byte chunks of a pair's words
      constexpr int IT = (64 * CHUNKS + 255) / 256;
      uint4 w[IT];
      uint32_t m[IT][2];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int id = tid + 256 * i, p = id / CHUNKS, c = id % CHUNKS, row = (2 * p) & 63;
        if (id >= 64 * CHUNKS) continue;
        const uint8_t* const res = sec0 + (p >> 5) * SEC + L::kRef + RSIDE;
        const int u0 = (4 * c) ^ v_unit_swizzle(p & 31, RROW / 2), g = u0 * (16 / RES) / 32;
        w[i] = *reinterpret_cast<const uint4*>(res + (p & 31) * 2 * RROW + c * 16);
        m[i][0] = *reinterpret_cast<const uint32_t*>(res + kTile * RROW + (row * NG + g) * 4);
        m[i][1] = *reinterpret_cast<const uint32_t*>(res + kTile * RROW + ((row + 1) * NG + g) * 4);
      }
      failed = !mbar_wait_bounded(kdone, KLO ? 1 : phase, kTcWaitLimitNs);
      if (__syncthreads_or(failed)) {
        failed = true;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int id = tid + 256 * i, p = id / CHUNKS, c = id % CHUNKS;
        if (id >= 64 * CHUNKS) continue;
        const int u0 = (4 * c) ^ v_unit_swizzle(p & 31, RROW / 2);
        constexpr int PER = 32 / RES, CPW = PER / 8;
        const int chunk0 = u0 * (16 / RES) / 8;           // its first channels, in 16-byte chunks
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t words[2] = {__byte_perm(w[i].x, w[i].y, e ? 0x7632 : 0x5410),
                                     __byte_perm(w[i].z, w[i].w, e ? 0x7632 : 0x5410)};
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t hi[PER / 2], lo[PER / 2];
            word_levels<RES, false>(words[k], m[i][e], hi, lo);
#pragma unroll
            for (int q = 0; q < CPW; ++q) {
              const int chunk = chunk0 + k * CPW + q;
              *reinterpret_cast<uint4*>(smem + L::e + (chunk / 8) * (kKeys * 128) + panel_offset(2 * p + e, chunk % 8)) =
                  make_uint4(hi[4 * q], hi[4 * q + 1], hi[4 * q + 2], hi[4 * q + 3]);
            }
          }
        }
      }
      fence_async_smem();
      tc_fence_before();
      __syncthreads();
      if (leader) {
        tc_fence_after();
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          tc_mma(tmem + 128, panel_desc(hs + (x / 4) * (128 * 128) + (x % 4) * 32),
                 panel_desc(es + (x / 4) * (kKeys * 128) + (x % 4) * 32), idv, x > 0);
        tc_commit(vdone);
      }
    }
    const int64_t at = (int64_t(unit) * a.v.tiles + tile) * L::kImg;
    uint64_t x[D / 4];             // K epilogue: key r, of every group channels 16 hh ..
    {
      const uint8_t* const sec = sec0 + (r >> 6) * SEC;
      const int row = r & 63;
      float al = 1.f;
      if (RES) al = __half2float(*reinterpret_cast<const __half*>(sec + L::kRef + kTile * (RROW + 4 * NG) + row * 2));
      al *= up[0];
      // words 2 hh and 2 hh + 1 of every group
      uint32_t w[2][NG];
      if constexpr (NG == 4) {   // (odd row pairs read them in the other order: distinct banks)
        const int swap = (r >> 1) & 1;
        uint4 y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          y[k] = *reinterpret_cast<const uint4*>(sec + row * (D / 2) + (2 * hh + (k ^ swap)) * 16);
        const uint4 y0 = swap ? y[1] : y[0], y1 = swap ? y[0] : y[1];
        w[0][0] = y0.x, w[0][1] = y0.y, w[0][2] = y0.z, w[0][3] = y0.w;
        w[1][0] = y1.x, w[1][1] = y1.y, w[1][2] = y1.z, w[1][3] = y1.w;
      } else {
        const uint4 y = *reinterpret_cast<const uint4*>(sec + row * (D / 2) + hh * 16);
        w[0][0] = y.x, w[0][1] = y.y, w[1][0] = y.z, w[1][1] = y.w;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float2 m = __half22float2(*reinterpret_cast<const __half2*>(sec + kTile * D / 2 + (row * NG + g) * 4));
        const float as = m.x * al, z = m.y * al;
        const uint64_t s01 = pack2(as, as * 0x1p-4f), s23 = pack2(as * 0x1p-8f, as * 0x1p-12f), zz = pack2(z, z);
        if constexpr (RES != 0) {
          uint32_t d[16];
          tc_ld16(tmem + lanes + 32 * g + 16 * hh, d);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[8 * g + i] = fma2(pack2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])),
                                *reinterpret_cast<const uint64_t*>(sign + g * 32 + 16 * hh + 2 * i), zz);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[8 * g + i] = zz;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) add_codes4(w[k][g], s01, s23, x + 8 * g + 4 * k);
      }
    }
    if (RES) {
      failed = !mbar_wait_bounded(vdone, phase, kTcWaitLimitNs);       // E is free
      tc_fence_after();
    }
    auto k_image = [&](uint8_t* img, bool low) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float x0, x1;
          unpack2(x[4 * i + k], x0, x1);
          w[k] = half2_sat(x0, x1);
          if (low) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            w[k] = half2_sat(x0 - f.x, x1 - f.y);
          }
        }
        const int g = i / 2, chunk = (g % 2) * 4 + 2 * hh + i % 2;
        *reinterpret_cast<uint4*>(img + (g / 2) * (kKeys * 128) + panel_offset(r, chunk)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    k_image(smem + L::e, false);
    // the chunk's own keys of the last cached tile over the rows behind the context
    if (old < kKeys) {
      __syncthreads();
      mixed_rows<D, 0>(a, b, h, n, ctx, t0, old, up[0], smem + L::e);
    }
    fence_async_smem();
    if (__syncthreads_or(failed)) {
      failed = true;
      break;
    }
    if (tid == 0) {
      bulk_s2g(a.k + at, smem_u32(smem + L::e), L::kImg);
      bulk_s2g_commit();
      if (L::v == L::e) bulk_s2g_wait_read();
    }
    if constexpr (KLO) {
      if (L::v == L::e) __syncthreads();                  // K's image has left
      k_image(smem + L::v, true);
      if (old < kKeys) {
        __syncthreads();
        mixed_rows<D, 1>(a, b, h, n, ctx, t0, old, up[0], smem + L::v);
      }
      fence_async_smem();
      __syncthreads();
      if (tid == 0) {
        bulk_s2g(a.klo + at, smem_u32(smem + L::v), L::kImg);
        bulk_s2g_commit();
        bulk_s2g_wait_read();
      }
    }
    // ---- V epilogue: channel ch, 32 keys at a time from k0 of record rec
    constexpr int QS = D / 64;
    const int ch = r & (D - 1), g = ch >> 5, u4 = (ch >> 2) * 4, nib = 4 * (ch & 3);
    const int part = D == 128 ? 0 : r >> 6;               // (D = 64: lanes 64 .. hold the channels again)
    const float sg = RES ? sign[D + ch] : 0.f;
    const uint64_t sg2 = pack2(sg, sg), base = pack2(-8388608.f, -8388608.f);
    if (KLO || L::v == L::e) __syncthreads();             // the image before has left
#pragma unroll 1
    for (int q = 0; q < QS; ++q) {
      const int k0 = hh * 64 + (D == 128 ? q : part) * 32;     // first key of these
      uint32_t d[32];
      if constexpr (RES != 0) {
        tc_ld32(tmem + 128 + lanes + k0, d);
        tc_wait_ld();
      }
      float v[32];
      const uint8_t* const words = sec0 + hh * SEC + SIDE + (D == 128 ? q : part) * 16 * D;
      const float2* const azk = az + ((k0 >> 1) * NG + g) * 2;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        constexpr int UNITS = D / 4;
        const int swz = UNITS == 32 ? 8 * (k & 3) : 8 * ((k >> 1) & 1);    // (16 pairs: k decides)
        const uint32_t word = *reinterpret_cast<const uint32_t*>(words + k * D + (u4 ^ (swz * 4))) >> nib;
        const float4 f = *reinterpret_cast<const float4*>(azk + k * NG * 2);
        uint64_t y = pack2(f.y, f.w);
        if constexpr (RES != 0)
          y = fma2(pack2(__uint_as_float(d[2 * k]), __uint_as_float(d[2 * k + 1])), sg2, y);
        const uint64_t code = pack2(__uint_as_float((word & 0xFu) | 0x4B000000u),
                                    __uint_as_float((word & 0xF0000u) | 0x4B000000u));
        unpack2(fma2(add2(code, base), pack2(f.x, f.z), y), v[2 * k], v[2 * k + 1]);
      }
      const int c0 = (D == 128 ? q : part) * 4;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = half2_sat(v[8 * c + 2 * k], v[8 * c + 2 * k + 1]);
        *reinterpret_cast<uint4*>(smem + L::v + hh * (D * 128) + panel_offset(ch, c0 + c)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (old < kKeys) {
      __syncthreads();
      mixed_rows<D, 2>(a, b, h, n, ctx, t0, old, up[1], smem + L::v);
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();                                      // (sections, az and D are free)
    tc_fence_after();
    if (tid == 0) {
      bulk_s2g(a.val + at, smem_u32(smem + L::v), L::kImg);
      bulk_s2g_commit();
    }
    phase ^= 1;
    loading = false;
  }
  if (tid == 0) {
    if (failed) {
      atomicOr(a.v.err, 1u);
      if (loading) mbar_wait_bounded(loaded, phase, kTcWaitLimitNs);     // (a copy that is still in flight)
    }
    bulk_s2g_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (RES && warp == 0) tc_free(tmem, 256);
}

// -------------------------------------------------------------------------------- attention

struct AttnArgs {
  ChunkView v;
  const uint16_t* q;
  int64_t qs0, qs1, qs2;
  int qvec;                // q rows allow 16-byte loads
  const uint8_t *k, *klo, *val;
  uint16_t* out;
  Schedule schedule;       // (SCHED)
  float* part;             // O images (below) of shared blocks, by row tile: SCHED [2 CTA + (0 first,
                           // 1 last)][2], else [unit][split][row_tiles]
  float2* stats;           // (m, l) of their rows, and LSE's
  int n_splits, row_tiles; // (not SCHED) row_tiles: of 128 rows, of a unit
  int units, blocks;       // row blocks (of 256) of a unit
  float scale_log2;
};

template <int D>
struct AttnSmem {
  static constexpr int kTileBytes = kKeys * D * 2;      // one K, V^T or Q tile
  static constexpr int q = 0, k = 2 * kTileBytes, v = k + 3 * kTileBytes, exps = v + 2 * kTileBytes;
  static constexpr int bars = exps + 2 * kRows * 4;
  static constexpr int total = bars + 256 + 1024;       // + alignment of the base
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

// 32 rows of queries (this warp's rows of a tile) -> fp16 in the swizzled tile image, each row
// scaled by a power of two so that its largest element lies in [2^14, 2^15); exps: the exponents,
// undone in the scores' scale.  `row_ptr(r)`: row r's values, or null (zeros).
template <int D, typename RowPtr>
__device__ __forceinline__ void store_queries(RowPtr row_ptr, bool vec, uint8_t* img, int* exps, int r0, int lane) {
  constexpr int LPR = D / 8, RPI = 32 / LPR;             // lanes per row, rows at a time
  const int c = lane % LPR, sub = lane / LPR;
  uint4 v[32 / RPI];
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const uint16_t* p = row_ptr(r0 + i * RPI + sub);
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p == nullptr) continue;
    if (vec) {
      v[i] = *reinterpret_cast<const uint4*>(p + 8 * c);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = uint32_t(p[8 * c + 2 * k]) | (uint32_t(p[8 * c + 2 * k + 1]) << 16);
      v[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 32 / RPI; ++i) {
    const int r = r0 + i * RPI + sub;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    float f[8], mx = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      mx = fmaxf(mx, fmaxf(fabsf(f[2 * k]), fabsf(f[2 * k + 1])));
    }
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(RQ_FULL_MASK, mx, o));
    // mx in [2^(x-127), 2^(x-126)), x its exponent field: scale by 2^(14 - (x - 127))
    const int x = int(__float_as_uint(mx) >> 23);
    const int e = x == 0 || x == 255 ? 0 : min(141 - x, 100);   // (0, subnormal, inf: as they are)
    const float up = __uint_as_float(uint32_t(127 + (e >> 1)) << 23);
    const float up2 = __uint_as_float(uint32_t(127 + e - (e >> 1)) << 23);
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = pack_half2(f[2 * k] * up * up2, f[2 * k + 1] * up * up2);
    *reinterpret_cast<uint4*>(img + (c / 8) * (kRows * 128) + panel_offset(r, c % 8)) =
        make_uint4(o[0], o[1], o[2], o[3]);
    if (c == 0) exps[r] = e;
  }
  __syncwarp();
}

// A row tile's O image in the workspace: 128 rows of D floats, the 16-byte chunk c of row r at
// chunk position c ^ (r % (D / 4)).
template <int D>
__device__ __forceinline__ int o_image_offset(int r, int c) {
  return r * (D * 4) + ((c ^ (r & (D / 4 - 1))) << 4);
}

__device__ __forceinline__ uint32_t times(uint32_t x, float f) { return __float_as_uint(__uint_as_float(x) * f); }

__device__ __forceinline__ void warpgroup_barrier(int i) {   // 128 threads of warpgroup 0 or 1
  if (i == 0)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else
    asm volatile("bar.sync 2, 128;" ::: "memory");
}

// The same, and whether `x` holds for any of them.
__device__ __forceinline__ bool warpgroup_any(int i, bool x) {
  uint32_t y;
  if (i == 0)
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y) : "r"(uint32_t(x)) : "memory");
  else
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y) : "r"(uint32_t(x)) : "memory");
  return y != 0u;
}

// A CTA's work is one or more segments: a row block of 256 query rows (two tiles of 128) and a range
// of its key tiles, every K and V tile shared by the two.  Warps 0-3 and 4-7: softmax of row tile 0
// and 1, a thread per row; warp 8: copies; warp 9: products.  While one row tile's softmax runs, the
// other's products do:  S_0 S_1 | P_0 V, S_0' | P_1 V, S_1' | ...
// Weights are 2^(S - m); m is raised only when one would exceed 2^15, to make the tile's largest 2^7
// (O is rescaled in tensor memory then); P overwrites S's columns.  The softmax warps take registers
// from the others, so that a row's 128 scores stay in registers.
// SCHED: the CTAs share the key tiles evenly (one CTA per SM): a block that lies in one CTA's range
// is stored, the others leave their (m, l, O) for merge_kernel, at most two per CTA.  Else one CTA
// takes one split of one row block.  Sharing evenly wins where a CTA gets many tiles (2048 tokens x
// 4 heads after 14336: 325 + 15 us against 376 + 34 us and 134 MB left to merge), splits where it
// gets few (a ragged first chunk of 1023: 45 us against 54, each segment's set-up counts).
// LSE: scores with K in two parts, no P and V; (m, l) per row and split are stored.
// Bound by the products: 515 GFLOP in 325 us, 1,585 TFLOP/s (the tensor pipe active 70 % of the time,
// at the clock that the power limit leaves); a chunk with few key tiles per CTA by each CTA's
// set-up and the latency of its first and last tiles.
template <int D, bool LSE, bool SCHED>
__global__ void __launch_bounds__(384, 1) attention_kernel(const __grid_constant__ AttnArgs a) {
  grid_wait();
  grid_next();
  extern __shared__ uint8_t raw[];
  using L = AttnSmem<D>;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  // barriers: K full [3], V full [2], S ready [row tile][2], P ready [2], Q ready, done.  S of a key
  // tile being ready also means that the values of the tile before are done, so the copies wait
  // for it and need no barriers of their own (each commit stalls the products).
  const uint32_t bar0 = smem_u32(bars);
  auto kfull = [&](int g) { return bar0 + 8 * (g % 3); };
  auto vfull = [&](int g) { return bar0 + 8 * (3 + (g & 1)); };
  auto sready = [&](int i, int c) { return bar0 + 8 * (5 + 2 * i + (c & 1)); };
  auto pready = [&](int i) { return bar0 + 8 * (9 + i); };
  const uint32_t qready = bar0 + 8 * 11, done = bar0 + 8 * 12;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 13);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the CTA's stretch [begin, end) of the line, and a pair at or before its start
  int begin = 0, end = 0, pair = 0, split_kt = 0;
  BlockInfo only{};                                          // (not SCHED) the CTA's row block
  if constexpr (SCHED) {
    const int2 cut = a.schedule.cut[blockIdx.x];
    begin = cut.x;
    pair = cut.y;
    end = a.schedule.cut[blockIdx.x + 1].x;
    if (begin == end) return;
  } else {
    pair = int(blockIdx.y) * a.units + int(blockIdx.x) / a.n_splits;
    only = block_info(a.v, pair % a.units, a.blocks - 1 - pair / a.units, LSE);
    const int split = int(blockIdx.x) % a.n_splits;
    if (only.tiles == 0) return;
    split_kt = int(int64_t(split) * only.tiles / a.n_splits);
    end = int(int64_t(split + 1) * only.tiles / a.n_splits) - split_kt;
  }
  // (one thread reads the error word: another CTA may be setting it)
  const bool flagged = __syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile unsigned*>(a.v.err) != 0u);

  // Walks the CTA's segments in order: next() is false behind the last one.
  struct Walk {
    const AttnArgs& a;
    int begin, x, end, p, split_kt, segments;
    BlockInfo block;
    int unit, r0, kt0, T;      // key tiles kt0 .. kt0 + T of the block
    bool whole, at_begin, two;
    __device__ __forceinline__ Walk(const AttnArgs& args, int begin_, int end_, int pair_, int split_kt_, const BlockInfo& only)
        : a(args), begin(begin_), x(begin_), end(end_), p(pair_), split_kt(split_kt_), segments(0), block(only) {}
    __device__ __forceinline__ void take(int pair) {
      unit = pair % a.units;
      r0 = (a.blocks - 1 - pair / a.units) * 2 * kRows;
      if constexpr (SCHED) block = block_info(a.v, unit, a.blocks - 1 - pair / a.units, LSE);
      two = r0 + kRows < block.rows;
    }
    __device__ __forceinline__ bool next() {
      if constexpr (!SCHED) {  // one segment (an empty split's has no tiles)
        if (segments++ > 0) return false;
        take(p);
        kt0 = split_kt;
        T = end;
        whole = !LSE && a.n_splits == 1;
        return true;
      }
      while (x < end) {
        while (a.schedule.at[p + 1] <= x) ++p;
        const int from = a.schedule.at[p], to = a.schedule.at[p + 1], stop = min(end, to);
        kt0 = tile_at(x, from);
        T = tile_at(stop, from) - kt0;
        whole = kt0 == 0 && stop == to;
        at_begin = begin >= from;
        x = stop;
        if (T == 0) continue;  // (a stretch inside the block's set-up)
        take(p);
        return true;
      }
      return false;
    }
  };

  if (warp == 9) tc_alloc(smem_u32(tslot), 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 9; ++i) mbar_init(bar0 + 8 * i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(pready(i), kRows);
    mbar_init(qready, 2 * kRows);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool failed = false;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const bool leader = elect_one();
    if (warp == 8 && leader && end > begin) {                       // ---- copies
      // K and V run ahead of the scores: a walk each, in tiles from the CTA's first
      Walk wk(a, begin, end, pair, split_kt, only), wv(wk), ws(wk);
      wk.T = wv.T = ws.T = 0;
      int nk = 0, nv = 0, jk = 0, jv = 0;                            // copies issued; tiles of the walk's segment
      bool more_k = true, more_v = true;
      auto load_k = [&]() {
        if (jk == wk.T) {
          jk = 0;
          if (!(more_k = wk.next())) return;
        }
        const int64_t at = (int64_t(wk.unit) * a.v.tiles + wk.kt0 + jk++) * L::kTileBytes;
        mbar_arrive_expect_tx(kfull(nk), L::kTileBytes);
        bulk_g2s(smem_u32(smem + L::k + (nk % 3) * L::kTileBytes), a.k + at, L::kTileBytes, kfull(nk));
        ++nk;
      };
      auto load_v = [&]() {
        if (jv == wv.T) {
          jv = 0;
          if (!(more_v = wv.next())) return;
        }
        const int64_t at = (int64_t(wv.unit) * a.v.tiles + wv.kt0 + jv++) * L::kTileBytes;
        mbar_arrive_expect_tx(vfull(nv), L::kTileBytes);
        bulk_g2s(smem_u32(smem + L::v + (nv & 1) * L::kTileBytes), (LSE ? a.klo : a.val) + at, L::kTileBytes, vfull(nv));
        ++nv;
      };
      for (int i = 0; i < 3 && more_k; ++i) {
        load_k();
        if (i < (LSE ? 2 : 1) && more_v) load_v();   // (with more of V the products could lap the waits below)
      }
      int c1 = 0, js = 0;                                            // tiles of row tile 1 so far (tile 0: g)
      for (int g = 0; more_v; ++g) {
        if (js == ws.T) {
          js = 0;
          if (!ws.next()) break;
        }
        ++js;
        // scores of tile g done, so the values of the tile before: room for K g + 3 and V g + 1
        // (LSE: V holds K's low parts, done with the scores: g + 2)
        const int i = ws.two ? 1 : 0, ci = i ? c1 : g;
        if (!mbar_wait_bounded(sready(i, ci), (ci >> 1) & 1, kTcWaitLimitNs)) {
          failed = true;
          break;
        }
        c1 += i;
        if (more_k) load_k();
        if (nv < g + (LSE ? 3 : 2)) load_v();
      }
      for (int j = max(0, nk - 3); j < nk; ++j) failed |= !mbar_wait_bounded(kfull(j), (j / 3) & 1, kTcWaitLimitNs);
      for (int j = max(0, nv - 2); j < nv; ++j) failed |= !mbar_wait_bounded(vfull(j), (j >> 1) & 1, kTcWaitLimitNs);
    } else if (warp == 9 && leader && end > begin) {                // ---- products
      constexpr uint32_t ids = f16_idesc(kRows, kKeys), ido = f16_idesc(kRows, D);
      int c1 = 0, g = 0, seg = 0;                                    // tiles of row tile 1, of the CTA (and row tile 0); segments
      bool good = true;
      auto scores = [&](int i, int gk, int ci) {
        const uint32_t q = smem_u32(smem + L::q + i * L::kTileBytes), k = smem_u32(smem + L::k + (gk % 3) * L::kTileBytes);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          tc_mma(tmem + 128 * i, panel_desc(q + (x / 4) * (kRows * 128) + (x % 4) * 32),
                 panel_desc(k + (x / 4) * (kKeys * 128) + (x % 4) * 32), ids, x > 0);
        if (LSE) {
          const uint32_t k2 = smem_u32(smem + L::v + (gk & 1) * L::kTileBytes);
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            tc_mma(tmem + 128 * i, panel_desc(q + (x / 4) * (kRows * 128) + (x % 4) * 32),
                   panel_desc(k2 + (x / 4) * (kKeys * 128) + (x % 4) * 32), ids, true);
        }
        tc_commit(sready(i, ci));
      };
      auto values = [&](int i, int gv, bool add) {
        const uint32_t v = smem_u32(smem + L::v + (gv & 1) * L::kTileBytes);
#pragma unroll
        for (int x = 0; x < kKeys / 16; ++x)
          tc_mma_ta(tmem + 256 + 128 * i, tmem + 128 * i + 8 * x, panel_desc(v + (x / 4) * (D * 128) + (x % 4) * 32),
                    ido, add || x > 0);
      };
      auto k_there = [&](int gk) {
        return mbar_wait_bounded(kfull(gk), (gk / 3) & 1, kTcWaitLimitNs) &&
               (!LSE || mbar_wait_bounded(vfull(gk), (gk >> 1) & 1, kTcWaitLimitNs));
      };
      for (Walk w(a, begin, end, pair, split_kt, only); good && w.next(); ++seg) {
        const int I = w.two ? 2 : 1;
        good = k_there(g) && mbar_wait_bounded(qready, seg & 1, kTcWaitLimitNs);
        tc_fence_after();
        if (good)
          for (int i = 0; i < I; ++i) scores(i, g, i ? c1 : g);
        for (int j = 0; j < w.T && good; ++j, ++g) {
          if (!LSE) good = mbar_wait_bounded(vfull(g), (g >> 1) & 1, kTcWaitLimitNs);
          if (good && j + 1 < w.T) good = k_there(g + 1);
          for (int i = 0; i < I && good; ++i) {
            const int ci = i ? c1++ : g;
            good = mbar_wait_bounded(pready(i), ci & 1, kTcWaitLimitNs);
            if (!good) break;
            tc_fence_after();
            if (!LSE) values(i, g, j > 0);
            if (j + 1 < w.T) scores(i, g + 1, ci + 1);
          }
        }
        tc_commit(done);
        // nothing in flight, no arrival outstanding when the CTA leaves (else the softmax waits for it)
        if (LSE || !good) good &= mbar_wait_bounded(done, seg & 1, kTcWaitLimitNs);
      }
      failed = !good;
    }
    __syncwarp();
  } else {                                                           // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int i = warp >> 2, r = threadIdx.x & (kRows - 1);
    const uint32_t lanes = uint32_t(warp & 3) << 21;                 // this warp's tensor-memory lanes
    const uint32_t tS = tmem + 128 * i + lanes, tO = tmem + 256 + 128 * i + lanes;
    int* const exps = reinterpret_cast<int*>(smem + L::exps) + i * kRows;
    uint8_t* const img = smem + L::q + i * L::kTileBytes;            // queries, then results going out
    int ci = 0, seg = 0;
    for (Walk w(a, begin, end, pair, split_kt, only); !failed && w.next(); ++seg) {
      const BlockInfo& x = w.block;
      const int row = w.r0 + i * kRows + r;
      const bool valid = row < x.rows;
      float m = -INFINITY, l = 0.f;
      int ev = 0;                                                    // O's exponent
      const uint16_t* const exps_of = a.v.exps + int64_t(w.unit) * a.v.tiles + w.kt0;
      int exps32 = lane < w.T ? exps_of[lane] : 0;                    // a lane's of the next 32 tiles
      if (w.T > 0) {
        if (i == 0 || w.two)
          store_queries<D>(
              [&](int rr) -> const uint16_t* {
                const int y = w.r0 + i * kRows + rr;
                if (y >= x.rows) return nullptr;
                const int j = (y + x.first) / a.v.heads, g = (y + x.first) % a.v.heads;
                return a.q + x.b * a.qs0 + j * a.qs1 + (int64_t(x.h) * a.v.heads + g) * a.qs2;
              },
              a.qvec, img, exps, (warp & 3) * 32, lane);
        fence_async_smem();
        mbar_arrive(qready);
      }
      if (i == 1 && !w.two) {    // no rows: only keeps step with the segments
        if (SCHED) failed = warpgroup_any(i, !mbar_wait_bounded(done, seg & 1, kTcWaitLimitNs));
        continue;
      }
      if (w.T > 0) {
        const float c = ldexpf(a.scale_log2, -exps[r]);
        const int lim = x.ctx + min((row + x.first) / a.v.heads, x.n - 1);   // last key the row sees
        const int clear = x.ctx + min((w.r0 + i * kRows + x.first) / a.v.heads, x.n - 1);   // every row of the tile sees these
        for (int jt = 0; jt < w.T; ++jt, ++ci) {
          if ((jt & 31) == 0 && jt > 0) exps32 = jt + lane < w.T ? exps_of[jt + lane] : 0;
          const int tile_exps = __shfl_sync(RQ_FULL_MASK, exps32, jt & 31), tile_ev = tile_exps >> 8;
          const float ct = c * power_of_two(-(tile_exps & 255));
          const bool good = mbar_wait_bounded(sready(i, ci), (ci >> 1) & 1, kTcWaitLimitNs);
          if (__any_sync(RQ_FULL_MASK, !good)) {                      // (the warp leaves as one)
            failed = true;
            break;
          }
          tc_fence_after();
          uint32_t s[kKeys];
#pragma unroll
          for (int y = 0; y < 4; ++y) tc_ld32(tS + 32 * y, s + 32 * y);
          tc_wait_ld();
          const int key0 = (w.kt0 + jt) * kKeys;
          if (key0 + kKeys - 1 > clear) {
            const int rel = lim - key0;
#pragma unroll
            for (int y = 0; y < kKeys; ++y)
              if (y > rel) s[y] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) mx[y] = __uint_as_float(s[y]);
#pragma unroll
          for (int y = 4; y + 4 < kKeys; y += 8)
#pragma unroll
            for (int z = 0; z < 4; ++z)
              mx[z] = fmaxf(mx[z], fmaxf(__uint_as_float(s[y + z]), __uint_as_float(s[y + z + 4])));
#pragma unroll
          for (int y = kKeys - 4; y < kKeys; ++y) mx[y & 3] = fmaxf(mx[y & 3], __uint_as_float(s[y]));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * ct;
          if (__any_sync(RQ_FULL_MASK, mt > m + kWeightTop) || (!LSE && tile_ev != ev)) {
            const float mn = mt > m + kWeightTop ? mt - kWeightHead : m;
            const float f = m == -INFINITY ? 0.f : ex2(m - mn);
            l *= f;
            m = mn;
            const float fo = f * power_of_two(tile_ev - ev);
            ev = tile_ev;
            if (!LSE && jt > 0) {
#pragma unroll 1
              for (int y = 0; y < D / 16; ++y) {
                uint32_t o[16];
                tc_ld16(tO + 16 * y, o);
                tc_wait_ld();
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * fo);
                tc_st16(tO + 16 * y, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : -m;
          const uint64_t c2 = pack2(ct, ct), m2 = pack2(ms, ms);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t p[32];
#pragma unroll
            for (int y = 0; y < 32; ++y) {
              const int k = half * 64 + 2 * y;
              float p0, p1;
              unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, m2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[y & 1] = add2(sum[y & 1], pack2(p0, p1));
              if (!LSE) p[y] = pack_half2(p0, p1);
            }
            if (!LSE) tc_st32(tS + 32 * half, p);
          }
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          if (!LSE) tc_wait_st();
          tc_fence_before();
          mbar_arrive(pready(i));
        }
        if (!failed && (!LSE || SCHED)) failed = !mbar_wait_bounded(done, seg & 1, kTcWaitLimitNs);
        failed = warpgroup_any(i, failed);                           // (the warps leave together: they share barriers)
        tc_fence_after();
      }
      // ---- store (a wait that gave up: NaN)
      const float nan = __int_as_float(0x7fc00000), down = power_of_two(-ev);
      const bool there = w.T > 0 && !failed;                         // O holds the segment's sums
      const int j = (row + x.first) / a.v.heads;
      const bool bad = !x.ok || flagged || failed || (valid && j >= a.v.first_bad[int64_t(x.b) * a.v.H + x.h]);
      if (LSE) {
        const int64_t tile = (int64_t(w.unit) * a.n_splits + blockIdx.x % a.n_splits) * a.row_tiles + w.r0 / kRows + i;
        if (valid) a.stats[tile * kRows + r] = bad ? make_float2(0.f, nan) : make_float2(m, l);
      } else if (!w.whole) {
        const int64_t tile = SCHED ? (2 * int64_t(blockIdx.x) + (w.at_begin ? 0 : 1)) * 2 + i
                                   : (int64_t(w.unit) * a.n_splits + blockIdx.x % a.n_splits) * a.row_tiles + w.r0 / kRows + i;
        a.stats[tile * kRows + r] = bad ? make_float2(0.f, nan) : make_float2(m, l);
        constexpr int HALF = D / 2;                                  // channels that fit the image at a time
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int y = 0; y < HALF / 32; ++y) {
            uint32_t o[32];
#pragma unroll
            for (int z = 0; z < 32; ++z) o[z] = 0u;
            if (there) {
              tc_ld32(tO + half * HALF + 32 * y, o);
              tc_wait_ld();
            }
#pragma unroll
            for (int z = 0; z < 8; ++z)
              *reinterpret_cast<uint4*>(img + o_image_offset<HALF>(r, 8 * y + z)) =
                  make_uint4(times(o[4 * z], down), times(o[4 * z + 1], down), times(o[4 * z + 2], down),
                             times(o[4 * z + 3], down));
          }
          fence_async_smem();
          warpgroup_barrier(i);
          if (r == 0) {
            bulk_s2g(a.part + (tile * 2 + half) * (kRows * HALF), smem_u32(img), kRows * HALF * 4);
            bulk_s2g_commit();
            bulk_s2g_wait_read();                                    // (the image may be written again)
          }
          warpgroup_barrier(i);
        }
      } else {
        constexpr int CR = D / 8;                                    // 16-byte chunks of a row of bf16
        const float inv = bad ? nan : down / l;
#pragma unroll 1
        for (int y = 0; y < D / 32; ++y) {
          uint32_t o[32];
#pragma unroll
          for (int z = 0; z < 32; ++z) o[z] = 0u;
          if (there) {
            tc_ld32(tO + 32 * y, o);
            tc_wait_ld();
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            uint32_t p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(o[8 * z + 2 * k]) * inv,
                                                            __uint_as_float(o[8 * z + 2 * k + 1]) * inv);
              p[k] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(img + r * (D * 2) + (((4 * y + z) ^ (r & (CR - 1))) << 4)) =
                make_uint4(p[0], p[1], p[2], p[3]);
          }
        }
        __syncwarp();
        const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll 4
        for (int k = lane; k < 32 * CR; k += 32) {                   // this warp's rows, 16 bytes a lane
          const int rr = (warp & 3) * 32 + k / CR, cc = k % CR, y = w.r0 + i * kRows + rr;
          if (y >= x.rows) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(img + rr * (D * 2) + ((cc ^ (rr & (CR - 1))) << 4));
          uint16_t* const o = a.out + ((int64_t(x.b) * a.v.n_new + y / a.v.heads) * a.v.H * a.v.heads +
                                       x.h * a.v.heads + y % a.v.heads) * D + 8 * cc;
          if (vec) {
            *reinterpret_cast<uint4*>(o) = v;
          } else {
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[2 * e] = uint16_t(q[e]);
              o[2 * e + 1] = uint16_t(q[e] >> 16);
            }
          }
        }
        __syncwarp();                                                // (the next queries overwrite the rows)
      }
      tc_fence_before();
    }
    if (r == 0) bulk_s2g_wait();
  }
  if (__syncthreads_or(failed) && threadIdx.x == 0) atomicOr(a.v.err, 1u);
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tc_free(tmem, 512);
}

// The row blocks that several CTAs share: 8 CTAs of 32 rows for each row block and unit (SCHED: for
// each cut, the first one inside a row block acts), a warp for four rows at a time.  Bound by HBM
// latency: a few dependent loads per warp (15 us after the 325 us above).
template <int D, bool SCHED>
__global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ AttnArgs a) {
  grid_wait();
  grid_next();
  constexpr int P = D / 32, HALF = D / 2;
  const int lane = threadIdx.x & 31;
  int p = blockIdx.x, from = 0, to = a.n_splits, start = 0, stop = 1;
  const int c = SCHED ? int(blockIdx.x) + 1 : 1;             // CTAs (splits) c - 1 .. have parts
  if constexpr (SCHED) {
    const int2 cut = a.schedule.cut[c];
    p = cut.y;
    start = a.schedule.cut[c - 1].x;
    stop = cut.x;
    from = a.schedule.at[p];
    to = a.schedule.at[p + 1];
    if (stop <= from || stop >= to || start > from) return;
  }
  const int unit = p % a.units, block = a.blocks - 1 - p / a.units;
  const BlockInfo info = block_info(a.v, unit, block, false);
  const bool flagged = *reinterpret_cast<volatile unsigned*>(a.v.err) != 0u;
  const int local = blockIdx.y * 32 + (threadIdx.x >> 5) * 4;        // four rows
  const int i = local / kRows;
  if (block * 2 * kRows + local >= info.rows) return;
  float M[4], l[4], o[4][P];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    M[k] = -INFINITY;
    l[k] = 0.f;
#pragma unroll
    for (int e = 0; e < P; ++e) o[k][e] = 0.f;
  }
  // CTA s has [start, stop) of the line
  for (int s = c - 1; start < to; ++s, start = stop, stop = !SCHED ? s + 1 : start < to ? a.schedule.cut[s + 1].x : start) {
    const int64_t tile = SCHED ? (2 * int64_t(s) + (start >= from ? 0 : 1)) * 2 + i
                               : (int64_t(unit) * a.n_splits + s) * a.row_tiles + block * 2 + i;
    // lane's channels P lane ..: in the half-row image lane / 16
    const uint8_t* img = reinterpret_cast<const uint8_t*>(a.part + (tile * 2 + lane / 16) * (kRows * HALF));
    const int byte = (lane % 16) * P * 4;
    float2 st[4];
    float v[4][P];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = (local + k) % kRows;
      st[k] = a.stats[tile * kRows + r];
      const uint8_t* src = img + o_image_offset<HALF>(r, byte / 16) + byte % 16;
      if constexpr (P == 4) {
        const float4 y = *reinterpret_cast<const float4*>(src);
        v[k][0] = y.x, v[k][1] = y.y, v[k][2] = y.z, v[k][3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(src);
        v[k][0] = y.x, v[k][1] = y.y;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (st[k].x == -INFINITY) continue;
      const float m = fmaxf(M[k], st[k].x), f0 = ex2(M[k] - m), f = ex2(st[k].x - m);
      M[k] = m;
      l[k] = fmaf(l[k], f0, f * st[k].y);
#pragma unroll
      for (int e = 0; e < P; ++e) o[k][e] = fmaf(o[k][e], f0, f * v[k][e]);
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = block * 2 * kRows + local + k;
    if (row >= info.rows) break;
    const int j = row / a.v.heads, g = row % a.v.heads;
    uint16_t* out = a.out + ((int64_t(info.b) * a.v.n_new + j) * a.v.H * a.v.heads + info.h * a.v.heads + g) * D + lane * P;
    const float inv = flagged ? __int_as_float(0x7fc00000) : 1.f / l[k];
#pragma unroll
    for (int e = 0; e < P; ++e) out[e] = float_to_bf16_bits(o[k][e] * inv);
  }
}

// ---------------------------------------------------------------------------------- weights

struct WeightArgs {
  ChunkView v;
  const uint16_t* q;
  int64_t qs0, qs1, qs2;
  int qvec;
  const uint8_t *k, *klo;
  uint8_t* qimg;           // [unit][row tile][image of 128 rows]
  float2* scale;           // [unit][row]: (score scale, -log2-sum-exp); (0, -inf): no row
  const float2* stats;     // [unit][split][padded row]
  float* weights;
  int n_splits, q_tiles, cap;
  float scale_log2;
};

// Operand images of the window's queries, each row's score scale and log2-sum-exp.  Bound by latency.
template <int D>
__global__ void __launch_bounds__(128) window_rows_kernel(const __grid_constant__ WeightArgs a) {
  grid_wait();
  grid_next();
  extern __shared__ __align__(1024) uint8_t img[];
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
  int n, ctx;
  if (!lens_of(a.v, b, n, ctx)) return;
  const int first = max(0, n - a.v.window) * a.v.heads, rows = n * a.v.heads - first;
  const int row = blockIdx.x * kRows + threadIdx.x;
  if (int(blockIdx.x) * kRows >= rows) return;
  __shared__ int exps[kRows];
  store_queries<D>(
      [&](int rr) -> const uint16_t* {
        const int x = int(blockIdx.x) * kRows + rr;
        if (x >= rows) return nullptr;
        const int j = (x + first) / a.v.heads, g = (x + first) % a.v.heads;
        return a.q + b * a.qs0 + j * a.qs1 + (int64_t(h) * a.v.heads + g) * a.qs2;
      },
      a.qvec, img, exps, (threadIdx.x >> 5) * 32, threadIdx.x & 31);
  float2 sc = make_float2(0.f, -INFINITY);
  if (row < rows) {
    const float2* st = a.stats + unit * a.n_splits * (int64_t(a.q_tiles) * kRows) + row;
    const int64_t step = int64_t(a.q_tiles) * kRows;
    float M = -INFINITY, l = 0.f;
    for (int s = 0; s < a.n_splits; ++s) M = fmaxf(M, st[s * step].x);
    for (int s = 0; s < a.n_splits; ++s) {
      const float2 x = st[s * step];
      if (x.x != -INFINITY) l = fmaf(ex2(x.x - M), x.y, l);
    }
    sc = make_float2(ldexpf(a.scale_log2, -exps[threadIdx.x]), -(M + log2f(l)));
  }
  a.scale[unit * (int64_t(a.q_tiles) * kRows) + row] = sc;
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(a.qimg + (unit * a.q_tiles + blockIdx.x) * (kRows * D * 2));
  for (int i = threadIdx.x; i < kRows * D * 2 / 16; i += 128) dst[i] = reinterpret_cast<const uint4*>(img)[i];
}

template <int D>
struct WeightSmem {
  static constexpr int kTileBytes = kKeys * D * 2;
  static constexpr int kStages = 1;                       // (two CTAs per SM)
  static constexpr int kStage = kTileBytes + kRows * 8;   // queries, scales
  static constexpr int k = 0, q = 2 * kTileBytes, bars = q + kStages * kStage;
  static constexpr int total = bars + 256 + 1024;
};

// One CTA per 128 keys: S^T = K Q^T with the keys as rows, so a key's weights add up in its
// thread's registers, in row order.  Row tiles alternate between two tensor-memory buffers and the
// two softmax warpgroups.  With few rows (one row tile per CTA) bound by the latency of its steps,
// copies, products, exponentials, which two CTAs per SM overlap (32 rows, 6,509 keys, 32 heads: 34 us);
// with many by the exponentials.
template <int D>
__global__ void __launch_bounds__(320, 2) weights_kernel(const __grid_constant__ WeightArgs a) {
  grid_wait();
  grid_next();
  extern __shared__ uint8_t raw[];
  using L = WeightSmem<D>;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  const uint32_t bar0 = smem_u32(bars);
  auto qfull = [&](int s) { return bar0 + 8 * s; };
  auto qfree = [&](int s) { return bar0 + 8 * (3 + s); };
  auto sready = [&](int i) { return bar0 + 8 * (6 + i); };
  auto sfree = [&](int i) { return bar0 + 8 * (8 + i); };
  const uint32_t kfull = bar0 + 8 * 10, done = bar0 + 8 * 11;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 12);
  __shared__ float other[kKeys];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
  int n, ctx;
  if (!lens_of(a.v, b, n, ctx) || n == 0) return;
  const int key0 = blockIdx.x * kKeys;
  if (key0 >= ctx + n) return;
  const int j0 = max(0, n - a.v.window);                 // first token of the window
  const int rows = (n - j0) * a.v.heads;
  // row tiles that see any of these keys
  const int from = max(0, key0 - ctx - j0) * a.v.heads / kRows, to = (rows + kRows - 1) / kRows;
  const int T = to - from;
  if (warp == 9) tc_alloc(smem_u32(tslot), 256);
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(qfull(i), 1);
      mbar_init(qfree(i), kRows + 1);                    // the products, and the scales' readers
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sready(i), 1);
      mbar_init(sfree(i), kRows);
    }
    mbar_init(kfull, 1);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool failed = false;
  float w = 0.f;
  if (warp == 8) {
    if (lane == 0) {
      const int64_t at = (unit * a.v.tiles + blockIdx.x) * L::kTileBytes;
      mbar_arrive_expect_tx(kfull, 2 * L::kTileBytes);
      bulk_g2s(smem_u32(smem + L::k), a.k + at, L::kTileBytes, kfull);
      bulk_g2s(smem_u32(smem + L::k + L::kTileBytes), a.klo + at, L::kTileBytes, kfull);
      int issued = 0;
      for (int j = 0; j < T; ++j, ++issued) {
        const int s = j % L::kStages;
        if (j >= L::kStages && !mbar_wait_bounded(qfree(s), (j / L::kStages - 1) & 1, kTcWaitLimitNs)) break;
        const uint32_t dst = smem_u32(smem + L::q + s * L::kStage);
        mbar_arrive_expect_tx(qfull(s), L::kStage);
        bulk_g2s(dst, a.qimg + (unit * a.q_tiles + from + j) * L::kTileBytes, L::kTileBytes, qfull(s));
        bulk_g2s(dst + L::kTileBytes, a.scale + (unit * a.q_tiles + from + j) * kRows, kRows * 8, qfull(s));
      }
      failed = issued < T || !mbar_wait_bounded(kfull, 0, kTcWaitLimitNs);
      for (int j = max(0, issued - L::kStages); j < issued; ++j) {
        failed |= !mbar_wait_bounded(qfull(j % L::kStages), (j / L::kStages) & 1, kTcWaitLimitNs);
        // (and no arrival outstanding when the CTA leaves)
        failed = failed || !mbar_wait_bounded(qfree(j % L::kStages), (j / L::kStages) & 1, kTcWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    if (elect_one()) {
      constexpr uint32_t id = f16_idesc(kKeys, kRows);
      bool good = mbar_wait_bounded(kfull, 0, kTcWaitLimitNs);
      for (int j = 0; j < T && good; ++j) {
        const int s = j % L::kStages, i = j & 1;
        good = mbar_wait_bounded(qfull(s), (j / L::kStages) & 1, kTcWaitLimitNs) &&
               (j < 2 || mbar_wait_bounded(sfree(i), ((j >> 1) - 1) & 1, kTcWaitLimitNs));
        if (!good) break;
        tc_fence_after();
        const uint32_t q = smem_u32(smem + L::q + s * L::kStage);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t k = smem_u32(smem + L::k + part * L::kTileBytes);
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            tc_mma(tmem + 128 * i, panel_desc(k + (x / 4) * (kKeys * 128) + (x % 4) * 32),
                   panel_desc(q + (x / 4) * (kRows * 128) + (x % 4) * 32), id, part > 0 || x > 0);
        }
        tc_commit(sready(i));
        tc_commit(qfree(s));
      }
      tc_commit(done);
      failed = !good | !mbar_wait_bounded(done, 0, kTcWaitLimitNs);
    }
    __syncwarp();
  } else {
    const int i = warp >> 2, key = key0 + (threadIdx.x & (kKeys - 1));
    const uint32_t lanes = uint32_t(warp & 3) << 21;
    // rows before this one do not see the key
    const int row_min = max(0, key - ctx - j0) * a.v.heads;
    const float down = power_of_two(-(a.v.exps[unit * a.v.tiles + blockIdx.x] & 255));
    for (int j = i; j < T; j += 2) {
      const int s = j % L::kStages;
      const bool good = mbar_wait_bounded(sready(i), (j >> 1) & 1, kTcWaitLimitNs) &&
                        mbar_wait_bounded(qfull(s), (j / L::kStages) & 1, kTcWaitLimitNs);
      if (__any_sync(RQ_FULL_MASK, !good)) {                          // (the warp leaves as one)
        failed = true;
        break;
      }
      tc_fence_after();
      const float4* sc = reinterpret_cast<const float4*>(smem + L::q + s * L::kStage + L::kTileBytes);
      const int rel = row_min - (from + j) * kRows;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t v[32];
        tc_ld32(tmem + 128 * i + lanes + 32 * x, v);
        tc_wait_ld();
#pragma unroll
        for (int y = 0; y < 32; y += 2) {
          const float4 f = sc[(32 * x + y) / 2];
          const float p0 = ex2(fmaf(__uint_as_float(v[y]) * down, f.x, f.y));
          const float p1 = ex2(fmaf(__uint_as_float(v[y + 1]) * down, f.z, f.w));
          sum[0] += 32 * x + y >= rel ? p0 : 0.f;
          sum[1] += 32 * x + y + 1 >= rel ? p1 : 0.f;
        }
      }
      w += sum[0] + sum[1];
      tc_fence_before();
      mbar_arrive(sfree(i));
      mbar_arrive(qfree(s));
    }
    if (i == 1) other[threadIdx.x & (kKeys - 1)] = w;
  }
  const bool gave_up = __syncthreads_or(failed);
  if (gave_up && threadIdx.x == 0) atomicOr(a.v.err, 1u);
  if (warp < 4) {
    const int key = key0 + threadIdx.x;
    if (key < ctx + n && key < a.cap && !gave_up)
      a.weights[(int64_t(b) * a.v.H + h) * a.cap + key] += w + other[threadIdx.x];
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tc_free(tmem, 256);
}

// ------------------------------------------------------------------------------------- host

size_t round1k(size_t n) { return (n + 1023) / 1024 * 1024; }

constexpr size_t kGroupBytes = size_t(4) << 30;   // images of the sequences handled together

struct TcLayout {
  int group;               // sequences handled together
  int tiles, blocks, r_tiles, wblocks, q_tiles, splits, wsplits, ctas;   // ctas: of the scheduled attention, or 0
  size_t first_bad, exps, schedule, k, klo, val, part, stats, qimg, scale, total;
};

constexpr int kMaxPairs = 8192;   // scheduled row blocks, at most: more keep every SM busy as they are
constexpr int kMinShare = 64;     // key tiles per CTA from which they are shared evenly

// Splits of the keys so that the CTAs (one per SM) come in few, even waves: least
// waves x (tiles per split + set-up), the set-up worth about two tiles.
int plan_tc_splits(int64_t ctas, int tiles) {
  const int64_t sms = device_sm_count();
  double best = 1e300;
  int found = 1;
  for (int s = 1; s <= tiles && s <= 64; ++s) {
    const int64_t waves = (ctas * s + sms - 1) / sms;
    const double cost = double(waves) * ((tiles + s - 1) / s + 2.0 + (s > 1 ? 0.5 : 0.0));
    if (cost < best - 1e-9) {
      best = cost;
      found = s;
    }
  }
  return found;
}

// most: sequences handled together, at most; lean: no key tiles shared between CTAs.
TcLayout tc_layout_of(const rq_shape& s, int n_new, int max_ctx, int window, int most, bool lean) {
  TcLayout l;
  const int heads = s.n_q_heads / s.n_kv_heads, D = s.head_dim;
  l.tiles = int((int64_t(max_ctx) + n_new + kKeys - 1) / kKeys);
  const int rows = n_new * heads, wrows = window * heads;
  l.blocks = (rows + 2 * kRows - 1) / (2 * kRows);
  l.wblocks = (wrows + 2 * kRows - 1) / (2 * kRows);
  l.q_tiles = (wrows + kRows - 1) / kRows;
  const size_t tile = size_t(kKeys) * D * 2;
  const size_t seq = size_t(s.n_kv_heads) * l.tiles * tile * (window ? 3 : 2);
  const size_t fit = kGroupBytes / (seq ? seq : 1);
  l.group = int(fit < 1 ? 1 : (fit > size_t(most) ? size_t(most) : fit));
  const size_t units = size_t(l.group) * s.n_kv_heads;
  const int64_t pairs = int64_t(units) * l.blocks;
  const int64_t work = pairs * l.tiles;
  l.ctas = !lean && pairs <= kMaxPairs && work >= int64_t(kMinShare) * device_sm_count() && work < (int64_t(1) << 29)
               ? device_sm_count() : 0;
  l.splits = l.ctas || lean ? 1 : plan_tc_splits(pairs, l.tiles);
  l.r_tiles = (rows + kRows - 1) / kRows;
  l.wsplits = window && !lean ? plan_tc_splits(int64_t(units) * l.wblocks, l.tiles) : 1;
  size_t o = kWsHeaderBytes;
  l.first_bad = o;
  o = round1k(o + size_t(s.batch) * s.n_kv_heads * 4);
  l.exps = o;
  o = round1k(o + units * l.tiles * 2);
  l.schedule = o;
  if (l.ctas) o = round1k(o + (size_t(l.ctas) + 1) * 8 + (size_t(pairs) + 1) * 4);
  l.k = o;
  o += units * l.tiles * tile;
  l.val = o;
  o += units * l.tiles * tile;
  l.klo = o;
  if (window) o += units * l.tiles * tile;
  // row tiles of shared blocks
  const size_t shared = l.ctas ? size_t(l.ctas) * 4 : l.splits > 1 ? units * l.splits * l.r_tiles : 0;
  l.part = o;
  o += shared * (size_t(kRows) * D * 4);
  l.stats = o;   // of the shared blocks, then of the window's rows
  const size_t wst = units * l.q_tiles * l.wsplits;
  o += (shared > wst ? shared : wst) * kRows * 8;
  l.qimg = o;
  o += units * l.q_tiles * (size_t(kRows) * D * 2);
  l.scale = o;
  o = round1k(o + units * l.q_tiles * kRows * 8);
  l.total = o;
  return l;
}

// The best plan within `budget`, else the smallest.
TcLayout tc_layout(const rq_shape& s, int n_new, int max_ctx, int window, size_t budget) {
  for (int most = s.batch;;) {
    for (bool lean : {false, true}) {
      const TcLayout l = tc_layout_of(s, n_new, max_ctx, window, most, lean);
      if (l.total <= budget || (lean && l.group == 1)) return l;
      if (lean) most = l.group / 2;
    }
  }
}

template <int D, int RES, bool KLO>
cudaError_t launch_rebuild(const RebuildArgs& r, int64_t items, bool after, cudaStream_t stream) {
  using L = RebuildSmem<D, RES, KLO>;
  static OncePerDevice once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(rebuild_kernel<D, RES, KLO>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
  });
  if (e != cudaSuccess) return e;
  if (items > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const int64_t ctas = int64_t(device_sm_count()) * 2;
  return launch_after(after, rebuild_kernel<D, RES, KLO>, unsigned(items < ctas ? items : ctas), 256, L::total, stream, r,
                      int(items));
}

template <int D>
cudaError_t launch_rebuild_any(const RebuildArgs& r, int64_t items, bool after, cudaStream_t stream) {
  if (r.bits == 0)
    return r.klo ? launch_rebuild<D, 0, true>(r, items, after, stream) : launch_rebuild<D, 0, false>(r, items, after, stream);
  if (r.bits == 2)
    return r.klo ? launch_rebuild<D, 2, true>(r, items, after, stream) : launch_rebuild<D, 2, false>(r, items, after, stream);
  return r.klo ? launch_rebuild<D, 4, true>(r, items, after, stream) : launch_rebuild<D, 4, false>(r, items, after, stream);
}

template <int D>
cudaError_t launch_tc(const rq_shape& s, const rq_cache& cache, const rq_paging* paging, const ChunkCall& c,
                      char* w, size_t ws_bytes, cudaStream_t stream) {
  const TcLayout l = tc_layout(s, c.n_new, c.max_ctx, c.window, ws_bytes);
  cudaError_t e;
  using AS = AttnSmem<D>;
  using WS = WeightSmem<D>;
  static OncePerDevice once;
  e = once([] {
    cudaError_t x;
    const cudaFuncAttribute smem = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if ((x = cudaFuncSetAttribute(chunk_image_kernel<D, true>, smem, 3 * kKeys * D * 2 + 128)) != cudaSuccess ||
        (x = cudaFuncSetAttribute(chunk_image_kernel<D, false>, smem, 2 * kKeys * D * 2 + 128)) != cudaSuccess ||
        (x = cudaFuncSetAttribute(attention_kernel<D, false, false>, smem, AS::total)) != cudaSuccess ||
        (x = cudaFuncSetAttribute(attention_kernel<D, false, true>, smem, AS::total)) != cudaSuccess ||
        (x = cudaFuncSetAttribute(attention_kernel<D, true, false>, smem, AS::total)) != cudaSuccess)
      return x;
    return cudaFuncSetAttribute(weights_kernel<D>, smem, WS::total);
  });
  if (e != cudaSuccess ||
      (e = cudaMemsetAsync(w + l.first_bad, 0x7f, size_t(s.batch) * s.n_kv_heads * 4, stream)) != cudaSuccess)
    return e;
  ChunkView v;
  v.n_lens = c.n_lens;
  v.ctx_lens = c.ctx_lens;
  v.err = reinterpret_cast<unsigned*>(w);
  v.first_bad = reinterpret_cast<int*>(w + l.first_bad);
  v.exps = reinterpret_cast<uint16_t*>(w + l.exps);
  v.H = s.n_kv_heads;
  v.heads = s.n_q_heads / s.n_kv_heads;
  v.n_new = c.n_new;
  v.max_ctx = c.max_ctx;
  v.window = c.window;
  v.tiles = l.tiles;
  const float scale = (s.softmax_scale > 0.f ? s.softmax_scale : 1.0f / sqrtf(float(s.head_dim))) * kLog2e;
  uint8_t* const wb = reinterpret_cast<uint8_t*>(w);
  const bool checked = l.group < s.batch;
  if (checked) {
    v.b0 = 0;
    const unsigned recs = paging ? unsigned((c.max_ctx + kTile - 1) / kTile) : 0u;
    check_kernel<<<dim3(recs / 256 + 1, unsigned(s.batch)), 256, 0, stream>>>(v, paging ? paging->block_table : nullptr,
                                                                              paging ? paging->max_pages : 0,
                                                                              paging ? paging->n_pages : 0);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  for (int b0 = 0; b0 < s.batch; b0 += l.group) {
    v.b0 = b0;
    const unsigned nb = unsigned(s.batch - b0 < l.group ? s.batch - b0 : l.group), H = unsigned(s.n_kv_heads);
    RebuildArgs r;
    r.v = v;
    r.data = cache.data;
    r.rec_bytes = record_bytes(s);
    r.bt = paging ? paging->block_table : nullptr;
    r.max_pages = paging ? paging->max_pages : 0;
    r.n_pages = paging ? paging->n_pages : 0;
    r.cap = s.capacity;
    r.bits = c.loop < s.n_loops - 1 ? s.res_bits[c.loop] : 0;
    r.sec_off = loop_section_offset(D, s.res_bits, c.loop);
    r.signs[0] = cache.rot_signs[0];
    r.signs[1] = cache.rot_signs[1];
    r.kv_new = c.kv_new + c.loop * c.kv_strides[3];
    r.ks0 = c.kv_strides[0];
    r.ks1 = c.kv_strides[1];
    r.kv_v = c.kv_strides[2];
    r.ks_h = c.kv_strides[4];
    r.k = wb + l.k;
    r.klo = c.window ? wb + l.klo : nullptr;
    r.val = wb + l.val;
    r.vec = reinterpret_cast<uintptr_t>(r.kv_new) % 16 == 0 && r.ks0 % 8 == 0 && r.ks1 % 8 == 0 &&
            r.kv_v % 8 == 0 && r.ks_h % 8 == 0;
    r.old_tiles = (c.max_ctx + kKeys - 1) / kKeys;
    if (c.max_ctx > 0 && (e = launch_rebuild_any<D>(r, int64_t(nb) * H * r.old_tiles, checked || b0 > 0, stream)) != cudaSuccess) return e;
    r.units = int(nb * H);
    r.blocks = l.blocks;
    r.schedule.pairs = r.units * r.blocks;
    r.schedule.grid = l.ctas;
    r.schedule.cut = reinterpret_cast<int2*>(w + l.schedule);
    r.schedule.at = l.ctas ? reinterpret_cast<int*>(w + l.schedule + (size_t(l.ctas) + 1) * 8) : nullptr;
    const dim3 own(unsigned((c.n_new + kKeys - 1) / kKeys) * H + 1, 1, nb);
    e = launch_after(checked || b0 > 0 || c.max_ctx > 0, c.window ? chunk_image_kernel<D, true> : chunk_image_kernel<D, false>, own, 256,
                     (c.window ? 3 : 2) * kKeys * D * 2 + 128, stream, r);
    if (e != cudaSuccess) return e;
    AttnArgs a;
    a.v = v;
    a.q = c.q;
    a.qs0 = c.q_strides[0];
    a.qs1 = c.q_strides[1];
    a.qs2 = c.q_strides[2];
    a.k = r.k;
    a.klo = r.klo;
    a.val = r.val;
    a.out = c.out;
    a.schedule = r.schedule;
    a.part = reinterpret_cast<float*>(w + l.part);
    a.stats = reinterpret_cast<float2*>(w + l.stats);
    a.n_splits = l.splits;
    a.row_tiles = l.r_tiles;
    a.units = r.units;
    a.blocks = l.blocks;
    a.qvec = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && a.qs0 % 8 == 0 && a.qs1 % 8 == 0 && a.qs2 % 8 == 0;
    a.scale_log2 = scale;
    if (l.ctas) {
      e = launch_after(true, attention_kernel<D, false, true>, unsigned(l.ctas), 384, AS::total, stream, a);
      if (e == cudaSuccess && l.ctas > 1)
        e = launch_after(true, merge_kernel<D, true>, dim3(unsigned(l.ctas - 1), 2 * kRows / 32), 256, 0, stream, a);
    } else {
      e = launch_after(true, attention_kernel<D, false, false>, dim3(nb * H * l.splits, unsigned(l.blocks)), 384, AS::total,
                       stream, a);
      if (e == cudaSuccess && l.splits > 1)
        e = launch_after(true, merge_kernel<D, false>, dim3(nb * H * l.blocks, 2 * kRows / 32), 256, 0, stream, a);
    }
    if (e != cudaSuccess) return e;
    if (!c.window) continue;
    a.n_splits = l.wsplits;
    a.row_tiles = l.q_tiles;
    a.blocks = l.wblocks;
    e = launch_after(true, attention_kernel<D, true, false>, dim3(nb * H * l.wsplits, unsigned(l.wblocks)), 384, AS::total,
                     stream, a);
    if (e != cudaSuccess) return e;
    WeightArgs x;
    x.v = v;
    x.q = c.q;
    x.qs0 = a.qs0;
    x.qs1 = a.qs1;
    x.qs2 = a.qs2;
    x.k = r.k;
    x.klo = r.klo;
    x.qimg = wb + l.qimg;
    x.scale = reinterpret_cast<float2*>(w + l.scale);
    x.stats = a.stats;
    x.weights = c.weights;
    x.n_splits = l.wsplits;
    x.qvec = a.qvec;
    x.q_tiles = l.q_tiles;
    x.cap = s.capacity;
    x.scale_log2 = scale;
    e = launch_after(true, window_rows_kernel<D>, dim3(unsigned(l.q_tiles), H, nb), kRows, kRows * D * 2, stream, x);
    if (e != cudaSuccess) return e;
    e = launch_after(true, weights_kernel<D>, dim3(unsigned(l.tiles), H, nb), 320, WS::total, stream, x);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t chunk_tc_workspace_bytes(const rq_shape& s, int n_new, int max_ctx, int window, size_t budget) {
  return tc_layout(s, n_new, max_ctx, window, budget).total;
}

cudaError_t launch_chunk_tc(const rq_shape& s, const rq_cache& cache, const rq_paging* paging,
                            const ChunkCall& c, void* ws, size_t ws_bytes, cudaStream_t stream) {
  char* const w = static_cast<char*>(ws);
  return s.head_dim == 128 ? launch_tc<128>(s, cache, paging, c, w, ws_bytes, stream)
                           : launch_tc<64>(s, cache, paging, c, w, ws_bytes, stream);
}

}  // namespace rq
