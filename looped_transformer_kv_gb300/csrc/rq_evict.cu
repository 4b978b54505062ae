// Eviction by accumulated attention weight: the slots to keep (rq_evict_select) and the move of
// their rows to the front of a cache (rq_evict_compact).
#include <cooperative_groups.h>

#include "rq_common.cuh"
#include "rq_kernels.h"

namespace cg = cooperative_groups;

namespace rq {
namespace {

// ------------------------------------------------------------------------------ select
//
// Weights become 32-bit keys of the same order.  A short row (at most 1024 slots): a slot's rank is
// counted directly, every key against every other.  A long one: the k-th largest key by radix
// selection.  Passes over the row count the keys' first 11 bits, the next 11 of those that share the
// k-th one's, and the last 10, as far as needed (a digit all of whose keys are kept ends it).  Then
// a pass counts and one writes, in slot order, every key above the k-th and, of its equals, the
// first ones.  A long row may be shared by a cluster of CTAs (each
// holds its part of the keys in shared memory, the counts are added over the cluster).
// Bytes: 4 per slot read once, 4 per kept slot written; what bounds it is the instructions of the
// passes (256 rows of up to 16,384 slots in 21 us, issue slots 64 % used), then their
// barriers.

constexpr int kSelThreads = 512;      // two CTAs per SM
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelMaxCluster = 8;
constexpr int kSelKeys = 48 * 1024;     // keys a CTA holds in shared memory, at most (192 KB)
constexpr int kShortRow = 1024;
constexpr uint32_t kHeld = 0xffffffffu; // key of a slot that is kept whatever its weight

// Same order as the weights; NaN above every number, -0 as +0; at least 2^21 (the key of -inf).
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xfffffffeu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

struct SelArgs {
  const float* weights;
  const int32_t* ctx_lens;
  int32_t* keep;
  int32_t* kept_lens;
  int H, cap, budget, n_first, n_last, slice;   // slice: keys of shared memory, 0: none
};

// Exclusive scan of one value per thread over the block (WARPS warps); total: the sum.
template <int WARPS>
__device__ __forceinline__ int block_exclusive_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(RQ_FULL_MASK, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = lane < WARPS ? warp_sums[lane] : 0, before = lane < warp ? s : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(RQ_FULL_MASK, s, o);
    before += __shfl_xor_sync(RQ_FULL_MASK, before, o);
  }
  total = s;
  __syncthreads();
  return before + x - v;
}

// A row of at most kShortRow slots per CTA of kShortRow / 4 threads: 4 consecutive slots a thread.
__global__ void __launch_bounds__(kShortRow / 4) evict_select_short_kernel(const __grid_constant__ SelArgs a) {
  const int bh = blockIdx.x, b = bh / a.H;
  const int n = a.ctx_lens[b];
  __shared__ __align__(16) uint32_t keys[kShortRow];
  __shared__ int warp_sums[32];
  const bool bad = n < 0 || n > a.cap;
  const int k = bad ? -1 : min(n, a.budget);
  if (bh % a.H == 0 && threadIdx.x == 0) a.kept_lens[b] = k;
  if (bad) return;
  int32_t* const out = a.keep + int64_t(bh) * a.budget;
  const float* const row = a.weights + int64_t(bh) * a.cap;
  const int t0 = threadIdx.x * 4;
  uint32_t mine[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i;
    mine[i] = t >= n ? 0u : (t < a.n_first || t >= n - a.n_last) ? kHeld : weight_key(row[t]);
  }
  *reinterpret_cast<uint4*>(keys + t0) = make_uint4(mine[0], mine[1], mine[2], mine[3]);
  __syncthreads();
  int rank[4] = {0, 0, 0, 0};           // keys above, and equal ones before
  for (int u = 0; u < (n + 3) / 4; ++u) {   // (slots behind n have key 0, below every other)
    const uint4 o = *reinterpret_cast<const uint4*>(keys + 4 * u);
    const uint32_t ok[4] = {o.x, o.y, o.z, o.w};
    const uint32_t eq = 4 * u < t0 ? 1u : 0u;   // earlier groups: an equal key counts as above
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) rank[i] += ok[e] > mine[i] - eq ? 1 : 0;
  }
#pragma unroll
  for (int i = 1; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < i; ++e) rank[i] += mine[e] == mine[i] ? 1 : 0;
  int c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) c += t0 + i < n && rank[i] < k ? 1 : 0;
  int total;
  int at = block_exclusive_scan<kShortRow / 128>(c, warp_sums, total);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (t0 + i < n && rank[i] < k) out[at++] = t0 + i;
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ SelArgs a) {
  cg::cluster_group cluster = cg::this_cluster();
  const int C = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int bh = blockIdx.x / C, b = bh / a.H;
  const int n = a.ctx_lens[b];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  extern __shared__ uint32_t keys[];
  __shared__ int hist[kBins];
  __shared__ int warp_sums[32];
  __shared__ int found[3], counts[2];     // (digit, rank among its keys, its keys); (kept, equal) of this CTA
  const bool bad = n < 0 || n > a.cap;
  const int k = bad ? -1 : min(n, a.budget);
  if (rank == 0 && bh % a.H == 0 && threadIdx.x == 0) a.kept_lens[b] = k;
  if (bad) return;                        // (the same for the whole cluster)
  int32_t* const out = a.keep + int64_t(bh) * a.budget;
  if (n <= a.budget) {                    // everything stays
    for (int t = rank * kSelThreads + threadIdx.x; t < n; t += C * kSelThreads) out[t] = t;
    return;
  }
  auto sync_all = [&]() {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  // this CTA's slots [t0, t1), a warp's [w0, w1): a multiple of 32 each
  const int per_warp = ((n + C * kSelWarps - 1) / (C * kSelWarps) + 31) / 32 * 32;
  const int t0 = min(n, rank * kSelWarps * per_warp), t1 = min(n, t0 + kSelWarps * per_warp);
  const int w0 = min(n, t0 + warp * per_warp), w1 = min(t1, w0 + per_warp);
  const float* const row = a.weights + int64_t(bh) * a.cap;
  const int held_from = n - a.n_last;
  const bool stored = t1 - t0 <= a.slice;
  // keys of slots base + 32 u + lane, U of them in flight; 0 behind the warp's slots
  constexpr int U = 8;
  auto fresh_keys = [&](int base, uint32_t (&key)[U]) {
    float w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) w[u] = row[min(base + 32 * u + lane, w1 - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) key[u] = base + 32 * u + lane < w1 ? weight_key(w[u]) : 0u;
    if (base < a.n_first || base + 32 * U > held_from) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = base + 32 * u + lane;
        if (t < w1 && (t < a.n_first || t >= held_from)) key[u] = kHeld;
      }
    }
  };
  auto load_keys = [&](int base, uint32_t (&key)[U]) {
    if (stored) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int t = base + 32 * u + lane;
        key[u] = t < w1 ? keys[t - t0] : 0u;
      }
    } else {
      fresh_keys(base, key);
    }
  };
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  // the first digits of every key (held keys are above every other: they count too)
  for (int base = w0; base < w1; base += 32 * U) {
    uint32_t key[U];
    fresh_keys(base, key);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = base + 32 * u + lane;
      if (t < w1) {
        if (stored) keys[t - t0] = key[u];
        atomicAdd(&hist[key[u] >> 21], 1);
      }
    }
  }
  uint32_t prefix = 0;                    // the k-th key's digits so far
  int need = k, bits = 0;                 // its rank among the keys that match them; their number
  for (int pass = 0;; ++pass) {
    sync_all();
    // counts of the cluster, a few digits per thread, from the highest down
    constexpr int PT = kBins / kSelThreads;
    int c[PT], sum = 0;
    const int top = kBins - 1 - PT * int(threadIdx.x);
#pragma unroll
    for (int i = 0; i < PT; ++i) c[i] = 0;
    for (int r = 0; r < C; ++r) {
      const int* const hr = C > 1 ? cluster.map_shared_rank(hist, r) : hist;
#pragma unroll
      for (int i = 0; i < PT; ++i) c[i] += hr[top - i];
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) sum += c[i];
    int total;
    int above = block_exclusive_scan<kSelWarps>(sum, warp_sums, total);
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      if (above < need && need <= above + c[i]) {
        found[0] = top - i;
        found[1] = need - above;
        found[2] = c[i];
      }
      above += c[i];
    }
    __syncthreads();
    const int width = pass == 2 ? 10 : 11;
    prefix = (prefix << width) | uint32_t(found[0]);
    bits += width;
    need = found[1];
    const int match = found[2];
    if (C > 1) cluster.sync();            // the counts have been read by everyone
    if (match == need || bits == 32) break;   // every match is kept, or they are equal
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const int next = bits == 11 ? 10 : 0;     // the next digit's lowest bit
    const uint32_t mask = bits == 11 ? 2047u : 1023u;
    for (int base = w0; base < w1; base += 32 * U) {
      uint32_t key[U];
      load_keys(base, key);
#pragma unroll
      for (int u = 0; u < U; ++u)         // (a slot behind the row has key 0, no key's digits)
        if (key[u] >> (32 - bits) == prefix) atomicAdd(&hist[(key[u] >> next) & mask], 1);
    }
  }
  // keys above `high` are kept, and the first `need` slots of low .. high
  const uint32_t low = bits == 32 ? prefix : prefix << (32 - bits);
  const uint32_t high = bits == 32 ? prefix : low | ((1u << (32 - bits)) - 1u);
  int kept = 0, equal = 0;
  for (int base = w0; base < w1; base += 32 * U) {
    uint32_t key[U];
    load_keys(base, key);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kept += key[u] > high ? 1 : 0;
      equal += key[u] >= low ? 1 : 0;
    }
  }
  equal -= kept;
  int kept_all, equal_all;
  const int kept_before = block_exclusive_scan<kSelWarps>(kept, warp_sums, kept_all);
  const int equal_before = block_exclusive_scan<kSelWarps>(equal, warp_sums, equal_all);
  if (threadIdx.x == 0) {
    counts[0] = kept_all;
    counts[1] = equal_all;
  }
  sync_all();
  int A = __shfl_sync(RQ_FULL_MASK, kept_before, 0), E = __shfl_sync(RQ_FULL_MASK, equal_before, 0);
  for (int r = 0; r < rank; ++r) {
    A += cluster.map_shared_rank(counts, r)[0];
    E += cluster.map_shared_rank(counts, r)[1];
  }
  const unsigned lower = (1u << lane) - 1u;
  for (int base = w0; base < w1; base += 32 * U) {
    uint32_t key[U];
    load_keys(base, key);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool above = key[u] > high, among = key[u] >= low && !above;
      const unsigned ma = __ballot_sync(RQ_FULL_MASK, above), me = __ballot_sync(RQ_FULL_MASK, among);
      const int e_here = E + __popc(me & lower);
      if (above || (among && e_here < need)) out[A + __popc(ma & lower) + min(e_here, need)] = base + 32 * u + lane;
      A += __popc(ma);
      E += __popc(me);
    }
  }
  if (C > 1) cluster.sync();   // (no CTA leaves while its counts may be read)
}

// ------------------------------------------------------------------------------ compact
//
// A 64-row tile of one section of `to` is made of units of at most 16 bytes; a thread loads the
// sources of its units into registers and stores them.  K rows, steps and offsets are contiguous
// per row; V code words hold two tokens, so a unit (4 words of a pair) takes the matching
// 16-bit halves of two source pairs.  V codes of a kept token whose pair neighbour is not kept cost
// twice their bytes, steps and offsets a whole 32-byte sector: 2,048 of up to 4,096 rows, 256 heads, 3
// residual loops: 488 MB wanted, 575 MB moved, in 119 us.  Neither wall is reached: 4.8 TB/s is 71 % of a
// plain copy's rate, and the address arithmetic of the 16-byte gathers uses 67 % of the issue slots.
// In place, 150 us for the same rows (128 out of place, timed alike); paged 160 and 132.
// In place, a row only moves to a lower slot.  A cluster of CTAs takes the tiles of one (sequence,
// kv-head, section) in ascending waves: all rows of a wave are read before any is written
// (cluster barrier), and later waves read only rows at or above their own tiles.

constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 3;      // units of a section's tile per thread, at most (768 / 256)
constexpr int kMoveCluster = 8;

struct MoveArgs {
  const uint8_t* src;
  uint8_t* dst;
  int64_t rec_bytes;
  const int32_t* src_bt;
  const int32_t* dst_bt;
  int src_max_pages, src_n_pages, dst_max_pages, dst_n_pages;
  const int32_t* keep;
  const int32_t* kept_lens;
  const float* weights;
  float* to_weights;
  int H, L, budget, src_cap, dst_cap, ctas;   // ctas: per (sequence, kv-head), out of place
  int8_t res_bits[RQ_MAX_LOOPS];
};

// One unit: what it is and where it starts within the section.
struct Unit {
  int off;        // byte offset of the unit in a tile's section (K-like kinds: of row 0)
  int row;        // row, or first row of the pair
  int bytes;      // 16, 8 or 2; 0: no unit
  int row_bytes;
  int chunk;      // K codes: 16-byte chunk of the row; V codes: group of 4 units
  bool v_codes;
};

// KIND: 0 the reference section, else a residual section of that many bits.
template <int D, int KIND>
__device__ __forceinline__ Unit unit_of(int i) {
  constexpr int NG = D / 32;
  constexpr bool residual = KIND != 0;
  constexpr int rb = D * (residual ? KIND : 4) / 8, chunks = rb / 16;
  constexpr int nc = kTile * chunks, per = nc + kTile + (residual ? kTile : 0);
  constexpr int side = kTile * (rb + NG * 4 + (residual ? 2 : 0));
  Unit u;
  u.v_codes = false;
  const bool v = i >= per;
  if (v) i -= per;
  const int base = v ? side : 0;
  u.bytes = 0;
  if (i >= per) return u;
  if (i < nc) {
    u.bytes = 16;
    u.off = base;
    u.chunk = i % chunks;
    if (v) {   // a pair's words: 2 rb bytes, `chunks` * 2 units of 16 bytes
      u.v_codes = true;
      u.chunk = i % (2 * chunks);
      u.row = i / (2 * chunks) * 2;
    } else {
      u.row = i / chunks;
    }
    u.row_bytes = rb;
  } else if (i < nc + kTile) {
    u.row = i - nc;
    u.chunk = 0;
    u.off = base + kTile * rb;
    u.row_bytes = u.bytes = NG * 4;
  } else {
    u.row = i - nc - kTile;
    u.chunk = 0;
    u.off = base + kTile * (rb + NG * 4);
    u.row_bytes = u.bytes = 2;
  }
  return u;
}

template <int D, bool IN_PLACE, int KIND>
__device__ __forceinline__ void move_section(const MoveArgs& a, int sect) {
  const int step = IN_PLACE ? kMoveCluster : a.ctas;        // CTAs of a (sequence, kv-head): tile step
  const int64_t bh = blockIdx.x / step;
  const int first_tile = blockIdx.x % step;
  const int b = int(bh / a.H), h = int(bh % a.H);
  const int kept = max(0, min(a.kept_lens[b], min(a.budget, a.dst_cap)));
  const int n_tiles = (kept + kTile - 1) / kTile;
  const int sec_off = sect == 0 ? 0 : loop_section_offset(D, a.res_bits, sect - 1);
  const int32_t* const keep = a.keep + bh * a.budget;
  const bool moves_weights = a.weights && sect == 0;
  __shared__ int64_t from[2][kTile];                 // record offset of each row's source, -1: none
  __shared__ int from_row[2][kTile];

  // offset of the record of a tile, -1 where the block table has no page for it
  auto record = [&](int tile, const int32_t* bt, int max_pages, int n_pages, int cap) -> int64_t {
    int64_t rec;
    if (bt) {
      const int pg = bt[int64_t(b) * max_pages + tile];
      if (pg < 0 || pg >= n_pages) return -1;
      rec = int64_t(pg) * a.H + h;
    } else {
      rec = bh * (cap / kTile) + tile;
    }
    return rec * a.rec_bytes + sec_off;
  };
  auto slot_of = [&](int tile) {                     // this thread's row of the tile: its source, or -1
    const int t = tile * kTile + threadIdx.x;
    if (threadIdx.x >= kTile || tile >= n_tiles || t >= kept) return -1;
    const int s = keep[t];
    return s >= 0 && s < a.src_cap ? s : -1;
  };

  // (in place every CTA of the cluster takes every wave's barrier)
  const int waves = IN_PLACE ? (n_tiles + step - 1) / step : max(0, (n_tiles - first_tile + step - 1) / step);
  int slot = slot_of(first_tile);
  for (int wave = 0; wave < waves; ++wave) {
    const int tile = first_tile + wave * step, buf = wave & 1;
    const int64_t dst =
        tile < n_tiles ? record(tile, a.dst_bt, a.dst_max_pages, a.dst_n_pages, a.dst_cap) : -1;
    if (threadIdx.x < kTile) {
      from[buf][threadIdx.x] =
          slot < 0 ? -1 : record(slot / kTile, a.src_bt, a.src_max_pages, a.src_n_pages, a.src_cap);
      from_row[buf][threadIdx.x] = slot & (kTile - 1);
    }
    __syncthreads();
    float wt = 0.f;
    if (moves_weights && slot >= 0) wt = a.weights[bh * a.src_cap + slot];
    slot = slot_of(tile + step);                     // the next wave's, while this one moves
    uint4 v[kMoveUnits][2];
    int live[kMoveUnits];          // bit 0: the (first) row has a source, bit 1: the pair's second;
                                   // V codes: bits 2, 3: it is the odd token of its source pair
#pragma unroll
    for (int i = 0; i < kMoveUnits; ++i) {
      const Unit u = unit_of<D, KIND>(threadIdx.x + i * kMoveThreads);
      live[i] = 0;
      if (u.bytes == 0 || dst < 0) continue;
      if (!u.v_codes) {
        const int64_t f = from[buf][u.row];
        if (f < 0) continue;
        live[i] = 1;
        const uint8_t* p = a.src + f + u.off + from_row[buf][u.row] * u.row_bytes + u.chunk * 16;
        if (u.bytes == 16) {
          v[i][0] = *reinterpret_cast<const uint4*>(p);
        } else if (u.bytes == 8) {
          const uint2 x = *reinterpret_cast<const uint2*>(p);
          v[i][0].x = x.x;
          v[i][0].y = x.y;
        } else {
          v[i][0].x = *reinterpret_cast<const uint16_t*>(p);
        }
      } else {
        // units 4 chunk .. + 3 of each token sit in 4 adjacent words of its pair (the swizzle
        // moves whole groups of 8 units)
        const int units = u.row_bytes / 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          v[i][e] = make_uint4(0u, 0u, 0u, 0u);
          const int64_t f = from[buf][u.row + e];
          if (f < 0) continue;
          const int r = from_row[buf][u.row + e], pair = r >> 1;
          live[i] |= (1 | ((r & 1) << 2)) << e;
          v[i][e] = *reinterpret_cast<const uint4*>(a.src + f + u.off + pair * (2 * u.row_bytes) +
                                                    ((4 * u.chunk) ^ v_unit_swizzle(pair, units)) * 4);
        }
      }
    }
    if (IN_PLACE) cg::this_cluster().sync();   // every row of the wave is read
#pragma unroll
    for (int i = 0; i < kMoveUnits; ++i) {
      if (live[i] == 0) continue;
      const Unit u = unit_of<D, KIND>(threadIdx.x + i * kMoveThreads);
      if (!u.v_codes) {
        uint8_t* p = a.dst + dst + u.off + u.row * u.row_bytes + u.chunk * 16;
        if (u.bytes == 16)
          *reinterpret_cast<uint4*>(p) = v[i][0];
        else if (u.bytes == 8)
          *reinterpret_cast<uint2*>(p) = make_uint2(v[i][0].x, v[i][0].y);
        else
          *reinterpret_cast<uint16_t*>(p) = uint16_t(v[i][0].x);
      } else {
        const int units = u.row_bytes / 2, pair = u.row >> 1;
        uint8_t* p = a.dst + dst + u.off + pair * (2 * u.row_bytes) +
                     ((4 * u.chunk) ^ v_unit_swizzle(pair, units)) * 4;
        // bytes of the first token from the first word's half, of the second from the second's
        const uint32_t pick = ((live[i] & 4) ? 0x32u : 0x10u) | ((live[i] & 8) ? 0x7600u : 0x5400u);
        const uint32_t w[4] = {__byte_perm(v[i][0].x, v[i][1].x, pick), __byte_perm(v[i][0].y, v[i][1].y, pick),
                               __byte_perm(v[i][0].z, v[i][1].z, pick), __byte_perm(v[i][0].w, v[i][1].w, pick)};
        if ((live[i] & 3) == 3) {
          *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {   // one token of the pair alone: its 16-bit halves
          const int e = (live[i] & 3) >> 1;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint16_t*>(p + 4 * k + 2 * e) = uint16_t(w[k] >> (16 * e));
        }
      }
    }
    if (moves_weights && threadIdx.x < kTile && tile * kTile + threadIdx.x < kept)
      a.to_weights[bh * a.dst_cap + tile * kTile + threadIdx.x] = wt;
  }
  // new tokens start at weight 0 (in place: after the last wave's barrier every source is read)
  if (moves_weights) {
    float* const w = a.to_weights + bh * a.dst_cap;
    for (int t = kept + first_tile * kMoveThreads + threadIdx.x; t < a.dst_cap; t += step * kMoveThreads) w[t] = 0.f;
  }
}

template <int D, bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, 6) evict_compact_kernel(const __grid_constant__ MoveArgs a) {
  const int sect = blockIdx.y;                       // 0: reference, 1 + l: loop l
  if (sect == 0)
    move_section<D, IN_PLACE, 0>(a, 0);
  else if (a.res_bits[sect - 1] == 2)
    move_section<D, IN_PLACE, 2>(a, sect);
  else
    move_section<D, IN_PLACE, 4>(a, sect);
}

template <typename Kernel, typename Args>
cudaError_t launch_clusters(Kernel kernel, dim3 grid, int threads, size_t smem, int cluster,
                            cudaStream_t stream, const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

}  // namespace

cudaError_t launch_evict_select(const float* weights, int batch, int n_kv_heads, int capacity,
                                const int32_t* ctx_lens, int budget, int n_first, int n_last,
                                int32_t* keep, int32_t* kept_lens, cudaStream_t stream) {
  SelArgs a;
  a.weights = weights;
  a.ctx_lens = ctx_lens;
  a.keep = keep;
  a.kept_lens = kept_lens;
  a.H = n_kv_heads;
  a.cap = capacity;
  a.budget = budget;
  a.n_first = n_first;
  a.n_last = n_last;
  const int64_t rows = int64_t(batch) * n_kv_heads;
  if (capacity <= kShortRow) {
    a.slice = 0;
    evict_select_short_kernel<<<unsigned(rows), kShortRow / 4, 0, stream>>>(a);
    return cudaGetLastError();
  }
  // CTAs per row: enough that the keys fit shared memory, more while the rows leave SMs free
  // and each CTA keeps a few thousand slots
  int C = 1;
  auto per_cta = [&](int c) { return (int64_t(capacity) / c + 32 * kSelWarps + 31) / 32 * 32; };   // (warps take 32s)
  while (C < kSelMaxCluster && (per_cta(C) > kSelKeys || (rows * C * 2 <= device_sm_count() && capacity / C >= 4096)))
    C *= 2;
  a.slice = per_cta(C) <= kSelKeys ? int(per_cta(C)) : 0;
  static OncePerDevice once;
  const cudaError_t e = once([] {
    return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  });
  if (e != cudaSuccess) return e;
  return launch_clusters(evict_select_kernel, dim3(unsigned(rows * C)), kSelThreads,
                         size_t(a.slice) * 4, C, stream, a);
}

cudaError_t launch_evict_compact(const rq_shape& s, const rq_cache& cache, const rq_paging* paging,
                                 const rq_shape& ts, const rq_cache& to, const rq_paging* to_paging,
                                 bool in_place, const int32_t* keep, int budget,
                                 const int32_t* kept_lens, const float* weights, float* to_weights,
                                 cudaStream_t stream) {
  MoveArgs a;
  a.src = cache.data;
  a.dst = to.data;
  a.rec_bytes = record_bytes(s);
  a.src_bt = paging ? paging->block_table : nullptr;
  a.src_max_pages = paging ? paging->max_pages : 0;
  a.src_n_pages = paging ? paging->n_pages : 0;
  a.dst_bt = to_paging ? to_paging->block_table : nullptr;
  a.dst_max_pages = to_paging ? to_paging->max_pages : 0;
  a.dst_n_pages = to_paging ? to_paging->n_pages : 0;
  a.keep = keep;
  a.kept_lens = kept_lens;
  a.weights = weights;
  a.to_weights = to_weights;
  a.H = s.n_kv_heads;
  a.L = s.n_loops;
  a.budget = budget;
  a.src_cap = s.capacity;
  a.dst_cap = ts.capacity;
  const int kept_most = budget < ts.capacity ? budget : ts.capacity;
  const int tiles = (kept_most + kTile - 1) / kTile;
  // four tiles per CTA hide the look-up of the sources behind the moves; fewer where that would
  // leave SMs idle
  const int64_t units = int64_t(s.batch) * s.n_kv_heads * s.n_loops;
  const int per = units * ((tiles + 3) / 4) >= 8 * int64_t(device_sm_count()) ? 4 : 1;
  a.ctas = (tiles + per - 1) / per;
  for (int l = 0; l < RQ_MAX_LOOPS; ++l) a.res_bits[l] = s.res_bits[l];
  const int64_t bh = int64_t(s.batch) * s.n_kv_heads;
  const int64_t x = bh * (in_place ? kMoveCluster : a.ctas);
  if (x > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const dim3 grid{unsigned(x), unsigned(s.n_loops), 1u};
  if (in_place) {
    if (s.head_dim == 128)
      return launch_clusters(evict_compact_kernel<128, true>, grid, kMoveThreads, 0, kMoveCluster, stream, a);
    return launch_clusters(evict_compact_kernel<64, true>, grid, kMoveThreads, 0, kMoveCluster, stream, a);
  }
  if (s.head_dim == 128)
    evict_compact_kernel<128, false><<<grid, kMoveThreads, 0, stream>>>(a);
  else
    evict_compact_kernel<64, false><<<grid, kMoveThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rq
