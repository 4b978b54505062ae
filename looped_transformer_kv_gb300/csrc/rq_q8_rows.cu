// Attention over the 8-bit cache for many query rows (include/rq_q8.h) on the 5th-generation tensor
// cores: blocks of 256 rows (two tiles of 128) share every tile of 128 keys.
//
//   S = Q K^T, O += P V as tcgen05 products of 128 x 128 tiles; S, P and O in tensor memory.
// Codes become fp16 operands exactly: a key tile takes the largest of its blocks' scales as its own, the
// codes of the others are multiplied by the power of two between them, down to 2^-kFold; in a tile whose
// scales lie further apart codes stay as they are, and scores and weights get their block's scale one by one
// (`careful`).  V's tile scale 2^e_V goes into the weights' exponent and is taken out of their sum again,
//   P = 2^((S 2^(e_K - e_q) - R) c + e_V - h),  l += 2^(h - e_V) sum P,
// so that tiles of different scales need no rescaling of O; 2^e_q is what brought the row's query into
// fp16's range.  R (a row's largest q K) and h are raised when a weight would exceed 2^15, to make the
// largest 2^7.  Tiles whose exponents do not allow the products to be drawn together, tiles of a V so small
// beside another's that weights would leave fp32's range before they are summed, and rows of huge scores
// take another loop over the scores (`careful`).
//
// The operands are made once, in the workspace (q8_query_kernel, q8_image_kernel), and copied from there.
// (A kernel that converted what it read, without the workspace, was slower from 33 rows on: its loads and
// conversions took registers from the softmax, 67 against 33 us for 260 rows after 500 slots.)
//
// Warps 0-3 and 4-7: softmax of row tile 0 and 1, a thread per row; warp 8: products; warp 9: copies.
// Bound by a row tile's chain, softmax and then products, two tiles taking turns: 2,048 tokens of 32 heads
// after 14,336 slots in 331 us, 1,560 TFLOP/s.
// CTAs (one per SM) share the work by the line of rq_q8_line.cuh; q8_join_kernel joins the partial results
// of divided units (in this kernel the code for it cost the main loop its registers: 460 against 375 us).
#include <type_traits>

#include "rq_q8_line.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr int kFold = 8;              // exponents of a tile's scales, at most, that go into its operands
constexpr int kApart = 4096;          // added to K's exponent of a tile whose scales do not
constexpr int kFarBelow = 40;         // V's exponent below a row's h: weights of 2^-86 are still summed
constexpr int kKeys = 128, kRowTile = 128, kBlockRows = 2 * kRowTile;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMostCtas = 1024;
using RowWalk = Walk<kBlockRows, kKeys>;

template <int D>
struct RowsSmem {
  static constexpr int kTile = kKeys * D * 2;               // one K, V or Q tile
  static constexpr int v = 0, k = 2 * kTile, q = 5 * kTile;   // V first: see v_desc
  static constexpr int bars = 7 * kTile, walks = bars + 256;
  static constexpr int kImage = 2 * kTile + 128, kQueryImage = kTile + 4 * kRowTile;   // of tiles in the workspace
  static constexpr int total = walks + 4 * int(sizeof(RowWalk)) + 1024;   // + alignment of the base
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

// V tile as the product's B operand, channels contiguous: panels of 64 channels, rows of 128 bytes a
// token; 8 tokens are 1024 bytes, panels kKeys * 128 bytes apart.
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(kKeys * 128 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void group_sync(int i) {         // 128 threads of softmax group 0 or 1
  if (i == 0)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else
    asm volatile("bar.sync 2, 128;" ::: "memory");
}
__device__ __forceinline__ bool group_any(int i, bool x) {
  uint32_t y;
  if (i == 0)
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y) : "r"(uint32_t(x)) : "memory");
  else
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y) : "r"(uint32_t(x)) : "memory");
  return y != 0u;
}

__device__ __forceinline__ uint32_t half2_pow2(int e) { return (uint32_t(15 + e) << 10) * 0x10001u; }   // 2^e twice, -14 <= e

// Two codes times the power of two f (bias: int8's -1152 f).
template <int FMT, int HALF>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t w, uint32_t f, uint32_t bias) {
  uint32_t out;
  if (FMT == RQ_Q8_INT8) {
    const uint32_t t = __byte_perm(w, 0x64646464u, HALF ? 0x4342 : 0x4140);
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out) : "r"(t), "r"(f), "r"(bias));
  } else {
    asm("mul.f16x2 %0, %1, %2;" : "=r"(out) : "r"(q8_pair<FMT, HALF>(w)), "r"(f));
  }
  return out;
}

// Bit y of the result: column y (0..31) lies in [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int lo, int hi) {
  const uint32_t below_hi = hi >= 32 ? ~0u : hi <= 0 ? 0u : (1u << hi) - 1u;
  const uint32_t below_lo = lo >= 32 ? ~0u : lo <= 0 ? 0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}

struct RowsArgs : Q8Line {
  uint8_t* images;       // operand tiles, [B][Hkv][list] of K, V, their exponents
  uint8_t* queries;      // [B][Hkv][row_tiles] of rows, their factors
  int32_t list, row_tiles;   // of one unit, at most
};

// Rows rr0 .. + ROWS of a tile of 128 query rows (row r0 of the sequence and on, `live` of them) to fp16
// operands, each times a power of two that brings its largest element into [2^14, 2^15) (bf16 values are
// exact then; at most 2^kMostUp); factors: its inverse.  One warp; a lane holds two runs of four
// channels that are turned into each other, so that it reads no angle that another lane reads (eight
// neighbouring channels a lane, partners by shuffles: 1,023 tokens of 4 x 16 heads in 19 us, now 13).
template <int D, int ROWS>
__device__ __forceinline__ void put_queries(const Q8Line& a, const Rows& x, int b, int h, int r0, int rr0, int live,
                                            uint8_t* tile, float* factors, int lane) {
  constexpr int LPR = D / 8, RPI = 32 / LPR, IT = ROWS / RPI, TOGETHER = IT < 2 ? IT : 2;   // (rows whose loads are in flight)
  const Q8Rope& rope = a.c.rope;
  const int qc = lane % LPR, apart = rope.table != nullptr && !rope.interleaved ? rope.rot / 8 : 0;
  const int first = qc < apart ? qc : 2 * qc, second = qc < apart ? qc + apart : 2 * qc + 1;   // (2 apart + 2 (qc - apart))
#pragma unroll 1
  for (int y0 = 0; y0 < IT; y0 += TOGETHER) {
    uint2 raw[TOGETHER][2];
    float4 angles[TOGETHER][2];                              // cos, sin of four pairs
    bool lost[TOGETHER], turned[TOGETHER];
#pragma unroll
    for (int y = 0; y < TOGETHER; ++y) {
      const int rr = rr0 + (y0 + y) * RPI + lane / LPR;
      const int j = (r0 + rr) / a.G, hq = h * a.G + (r0 + rr) % a.G;
      raw[y][0] = raw[y][1] = make_uint2(0u, 0u);
      lost[y] = turned[y] = false;
      if (rr >= live) continue;
      const uint16_t* const row = a.c.q + b * a.c.q_strides[0] + j * a.c.q_strides[1] + hq * a.c.q_strides[2];
      raw[y][0] = q8_load4(row + 4 * first, a.qvec);
      raw[y][1] = q8_load4(row + 4 * second, a.qvec);
      if (rope.table == nullptr) continue;
      const int p = rope.positions ? rope.positions[int64_t(b) * a.c.n_new + j] : x.ctx + j;
      lost[y] = p < 0 || p >= rope.n_pos;
      turned[y] = !lost[y] && 8 * qc < rope.rot;
      if (!turned[y]) continue;
      const float4* const at = reinterpret_cast<const float4*>(rope.table + int64_t(p) * rope.rot + 8 * qc);
      angles[y][0] = at[0];
      angles[y][1] = at[1];
    }
#pragma unroll
    for (int y = 0; y < TOGETHER; ++y) {
      const int rr = rr0 + (y0 + y) * RPI + lane / LPR;
      float f[8];
      q8_floats(make_uint4(raw[y][0].x, raw[y][0].y, raw[y][1].x, raw[y][1].y), f);
      if (turned[y]) {
        const float cs[8] = {angles[y][0].x, angles[y][0].y, angles[y][0].z, angles[y][0].w,
                             angles[y][1].x, angles[y][1].y, angles[y][1].z, angles[y][1].w};
        if (apart == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) q8_turn(f[2 * k], f[2 * k + 1], cs[2 * k], cs[2 * k + 1]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) q8_turn(f[k], f[k + 4], cs[2 * k], cs[2 * k + 1]);
        }
      }
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(f[k]));
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(RQ_FULL_MASK, mx, o));
      const int ex = int(__float_as_uint(mx) >> 23);
      const int e = mx == 0.f || ex == 255 ? 0 : min(141 - ex, kMostUp);
      const float up = q8_pow2(e >> 1), up2 = q8_pow2(e - (e >> 1));
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = pack_half2(f[2 * k] * up * up2, f[2 * k + 1] * up * up2);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int run = k ? second : first, chunk = run / 2;
        *reinterpret_cast<uint2*>(tile + (chunk / 8) * (kRowTile * 128) + panel_offset(rr, chunk % 8) + 8 * (run & 1)) =
            make_uint2(o[2 * k], o[2 * k + 1]);
      }
      if (qc == 0)
        factors[rr] = lost[y] ? __int_as_float(0x7fc00000) : q8_pow2(-e);
    }
  }
}

// One key tile of 128 slots from codes to operands by 128 threads, a thread the same 16 channels of
// every 16th (d = 64: 32nd) row.
template <int D, int FMT>
struct Converter {
  static constexpr int CPR = D / 16;                         // 16-byte chunks of a row
  static constexpr int PIECES = kKeys * CPR / 128;           // of a thread and K or V tile
  const Q8Line& a;
  const int tid, lane, row0, c, first;
  const uint32_t panel;
  int64_t rec[2];                                            // records of the tile's halves; -1: no page, -2: not there
  float scale;                                               // lane l < 16: block l % 8 of K (l < 8) or V
  uint32_t factor, lost;                                     // of take_scales: 2^(e - top) of the same (1: not folded); K's blocks to spoil
  uint32_t exps;                                             // ... lane 4 k of the first 16: exponents of four blocks, a byte each
  int at[2], end, oldest;                                    // slots of the halves' first rows; what is seen

  // (rows of a thread's pieces differ by multiples of 16, so the chunk is the same; `first`: which half
  // is stored first, so that neighbours meet distinct banks)
  __device__ __forceinline__ Converter(const Q8Line& line, int t, int l)
      : a(line), tid(t), lane(l), row0(t / CPR), c((t % CPR) ^ q8_swizzle<D>(t / CPR)),
        first(D == 128 && c >= 4 ? 1 : 0), panel(uint32_t(c / 4) * (kKeys * 128)), scale(1.f), factor(0u), lost(0u), exps(0u) {}

  __device__ __forceinline__ int64_t record(const Rows& x, int b, int h, int v) const {
    if (v >= x.tiles) return -2;
    const int64_t r = a.v.record(b, h, x.tile(v));
    if (r == -1) {
      grid_wait();                                           // (the kernel before clears it)
      atomicOr(a.err, 1u);
    }
    return r;
  }
  __device__ __forceinline__ void load(uint4 (&reg)[PIECES], int kv) const {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int half = p >= PIECES / 2;
      reg[p] = make_uint4(0u, 0u, 0u, 0u);
      if (rec[half] >= 0)
        reg[p] = __ldg(reinterpret_cast<const uint4*>(a.v.codes + rec[half] * a.v.rec_codes + kv * (kQ8Tile * D)) + tid +
                       (p - half * (PIECES / 2)) * 128);
    }
  }
  __device__ __forceinline__ void load_scales() {
    const int64_t r = lane & 4 ? rec[1] : rec[0];
    scale = r >= 0 && lane < 16 ? a.v.scales[r * a.v.rec_scales + (lane >> 3) * 4 + (lane & 3)] : 1.f;
  }
  // The tile's exponents of K and V, from its blocks that hold something; the tile begins at place v.
  __device__ __forceinline__ int2 take_scales(const Rows& x, int v) {
    const int half = lane >> 2 & 1;
    const int64_t r = half ? rec[1] : rec[0];
#pragma unroll
    for (int k = 0; k < 2; ++k) at[k] = v + k < x.tiles ? x.tile(v + k) * kQ8Tile : 1 << 30;   // (not there: behind the end)
    end = x.end;
    oldest = x.oldest;
    const int first = (half ? at[1] : at[0]) + (lane & 3) * kQ8Block;          // the block's first slot
    const bool live = r >= 0 && lane < 16 && first < end && (first + kQ8Block > oldest || first < a.c.n_sink);
    const bool nan = live && !(scale < INFINITY);
    const int e = live && !nan ? q8_exponent(scale) : -1000;
    int top = e, least = e == -1000 ? 1000 : e;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      top = max(top, __shfl_xor_sync(RQ_FULL_MASK, top, o));
      least = min(least, __shfl_xor_sync(RQ_FULL_MASK, least, o));
    }
    if (top == -1000) top = least = 0;
    const bool folded = top - least <= kFold;
    factor = e == -1000 ? 0u : half2_pow2(folded ? e - top : 0);
    exps = uint32_t((folded || e == -1000 ? top : e) & 255) << (8 * (lane & 3));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) exps |= __shfl_xor_sync(RQ_FULL_MASK, exps, o);
    const int apart = __any_sync(RQ_FULL_MASK, !folded) ? kApart : 0;
    // (a scale that is not a number, K's or V's, spoils the scores: V then only meets weights of tokens
    // that see the block)
    const uint32_t nans = __ballot_sync(RQ_FULL_MASK, nan || (r == -1 && lane < 16));
    lost = (nans | (nans >> 8)) & 255u;
    return make_int2(__shfl_sync(RQ_FULL_MASK, top, 0) + apart, __shfl_sync(RQ_FULL_MASK, top, 8));
  }
  // Operands of K or V.
  __device__ __forceinline__ void put(const uint4 (&reg)[PIECES], uint8_t* tile, int kv) const {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const int row = row0 + p * (128 / CPR), blk = row >> 4;
      const uint32_t f = __shfl_sync(RQ_FULL_MASK, factor, 8 * kv + blk);
      uint32_t bias;
      asm("mul.f16x2 %0, %1, %2;" : "=r"(bias) : "r"(f), "r"(0xe480e480u));   // -1152 f
      const uint32_t wd[4] = {reg[p].x, reg[p].y, reg[p].z, reg[p].w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t y = q8_word<FMT>(wd[k]);
        o[2 * k] = scaled_pair<FMT, 0>(y, f, bias);
        o[2 * k + 1] = scaled_pair<FMT, 1>(y, f, bias);
      }
      // (slots that no token sees may hold anything, in V codes that are not numbers too)
      const int slot = (row < kQ8Tile ? at[0] : at[1]) + row % kQ8Tile;
      const bool spoil = kv == 0 && (lost >> blk & 1u);
      const bool none = kv == 1 && (slot >= end || (slot < oldest && slot >= a.c.n_sink));
      if (spoil || none)
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = none ? 0u : 0x7fff7fffu;
      uint8_t* const at = tile + panel;
      const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
      const int ch = 2 * (c & 3);
      *reinterpret_cast<uint4*>(at + panel_offset(row, ch + first)) = first ? hi : lo;
      *reinterpret_cast<uint4*>(at + panel_offset(row, ch + 1 - first)) = first ? lo : hi;
    }
  }
};

// The schedule, and beside it the operand tiles of the queries, kQueryRows rows a warp.  (Small calls wait
// for a warp's rounds of loads, large ones for CTAs that begin: with 4, 8 and 16 rows a warp 17 tokens of 3
// sequences take 14.1, 14.3 and 15.0 us, 1,023 tokens of 4 x 16 heads 72, 71 and 71.)
constexpr int kQueryRows = 8, kQueryParts = kRowTile / (8 * kQueryRows);   // CTAs of a row tile

template <int D>
__global__ void __launch_bounds__(256, 4) q8_query_kernel(const __grid_constant__ RowsArgs a) {
  grid_next();
  using L = RowsSmem<D>;
  if (blockIdx.x == 0) {
    cut_line<kBlockRows, kKeys, 256>(a);
    return;
  }
  const unsigned tile = (blockIdx.x - 1) / kQueryParts, part = (blockIdx.x - 1) % kQueryParts;
  const int unit = int(tile / unsigned(a.row_tiles)), b = unit / a.v.H, h = unit % a.v.H;
  const int t = int(tile % unsigned(a.row_tiles));
  const Rows x = sequence_of(a, b);
  const int live = x.ok ? x.n * a.G - t * kRowTile : 0;
  if (live <= 0) return;
  uint8_t* const image = a.queries + (int64_t(unit) * a.row_tiles + t) * L::kQueryImage;
  put_queries<D, kQueryRows>(a, x, b, h, t * kRowTile, int(part * 8 + (threadIdx.x >> 5)) * kQueryRows, live, image,
                             reinterpret_cast<float*>(image + L::kTile), threadIdx.x & 31);
}

// Operand tiles of K and V: 128 threads each for one key tile.  They need nothing of the queries' kernel and
// run beside it; it is complete when this one is.  Bound by HBM: 14,336 + 2,048 slots of 8
// heads, 33 MB of codes to 67 MB of operands, in 19 us.
template <int D, int FMT>
__global__ void __launch_bounds__(256) q8_image_kernel(const __grid_constant__ RowsArgs a) {
  grid_next();
  using L = RowsSmem<D>;
  const int lane = threadIdx.x & 31, kv = threadIdx.x >> 7;
  const int u = int(blockIdx.x % unsigned(a.list));
  const int unit = int(blockIdx.x / unsigned(a.list)), b = unit / a.v.H, h = unit % a.v.H;
  const Rows x = sequence_of(a, b);
  if (2 * u >= x.tiles) {
    grid_wait();
    return;
  }
  Converter<D, FMT> to(a, threadIdx.x & 127, lane);
  to.rec[0] = to.record(x, b, h, 2 * u);
  to.rec[1] = to.record(x, b, h, 2 * u + 1);
  uint4 reg[Converter<D, FMT>::PIECES];
  to.load(reg, kv);
  to.load_scales();
  const int2 e = to.take_scales(x, 2 * u);
  uint8_t* const image = a.images + (int64_t(unit) * a.list + u) * L::kImage;
  to.put(reg, image + kv * L::kTile, kv);
  if (threadIdx.x == 0) *reinterpret_cast<int2*>(image + 2 * L::kTile) = e;
  if (threadIdx.x < 16 && (threadIdx.x & 3) == 0) *reinterpret_cast<uint32_t*>(image + 2 * L::kTile + 16 + threadIdx.x) = to.exps;
  grid_wait();
}

// Exponents of tile t of the walk's segment: K's (and whether its blocks lie apart) and V's; 16 bytes on,
// those of its blocks, a byte each.
template <int D, typename W>
__device__ __forceinline__ const int2* image_exps(const RowsArgs& a, const W& w, int t) {
  return reinterpret_cast<const int2*>(a.images + ((int64_t(w.b) * a.v.H + w.h) * a.list + w.x.step(w.kt0 + t)) * RowsSmem<D>::kImage +
                                       2 * RowsSmem<D>::kTile);
}

__device__ __forceinline__ void store32(void* to, const uint4& a, const uint4& b) {   // 32 bytes, aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(to), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}
__device__ __forceinline__ uint4 bf16_row(const float (&v)[8], float inv, float up) {   // times inv up^2
  uint32_t p[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 u = __floats2bfloat162_rn(v[2 * k] * inv * up * up, v[2 * k + 1] * inv * up * up);
    p[k] = *reinterpret_cast<const uint32_t*>(&u);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

template <int D>
__global__ void __launch_bounds__(384, 1) q8_rows_kernel(const __grid_constant__ RowsArgs a) {
  grid_wait();
  grid_next();
  const int me = int(blockIdx.x);
  if (me >= *a.used) return;
  extern __shared__ uint8_t raw[];
  using L = RowsSmem<D>;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  // barriers: K full [3], V full [2], step [8], S of row tile 0 [2], P ready [row
  // tile][half], Q ready, drained.
  // A step ends with the last row tile's scores of a tile (and the values of the tile before), or with
  // the values of a segment's last tile: T + 1 steps for T tiles.  It frees K and V tiles.
  const uint32_t bar0 = smem_u32(bars);
  auto kfull = [&](int g) { return bar0 + 8 * (g % 3); };
  auto vfull = [&](int g) { return bar0 + 8 * (3 + (g & 1)); };
  auto step = [&](int n) { return bar0 + 8 * (5 + (n & 7)); };
  auto sready = [&](int c) { return bar0 + 8 * (13 + (c & 1)); };
  auto pready = [&](int i, int half) { return bar0 + 8 * (15 + 2 * i + half); };
  const uint32_t qready = bar0 + 8 * 19, drained = bar0 + 8 * 20;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 21);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 8) tc_alloc(smem_u32(tslot), 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(bar0 + 8 * i, 1);
    for (int i = 5; i < 15; ++i) mbar_init(bar0 + 8 * i, 1);
    for (int i = 15; i < 19; ++i) mbar_init(bar0 + 8 * i, kRowTile);
    mbar_init(qready, 3);                                    // the copy, both softmax groups
    mbar_init(drained, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Cut from = a.cut[me];
  const int64_t to_pos = a.cut[me + 1].pos;
  RowWalk* const walks = reinterpret_cast<RowWalk*>(smem + L::walks);           // of the softmax groups, products, copies
  bool failed = false;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const bool leader = elect_one();
    if (warp == 9 && leader) {                        // ---- copies of operand tiles
      RowWalk& w = walks[3];
      w.begin(from, to_pos);
      int seg = 0;                                           // segments whose queries are on their way
      int g = 0, n0 = 0;                                     // tiles so far; g's step is n0 + g
      int sk[3] = {-1, -1, -1};                              // steps that end with K tile g - 1, g - 2, g - 3
      while (!failed && w.next(a)) {
        if (!w.x.ok) continue;
        const uint8_t* const unit = a.images + (int64_t(w.b) * a.v.H + w.h) * a.list * RowsSmem<D>::kImage;
        const uint8_t* const queries = a.queries + ((int64_t(w.b) * a.v.H + w.h) * a.row_tiles + w.block * (kBlockRows / kRowTile)) * L::kQueryImage;
        const int row_tiles = w.x.rows > kRowTile ? 2 : 1;
        for (int t = 0; t < w.T; ++t, ++g) {
          const uint8_t* const tile = unit + w.x.step(w.kt0 + t) * int64_t(RowsSmem<D>::kImage);
          if (g >= 3) failed = !mbar_wait_bounded(step(sk[2]), (sk[2] >> 3) & 1, kWaitNs);
          if (failed) break;
          mbar_arrive_expect_tx(kfull(g), L::kTile);
          bulk_g2s(smem_u32(smem + L::k + (g % 3) * L::kTile), tile, L::kTile, kfull(g));
          if (t == 0) {                                      // queries, once the last scores need those before no more
            if (g > 0) failed = !mbar_wait_bounded(step(sk[0]), (sk[0] >> 3) & 1, kWaitNs);
            if (failed) {
              ++g;
              break;
            }
            mbar_arrive_expect_tx(qready, row_tiles * L::kTile);
            for (int i = 0; i < row_tiles; ++i) bulk_g2s(smem_u32(smem + L::q + i * L::kTile), queries + i * L::kQueryImage, L::kTile, qready);
            ++seg;
          }
          if (g >= 2) failed = !mbar_wait_bounded(step(sk[1] + 1), ((sk[1] + 1) >> 3) & 1, kWaitNs);
          if (failed) {
            ++g;
            break;
          }
          mbar_arrive_expect_tx(vfull(g), L::kTile);
          bulk_g2s(smem_u32(smem + L::v + (g & 1) * L::kTile), tile + L::kTile, L::kTile, vfull(g));
          sk[2] = sk[1];
          sk[1] = sk[0];
          sk[0] = n0 + g;
        }
        ++n0;
      }
      // copies land before the CTA leaves
      for (int k = max(0, g - 3); failed && k < g; ++k) mbar_wait_bounded(kfull(k), (k / 3) & 1, kWaitNs);
      for (int k = max(0, g - 2); failed && k < g; ++k) mbar_wait_bounded(vfull(k), (k >> 1) & 1, kWaitNs);
      if (failed && seg > 0) mbar_wait_bounded(qready, (seg - 1) & 1, kWaitNs);
    } else if (warp == 8 && leader) {                        // ---- products
      constexpr uint32_t ids = f16_idesc(kRowTile, kKeys), ido = f16_idesc(kRowTile, D) | (1u << 16);   // (B: channels contiguous)
      int g = 0, c0 = 0, c1 = 0, n = 0, seg = 0;             // tiles; P's of row tile 0, 1; steps; segments
      int s0 = 0;                                            // S's of row tile 0 with a row tile 1
      bool good = true;
      auto scores = [&](int i, int gk) {
        const uint32_t q = smem_u32(smem + L::q + i * L::kTile), k = smem_u32(smem + L::k + (gk % 3) * L::kTile);
#pragma unroll
        for (int y = 0; y < D / 16; ++y)
          tc_mma(tmem + 128 * i, panel_desc(q + (y / 4) * (kRowTile * 128) + (y % 4) * 32),
                 panel_desc(k + (y / 4) * (kKeys * 128) + (y % 4) * 32), ids, y > 0);
      };
      auto values = [&](int i, int gv, int parity, bool add) {       // false: a wait gave up
        const uint32_t v = smem_u32(smem + L::v + (gv & 1) * L::kTile);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_bounded(pready(i, half), parity, kWaitNs)) return false;
          tc_fence_after();
#pragma unroll
          for (int y = 4 * half; y < 4 * half + 4; ++y)
            tc_mma_ta(tmem + 256 + 128 * i, tmem + 128 * i + 8 * y, v_desc(v + y * 2048), ido, add || y > 0);
        }
        return true;
      };
      RowWalk& w = walks[2];
      w.begin(from, to_pos);
      while (good && w.next(a)) {
        if (!w.x.ok) continue;
        const bool two = w.x.rows > kRowTile;
        good = mbar_wait_bounded(kfull(g), (g / 3) & 1, kWaitNs) && mbar_wait_bounded(qready, seg & 1, kWaitNs);
        ++seg;
        tc_fence_after();
        if (!good) break;
        scores(0, g);
        if (two) {
          tc_commit(sready(s0++));
          scores(1, g);
        }
        tc_commit(step(n++));
        for (int j = 0; j < w.T && good; ++j, ++g) {
          good = mbar_wait_bounded(vfull(g), (g >> 1) & 1, kWaitNs);
          const bool more = j + 1 < w.T;
          if (good && more) good = mbar_wait_bounded(kfull(g + 1), ((g + 1) / 3) & 1, kWaitNs);
          if (!good) break;
          good = values(0, g, c0++ & 1, j > 0);
          if (!good) break;
          if (more) scores(0, g + 1);
          if (two) {
            if (more) tc_commit(sready(s0++));
            good = values(1, g, c1++ & 1, j > 0);
            if (!good) break;
            if (more) scores(1, g + 1);
          }
          tc_commit(step(n++));
        }
      }
      if (!good) {                                           // nothing in flight when the CTA leaves
        tc_commit(drained);
        mbar_wait_bounded(drained, 0, kWaitNs);
        failed = true;
      }
    }
    __syncwarp();
  } else {                                                   // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int i = warp >> 2, r = threadIdx.x & (kRowTile - 1);
    const uint32_t lanes = uint32_t(warp & 3) << 21;          // this warp's tensor-memory lanes
    const uint32_t tS = tmem + 128 * i + lanes, tO = tmem + 256 + 128 * i + lanes;
    int g = 0, n0 = 0, s0 = 0, seg = 0;
    RowWalk& w = walks[i];                                     // the group's first thread walks
    if (r == 0) w.begin(from, to_pos);
    for (;;) {                                                 // (failed: nothing is waited for any more, results are NaN)
      group_sync(i);
      if (r == 0) w.next(a);
      group_sync(i);
      if (!w.more) break;
      const Rows& x = w.x;
      const int r0 = w.block * kBlockRows + i * kRowTile;      // the row tile's first row
      const bool two = x.rows > kRowTile, mine = i == 0 || two;
      const int row = r0 + r;
      float factor = 0.f;
      if (x.ok && !failed) {
        const uint8_t* const image = a.queries + ((int64_t(w.b) * a.v.H + w.h) * a.row_tiles + r0 / kRowTile) * L::kQueryImage;
        if (r == 0) mbar_arrive(qready);                       // (the products keep to a segment with both groups)
        if (mine) factor = *reinterpret_cast<const float*>(image + L::kTile + 4 * r);
        // Group 1 has segments without rows, in which nothing ties it to the products' steps: it waits for
        // its segment to begin, a phase whose successor needs its own arrival.  (The steps' ring tells one
        // lap from the next but not from the one after: it could neither run ahead nor poll along.)
        if (i == 1) failed = group_any(1, !mbar_wait_bounded(qready, seg & 1, kWaitNs));
        ++seg;
      }
      const float c = a.scale_log2;
      float R = -INFINITY, h = 0.f, l = 0.f;
      if (!mine) {                                             // no rows
        if (!x.ok || failed) continue;
        g += w.T;
        ++n0;
        continue;
      }
      if (x.ok && !failed) {
        // exponents of a tile's K for which 2^(e_K - e_q) and its product with c are far from fp32's ends
        // for all rows of the warp: from ke_min to ke_max
        const int fe = q8_exponent(factor);
        const bool tame = c > 0x1p-30f && c < 0x1p30f;
        const int ke_min = tame ? -90 - __reduce_min_sync(RQ_FULL_MASK, fe) : 1, ke_max = tame ? 90 - __reduce_max_sync(RQ_FULL_MASK, fe) : 0;
        const int own = x.ctx + min(row / a.G, x.n - 1);       // the row's own slot
        const int own0 = x.ctx + r0 / a.G, own1 = x.ctx + min((r0 + kRowTile - 1) / a.G, x.j1);   // of the tile's rows
        const int win = a.c.window > 0 ? a.c.window : 1 << 30, sinks = a.c.window > 0 ? a.c.n_sink : 0;
        int2 ee32 = make_int2(0, 0);                           // a lane's exponents of 32 tiles
        bool huge = false;                                     // scores beyond 2^20 in some row of the warp
        int h_top = kNoScale;                                  // the largest h of the warp's rows
        for (int t = 0; t < w.T; ++t, ++g) {
          // ---- before the scores are there: the tile's exponents, and what of it the warp's rows see
          if ((t & 31) == 0) ee32 = t + lane < w.T ? *image_exps<D>(a, w, t + lane) : make_int2(0, 0);
          const int2 ee = make_int2(__shfl_sync(RQ_FULL_MASK, ee32.x, t & 31), __shfl_sync(RQ_FULL_MASK, ee32.y, t & 31));
          int at[2];
          bool clear[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int v = 2 * x.step(w.kt0 + t) + half;
            at[half] = v < x.tiles ? x.tile(v) * kQ8Tile : 1 << 30;            // (not there: behind every row)
            clear[half] = at[half] + 63 <= own0 && (at[half] > own1 - win || at[half] + 63 < sinks);
          }
          const int n = n0 + g;
          bool good;
          if (i == 0 && two) {
            good = mbar_wait_bounded(sready(s0), (s0 >> 1) & 1, kWaitNs);
            ++s0;
          } else {
            good = mbar_wait_bounded(step(n), (n >> 3) & 1, kWaitNs);
          }
          if (__any_sync(RQ_FULL_MASK, !good)) {               // (the warp leaves as one)
            failed = true;
            break;
          }
          tc_fence_after();
          const float ev = float(ee.y);
          // O, whose unit changes with h and R, times f (a lane's row); every lane of the warp calls it
          auto rescale = [&](float f) {
            if (t == 0) return;
#pragma unroll 1
            for (int y = 0; y < D / 16; ++y) {
              uint32_t o[16];
              tc_ld16(tO + 16 * y, o);
              tc_wait_ld();
#pragma unroll
              for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
              tc_st16(tO + 16 * y, o);
            }
          };
          // rows of `over` get Rn for R, and an h that makes the largest of 2^(wn - h) 2^kWeightHead
          auto raise = [&](bool over, float Rn, float wn) {
            float f = 1.f, fo = 1.f;                           // of l, and of O
            if (over) {
              const float hn = wn - kWeightHead;
              if (R == -INFINITY) {
                f = fo = 0.f;
                h = hn;
              } else {
                const float d = (R - Rn) * c, h0 = h;
                h = fmaxf(hn, h + d);
                f = ex2(d);
                fo = ex2(d + (h0 - h));
              }
              R = Rn;
            }
            l *= f;
            huge = __any_sync(RQ_FULL_MASK, fabsf(R * c) > 0x1p20f && R != -INFINITY);
            h_top = __reduce_max_sync(RQ_FULL_MASK, R == -INFINITY ? kNoScale : int(ceilf(h)));
            rescale(fo);
          };
          auto weights_there = [&](int half) {                 // the values of its 64 keys may begin
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(pready(i, half));
          };
          auto seen_by = [&](int half, int q) {                // bit y: the row sees key 64 half + 32 q + y
            const int first = (half ? at[1] : at[0]) + 32 * q, hi = own - first + 1, lo = hi - win, sk = sinks - first;
            return range_bits(lo, hi) | range_bits(0, min(sk, hi));
          };
          bool slow = ee.x < ke_min || ee.x > ke_max || ee.y < h_top - kFarBelow;
          if (!slow) {
            uint32_t s[kKeys];
#pragma unroll
            for (int y = 0; y < 4; ++y) tc_ld32(tS + 32 * y, s + 32 * y);
            const float kq = q8_pow2(ee.x) * factor;
            tc_wait_ld();
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (clear[half]) continue;
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                const uint32_t seen = seen_by(half, q);
#pragma unroll
                for (int y = 0; y < 32; ++y)
                  if (!(seen >> y & 1u)) s[half * 64 + 32 * q + y] = 0xff800000u;
              }
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
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kq;
            const bool over = R == -INFINITY ? top > R : fmaf(top - R, c, ev - h) > kWeightTop;
            if (__any_sync(RQ_FULL_MASK, over)) {
              const float Rn = fmaxf(R, top);
              raise(over, Rn, fmaf(top - Rn, c, ev));
            }
            slow = huge;
            if (!slow) {
              const float mul = kq * c, add = fmaf(R == -INFINITY ? 0.f : -R, c, ev - h);
              const uint64_t c2 = pack2(mul, mul), h2 = pack2(add, add);
              uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                uint32_t p[32];
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                  const int k = half * 64 + 2 * y;
                  float p0, p1;
                  unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, h2), p0, p1);
                  p0 = ex2(p0);
                  p1 = ex2(p1);
                  sum[y & 1] = add2(sum[y & 1], pack2(p0, p1));
                  p[y] = pack_half2(p0, p1);
                }
                tc_st32(tS + 32 * half, p);
                weights_there(half);
              }
              float a0, a1;
              unpack2(add2(sum[0], sum[1]), a0, a1);
              l = fmaf(a0 + a1, ex2(h - ev), l);               // (h - ev: kFarBelow at most)
            }
          }
          if (slow) {
            // careful: scores as q K (the power of two in two steps, of the same direction), and differences
            // before the product with c, exactly: scores of any size cancel without a residue.  Every block has
            // its own exponents.  Twice over the scores in tensor memory, 32 keys at a time (the weights of some
            // lie where only scores did that were read before).
            const uint4 eb = *reinterpret_cast<const uint4*>(image_exps<D>(a, w, t) + 2);
            auto exponent = [](uint32_t lo, uint32_t hi, int b) { return int((b & 4 ? hi : lo) << (24 - 8 * (b & 3))) >> 24; };
            auto scores = [&](int y, float (&z)[32]) {
              uint32_t s[32];
              tc_ld32(tS + 32 * y, s);
              const uint32_t seen = (y >> 1 ? clear[1] : clear[0]) ? ~0u : seen_by(y >> 1, y & 1);
              tc_wait_ld();
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const int x2 = exponent(eb.x, eb.y, 2 * y + b) + fe;
                const float k1 = q8_pow2(x2 >> 1), k2 = q8_pow2(x2 - (x2 >> 1)) + (factor - factor);   // (no number: stays so)
#pragma unroll
                for (int k = 16 * b; k < 16 * b + 16; ++k) z[k] = seen >> k & 1u ? __uint_as_float(s[k]) * k1 * k2 : -INFINITY;
              }
            };
            float Rn = R, wn = -INFINITY, z[32];               // the largest score; of the blocks' weights, against Rn
#pragma unroll 1
            for (int y = 0; y < 4; ++y) {
              scores(y, z);
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                float top = -INFINITY;
#pragma unroll
                for (int k = 16 * b; k < 16 * b + 16; ++k) top = fmaxf(top, z[k]);
                if (top > Rn) {
                  wn += (Rn - top) * c;
                  Rn = top;
                }
                wn = fmaxf(wn, fmaf(top - Rn, c, float(exponent(eb.z, eb.w, 2 * y + b))));   // (nothing so far: the first)
              }
            }
            const float up = (Rn - R) * c;
            const bool over = R == -INFINITY ? Rn > R : up > kWeightTop || wn + up - h > kWeightTop;
            if (__any_sync(RQ_FULL_MASK, over)) raise(over, Rn, wn);
            const float r = R == -INFINITY ? 0.f : R;
#pragma unroll 1
            for (int y = 0; y < 4; ++y) {
              scores(y, z);
              uint32_t p[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const float a0 = (z[2 * k] - r) * c, a1 = (z[2 * k + 1] - r) * c;
                const float eh = float(exponent(eb.z, eb.w, 2 * y + k / 8)) - h;
                l += ex2(a0) + ex2(a1);
                p[k] = pack_half2(ex2(a0 + eh), ex2(a1 + eh));
              }
              tc_st16(tS + 16 * y, p);
              if (y & 1) weights_there(y >> 1);
            }
          }
        }
        if (!failed) {
          const int last_step = n0 + g;
          failed = !mbar_wait_bounded(step(last_step), (last_step >> 3) & 1, kWaitNs);
        }
        ++n0;
        failed = group_any(i, failed);                         // (the warps leave together: they share barriers)
        tc_fence_after();
      }
      // ---- results (a wait that gave up: NaN)
      const float nan = __int_as_float(0x7fc00000);
      const bool there = x.ok && !failed;                      // O holds the segment's sums
      const bool whole = w.kt0 == 0 && w.T == x.V;
      const bool valid = i * kRowTile + r < x.rows;
      if (!whole) {
        int first, last;
        w.sharers(a.prefix[int64_t(a.B) * a.blocks], *a.used, first, last);
        const int64_t at = (2 * int64_t(me) + (w.kt0 == 0)) * kBlockRows + i * kRowTile;
        float* const part = a.part + at * D;                   // [D / 4][128 rows][4]
        a.stats[at + r] = make_float4(R * c, h, there ? l : nan, 0.f);
#pragma unroll 1
        for (int y = 0; y < D / 32; ++y) {
          uint32_t o[32];
#pragma unroll
          for (int z = 0; z < 32; ++z) o[z] = 0u;
          if (there) {
            tc_ld32(tO + 32 * y, o);
            tc_wait_ld();
          }
          if (!valid) continue;
#pragma unroll
          for (int z = 0; z < 8; ++z)
            *reinterpret_cast<uint4*>(part + ((8 * y + z) * kRowTile + r) * 4) = make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
        }
        if (i == 0 && r == 0 && w.kt0 == 0)                     // (told by the CTA where the unit begins)
          a.parted[me] = {w.b, w.h, w.block * kBlockRows, x.rows, first, last};
        tc_fence_before();
        continue;
      }
      const float inv = there ? (l == 0.f ? 0.f : 1.f / l) : nan, up = ex2(0.5f * h);
      uint16_t* const out = a.c.out + ((int64_t(w.b) * a.c.n_new + row / a.G) * a.Hq + w.h * a.G + row % a.G) * D;
      const uintptr_t odd = reinterpret_cast<uintptr_t>(a.c.out) & 31;
#pragma unroll 1
      for (int y = 0; y < D / 32; ++y) {
        uint32_t o[32];
#pragma unroll
        for (int z = 0; z < 32; ++z) o[z] = 0u;
        if (there) {
          tc_ld32(tO + 32 * y, o);
          tc_wait_ld();
        }
        if (!valid) continue;
        uint4 q[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(o[8 * z + k]);
          q[z] = bf16_row(v, inv, up);
        }
        if (odd == 0) {                                        // (whole sectors)
          store32(out + 32 * y, q[0], q[1]);
          store32(out + 32 * y + 16, q[2], q[3]);
        } else {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            uint16_t* const to = out + 32 * y + 8 * z;
            if (odd == 16) {
              *reinterpret_cast<uint4*>(to) = q[z];
              continue;
            }
            const uint32_t u[4] = {q[z].x, q[z].y, q[z].z, q[z].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              to[2 * k] = uint16_t(u[k]);
              to[2 * k + 1] = uint16_t(u[k] >> 16);
            }
          }
        }
      }
      tc_fence_before();
    }
  }
  if (__syncthreads_or(failed) && threadIdx.x == 0) atomicOr(a.err, 1u);
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tc_free(tmem, 512);
}

// The divided units: a CTA joins 32 rows of one, a thread 16 channels of a row, its parts in order and the
// loads of four at a time.  A part's m is st.x (-inf: nothing seen), h st.y, l st.z.
template <int D>
__global__ void __launch_bounds__(2 * D) q8_join_kernel(const __grid_constant__ RowsArgs a) {
  grid_wait();
  const Parted u = a.parted[blockIdx.x];
  const int row = int(blockIdx.y) * 32 + (threadIdx.x & 31), y = threadIdx.x >> 5;
  if (row >= u.rows) return;
  const int tile = row / kRowTile * kRowTile, r = row % kRowTile;
  auto place = [&](int k) { return (2 * int64_t(k) + (k == u.first)) * kBlockRows + tile; };
  Join x = Join::none();
  float o[16];
#pragma unroll
  for (int z = 0; z < 16; ++z) o[z] = 0.f;
  for (int k = u.first; k <= u.last; k += 4) {
    float4 st[4], v[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      st[e] = make_float4(-INFINITY, float(kNoScale), 0.f, 0.f);
      if (k + e > u.last) continue;
      st[e] = a.stats[place(k + e) + r];
      const float4* const part = reinterpret_cast<const float4*>(a.part + place(k + e) * D) + 4 * y * kRowTile + r;
#pragma unroll
      for (int z = 0; z < 4; ++z) v[e][z] = part[z * kRowTile];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (k + e > u.last) continue;
      const float to = fmaxf(x.M, st[e].x);
      x.sum = fmaf(ex2(st[e].x - to), st[e].z, x.sum * ex2(x.M - to));   // (a part that gave up is NaN)
      x.M = to;
      const float f0 = x.raise(st[e].x, st[e].y), f = x.factor(st[e].x, st[e].y);
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        o[4 * z] = fmaf(f, v[e][z].x, o[4 * z] * f0);
        o[4 * z + 1] = fmaf(f, v[e][z].y, o[4 * z + 1] * f0);
        o[4 * z + 2] = fmaf(f, v[e][z].z, o[4 * z + 2] * f0);
        o[4 * z + 3] = fmaf(f, v[e][z].w, o[4 * z + 3] * f0);
      }
    }
  }
  const float inv = x.inverse(), up = ex2(0.5f * x.unit());
  const int j = (u.r0 + row) / a.G, hq = u.h * a.G + (u.r0 + row) % a.G;
  uint16_t* const to = a.c.out + ((int64_t(u.b) * a.c.n_new + j) * a.Hq + hq) * D + 16 * y;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    float w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = o[8 * z + k];
    const uint4 q = bf16_row(w, inv, up);
    if ((reinterpret_cast<uintptr_t>(a.c.out) & 15) == 0) {
      *reinterpret_cast<uint4*>(to + 8 * z) = q;
    } else {
      const uint32_t p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        to[8 * z + 2 * k] = uint16_t(p[k]);
        to[8 * z + 2 * k + 1] = uint16_t(p[k] >> 16);
      }
    }
  }
}

// Key tiles of one unit's list, at most.
template <typename Shape>
int rows_list(const Shape& s, int n_new, int max_ctx, int window, int n_sink) {
  int64_t slots = std::min<int64_t>(int64_t(max_ctx) + n_new, s.capacity), tiles = (slots + 63) / 64;
  if (window > 0)      // sinks, the window and the new tokens, each from an edge of its own
    tiles = std::min<int64_t>(tiles, (int64_t(n_sink) + 63) / 64 + (int64_t(window) + n_new + 63) / 64 + 1);
  return int((tiles + 1) / 2);
}

struct RowsPlan {
  Q8Layout line;
  int list, row_tiles, group;   // sequences handled together
  size_t images, queries;       // bytes of a sequence's operand tiles
  size_t total;
};

constexpr size_t kGroupBytes = size_t(2) << 30;   // operand tiles of the sequences handled together

RowsPlan rows_plan(const rq_q8_shape& s, int n_new, int max_ctx, int window, int n_sink) {
  RowsPlan p = {};
  p.line = q8_layout(s, n_new, max_ctx, kBlockRows, kKeys, std::min(device_sm_count(), kMostCtas));
  p.total = p.line.total;
  const int64_t rows = int64_t(n_new) * (s.n_q_heads / s.n_kv_heads);
  p.list = rows_list(s, n_new, max_ctx, window, n_sink);
  p.row_tiles = int((rows + kRowTile - 1) / kRowTile);
  const bool wide = s.head_dim == 128;
  p.images = size_t(s.n_kv_heads) * p.list * (wide ? RowsSmem<128>::kImage : RowsSmem<64>::kImage);
  p.queries = size_t(s.n_kv_heads) * p.row_tiles * (wide ? RowsSmem<128>::kQueryImage : RowsSmem<64>::kQueryImage);
  const size_t per = p.images + p.queries;
  p.group = int(std::max<size_t>(1, std::min<size_t>(s.batch, kGroupBytes / per)));
  p.total += std::min(per * size_t(s.batch), std::max(per, kGroupBytes));
  return p;
}

template <int D, int FMT>
cudaError_t launch(const RowsArgs& a, cudaStream_t stream) {
  using L = RowsSmem<D>;
  static OncePerDevice once;
  cudaError_t e = once([] {
    return cudaFuncSetAttribute(q8_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
  });
  if (e != cudaSuccess) return e;
  q8_query_kernel<D><<<1 + unsigned(a.B) * a.v.H * unsigned(a.row_tiles) * kQueryParts, 256, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after(true, q8_image_kernel<D, FMT>, dim3(unsigned(a.B) * a.v.H * unsigned(a.list)), 256, 0, stream, a);
  if (e != cudaSuccess) return e;
  if ((e = launch_after(true, q8_rows_kernel<D>, dim3(unsigned(a.n_ctas)), 384, L::total, stream, a)) != cudaSuccess) return e;
  const int rows = int(std::min<int64_t>(kBlockRows, int64_t(a.c.n_new) * a.G));
  return launch_after(true, q8_join_kernel<D>, dim3(unsigned(a.n_ctas), unsigned((rows + 31) / 32)), 2 * D, 0, stream, a);
}

}  // namespace

size_t q8_rows_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx, int window, int n_sink) {
  return rows_plan(s, n_new, max_ctx, window, n_sink).total;
}

cudaError_t launch_q8_rows(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                           const Q8Call& c, void* ws, cudaStream_t stream) {
  const RowsPlan p = rows_plan(s, c.n_new, c.max_ctx, c.window, c.n_sink);
  RowsArgs a = {};
  static_cast<Q8Line&>(a) = q8_line(s, cache, paging, c, kBlockRows);
  q8_place(a, p.line, ws);
  a.least = 2;
  a.images = static_cast<uint8_t*>(ws) + p.line.total;
  a.list = p.list;
  a.row_tiles = p.row_tiles;
  a.queries = a.images + p.images * size_t(p.group);
  for (int b0 = 0; b0 < s.batch; b0 += p.group) {            // (a group's kernels use the workspace after the one before)
    RowsArgs g = a;
    g.B = std::min(p.group, s.batch - b0);
    g.clear = b0 == 0;
    g.c.q += b0 * c.q_strides[0];
    g.c.out += int64_t(b0) * c.n_new * s.n_q_heads * s.head_dim;
    g.c.ctx_lens += b0;
    if (c.n_lens) g.c.n_lens += b0;
    if (c.rope.positions) g.c.rope.positions += int64_t(b0) * c.n_new;
    if (paging) {
      g.v.bt += int64_t(b0) * g.v.max_pages;
    } else {
      const int64_t records = int64_t(b0) * g.v.H * g.v.tiles;
      g.v.codes += records * g.v.rec_codes;
      g.v.scales += records * g.v.rec_scales;
    }
    cudaError_t e;
    if (s.head_dim == 128)
      e = s.format == RQ_Q8_INT8 ? launch<128, RQ_Q8_INT8>(g, stream) : launch<128, RQ_Q8_E4M3>(g, stream);
    else
      e = s.format == RQ_Q8_INT8 ? launch<64, RQ_Q8_INT8>(g, stream) : launch<64, RQ_Q8_E4M3>(g, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// -------------------------------------------------------------------------------- both kernels

namespace {

// Rows of a kv-head from which the tensor-core kernel is taken.
constexpr int64_t kManyRows = 33;

int64_t rows_of_call(const rq_q8_shape& s, int n_new) { return int64_t(n_new) * (s.n_q_heads / s.n_kv_heads); }

}  // namespace

// What a call takes, and never less than any call with fewer new tokens or a shorter context: few rows
// may need more, as more CTAs share them.
size_t q8_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx, int window, int n_sink) {
  size_t most = 0;
  const int heads = s.n_q_heads / s.n_kv_heads;
  for (int rows : {8, 16, 32}) {
    const int n = std::min(n_new, std::max(1, rows / heads));
    if (rows_of_call(s, n) < kManyRows) most = std::max(most, q8_stream_workspace_bytes(s, n, max_ctx));
  }
  if (rows_of_call(s, n_new) >= kManyRows) most = std::max(most, q8_rows_workspace_bytes(s, n_new, max_ctx, window, n_sink));
  return most;
}

cudaError_t launch_q8_attention(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                                const Q8Call& c, void* ws, cudaStream_t stream) {
  return rows_of_call(s, c.n_new) >= kManyRows ? launch_q8_rows(s, cache, paging, c, ws, stream)
                                               : launch_q8_stream(s, cache, paging, c, ws, stream);
}

}  // namespace rq
