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
// score's fp32 scale).  Collected weights need more: their scores take K as two fp16 parts.
#include "rq_common.cuh"
#include "rq_kernels.h"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr int kKeys = 128;                 // keys per tile (two cache records)
constexpr int kRows = 128;                 // query rows per tile
constexpr float kStateMax = 65504.f;
constexpr float kSlack = 8.f;              // log2 units a maximum may grow before O is rescaled
constexpr uint64_t kTcWaitLimitNs = 2000000000ull;

__device__ __forceinline__ float code_float(uint32_t code) {   // exact integer below 2^23
  return __uint_as_float(0x4B000000u | code) - 8388608.f;
}

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
  int b0, H, heads, n_new, max_ctx, window, tiles;   // tiles: key tiles per (sequence, head)
};

__device__ __forceinline__ bool lens_of(const ChunkView& v, int b, int& n, int& ctx) {
  n = v.n_lens ? v.n_lens[b] : v.n_new;
  ctx = v.ctx_lens[b];
  return n >= 0 && n <= v.n_new && ctx >= 0 && ctx <= v.max_ctx;
}

// ---------------------------------------------------------------------------------- rebuild

struct RebuildArgs {
  ChunkView v;
  const uint8_t* data;
  int64_t rec_bytes;
  const int32_t* bt;
  int max_pages, n_pages, cap;
  int bits, sec_off;             // residual bits (0: final loop), offset of the loop's section
  const int8_t* signs[2];
  const uint16_t* kv_new;
  int64_t ks0, ks1, kv_v, ks_h;
  uint8_t *k, *klo, *val;        // images [unit][tile][...]; klo may be null
};

// Codes of one token's row -> x[ch] = fma(step, code, offset-term): ADD adds to x.
template <int D, int BITS, bool V, bool ADD>
__device__ __forceinline__ void add_level(const uint8_t* codes, const uint8_t* meta, int r, float a,
                                          float (&x)[D]) {
  constexpr int NG = D / 32, RB = D * BITS / 8;
  float s[NG], z[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const float2 m = __half22float2(*reinterpret_cast<const __half2*>(meta + (r * NG + g) * 4));
    s[g] = m.x * a;
    z[g] = m.y * a;
  }
  auto put = [&](int ch, uint32_t code) {
    const int g = ch / 32;
    x[ch] = fmaf(s[g], code_float(code), ADD ? x[ch] + z[g] : z[g]);
  };
  constexpr uint32_t MASK = (1u << BITS) - 1u;
  if constexpr (!V) {   // words group-interleaved: word s holds channels of group s % NG
    constexpr int PER = 32 / BITS;
#pragma unroll
    for (int w = 0; w < RB / 4; ++w) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(codes + r * RB + w * 4);
#pragma unroll
      for (int i = 0; i < PER; ++i) put((w % NG) * 32 + (w / NG) * PER + i, (word >> (i * BITS)) & MASK);
    }
  } else {              // token pairs: unit u at word u ^ swizzle, this token's half
    constexpr int PER = 16 / BITS, UNITS = RB / 2;
    const int p = r >> 1;
    const uint8_t* row = codes + p * 2 * RB + (r & 1) * 2;
    const int sw = v_unit_swizzle(p, UNITS);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const uint32_t unit = *reinterpret_cast<const uint16_t*>(row + (u ^ sw) * 4);
#pragma unroll
      for (int i = 0; i < PER; ++i) put(u * PER + i, (unit >> (i * BITS)) & MASK);
    }
  }
}

template <int D, bool V>
__device__ __forceinline__ void rebuild_row(const uint8_t* sec, int bits, const float* sign, int r,
                                            float (&x)[D]) {
  constexpr int NG = D / 32;
  constexpr int REF = kTile * (D / 2 + 4 * NG);             // bytes of one side of the reference
  const uint8_t* ref = sec + (V ? REF : 0);
  if (bits == 0) {
    add_level<D, 4, V, false>(ref, ref + kTile * D / 2, r, 1.f, x);
    return;
  }
  const int rb = D * bits / 8, side = kTile * (rb + 4 * NG + 2);
  const uint8_t* res = sec + 2 * REF + (V ? side : 0);
  const float a = __half2float(*reinterpret_cast<const __half*>(res + kTile * (rb + 4 * NG) + r * 2));
  if (bits == 2)
    add_level<D, 2, V, false>(res, res + kTile * rb, r, 1.f, x);
  else
    add_level<D, 4, V, false>(res, res + kTile * rb, r, 1.f, x);
#pragma unroll
  for (int h = 1; h < D; h <<= 1)
#pragma unroll
    for (int i = 0; i < D; ++i)
      if ((i & h) == 0) {
        const float u = x[i], w = x[i + h];
        x[i] = u + w;
        x[i + h] = u - w;
      }
#pragma unroll
  for (int i = 0; i < D; i += 4) {
    const float4 sg = *reinterpret_cast<const float4*>(sign + i);
    x[i] *= sg.x;
    x[i + 1] *= sg.y;
    x[i + 2] *= sg.z;
    x[i + 3] *= sg.w;
  }
  add_level<D, 4, V, true>(ref, ref + kTile * D / 2, r, a, x);
}

template <int D>
constexpr int rebuild_smem() {   // sections, signs, images, barrier
  return kTile * (D + 8 * (D / 32)) + kTile * (D + 8 * (D / 32) + 4) + 2 * D * 4 + 3 * 64 * D * 2 + 16;
}

// One CTA per 64 keys of a (sequence, kv-head): a thread per key and side (K, V) holds the row's
// D channels in registers, so the Hadamard transform needs no exchange.  Bound by instruction
// issue (about 2,200 per row) together with HBM (one loop's record read, 4 D bytes written).
template <int D>
__global__ void __launch_bounds__(128) rebuild_kernel(const __grid_constant__ RebuildArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int NG = D / 32;
  constexpr int REF = kTile * (D + 8 * NG);
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  int n, ctx;
  if (!lens_of(a.v, b, n, ctx)) {
    if (threadIdx.x == 0) atomicOr(a.v.err, 1u);
    return;
  }
  const int t0 = blockIdx.x * kTile, total = n > 0 ? ctx + n : 0;
  if (t0 >= (total + kKeys - 1) / kKeys * kKeys) return;
  uint8_t* const img_k = smem;
  uint8_t* const img_lo = smem + 64 * D * 2;
  uint8_t* const img_v = smem + 2 * 64 * D * 2;
  float* const sign = reinterpret_cast<float*>(smem + 3 * 64 * D * 2);      // [2][D]
  uint8_t* const sec = smem + 3 * 64 * D * 2 + 2 * D * 4;
  uint64_t* const bar = reinterpret_cast<uint64_t*>(sec + REF + kTile * (D + 8 * NG + 4));
  const bool cached = t0 < ctx;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(bar), 1);
    fence_mbar_init();
    if (cached) {
      int64_t rec;
      if (a.bt) {
        int pg = a.bt[int64_t(b) * a.max_pages + blockIdx.x];
        if (pg < 0 || pg >= a.n_pages) {
          atomicOr(a.v.err, 1u);
          pg = 0;
        }
        rec = int64_t(pg) * a.v.H + h;
      } else {
        rec = (int64_t(b) * a.v.H + h) * (a.cap / kTile) + blockIdx.x;
      }
      const uint8_t* src = a.data + rec * a.rec_bytes;
      const uint32_t res = a.bits ? uint32_t(loop_section_bytes(D, a.bits)) : 0u;
      mbar_arrive_expect_tx(smem_u32(bar), uint32_t(REF) + res);
      bulk_g2s(smem_u32(sec), src, uint32_t(REF), smem_u32(bar));
      if (res) bulk_g2s(smem_u32(sec + REF), src + a.sec_off, res, smem_u32(bar));
    }
  }
  const float inv_sqrt_d = (D == 128) ? 0.08838834764831845f : 0.125f;
  for (int i = threadIdx.x; i < 2 * D; i += 128)
    sign[i] = float(a.signs[i / D][int64_t(h) * D + i % D]) * inv_sqrt_d;
  __syncthreads();
  const bool arrived = !cached || mbar_wait_bounded(smem_u32(bar), 0, kTcWaitLimitNs);
  if (!arrived) atomicOr(a.v.err, 1u);
  const bool is_v = threadIdx.x >= 64;
  const int r = threadIdx.x & 63, t = t0 + r;
  float x[D];
  if (t < ctx && arrived) {
    if (is_v)
      rebuild_row<D, true>(sec, a.bits, sign + D, r, x);
    else
      rebuild_row<D, false>(sec, a.bits, sign, r, x);
  } else if (t >= ctx && t < total) {
    const uint16_t* p = a.kv_new + b * a.ks0 + (t - ctx) * a.ks1 + h * a.ks_h + (is_v ? a.kv_v : 0);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < D; ++i) {
      x[i] = bf16_bits_to_float(p[i]);
      bad |= !(fabsf(x[i]) <= kStateMax);
    }
    if (bad) {   // its own and later rows become NaN; the image keeps a zero row
      atomicMin(a.v.first_bad + int64_t(b) * a.v.H + h, t - ctx);
#pragma unroll
      for (int i = 0; i < D; ++i) x[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < D; ++i) x[i] = 0.f;
  }
  if (!is_v) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = x[8 * c + 2 * k], x1 = x[8 * c + 2 * k + 1];
        hi[k] = half2_sat(x0, x1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[k]));
        lo[k] = half2_sat(x0 - f.x, x1 - f.y);
      }
      const uint32_t o = (c / 8) * (64 * 128) + panel_offset(r, c % 8);
      *reinterpret_cast<uint4*>(img_k + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (a.klo) *reinterpret_cast<uint4*>(img_lo + o) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  } else {   // transposed: panel row = channel, column = key
#pragma unroll
    for (int d = 0; d < D; d += 2) {
      const uint32_t w = half2_sat(x[d], x[d + 1]);
      *reinterpret_cast<uint16_t*>(img_v + panel_offset(d, r >> 3) + (r & 7) * 2) = uint16_t(w);
      *reinterpret_cast<uint16_t*>(img_v + panel_offset(d + 1, r >> 3) + (r & 7) * 2) = uint16_t(w >> 16);
    }
  }
  fence_async_smem();
  __syncthreads();
  if (threadIdx.x == 0) {
    const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
    const int tile = blockIdx.x >> 1, half = blockIdx.x & 1;
    const int64_t at = (unit * a.v.tiles + tile) * (kKeys * D * 2);
#pragma unroll
    for (int p = 0; p < D / 64; ++p) {
      const int64_t o = at + p * (kKeys * 128) + half * (64 * 128);
      bulk_s2g(a.k + o, smem_u32(img_k + p * 64 * 128), 64 * 128);
      if (a.klo) bulk_s2g(a.klo + o, smem_u32(img_lo + p * 64 * 128), 64 * 128);
    }
    bulk_s2g(a.val + at + half * (D * 128), smem_u32(img_v), D * 128);
    bulk_s2g_commit_wait();
  }
}

// -------------------------------------------------------------------------------- attention

struct AttnArgs {
  ChunkView v;
  const uint16_t* q;
  int64_t qs0, qs1, qs2;
  const uint8_t *k, *klo, *val;
  uint16_t* out;
  float* part;             // [unit][row][split][4 + D] (m, l, pad, O), or null: one split
  float2* stats;           // (LSE) [unit][row][split] (m, l)
  int n_splits, max_rows;  // max_rows: rows of a unit (n_new * heads, or the window's)
  float scale_log2;
};

template <int D>
struct AttnSmem {
  static constexpr int kTileBytes = kKeys * D * 2;      // one K, V^T or Q tile
  static constexpr int q = 0, k = 2 * kTileBytes, v = k + 2 * kTileBytes, bars = v + 2 * kTileBytes;
  static constexpr int total = bars + 256 + 1024;       // + alignment of the base
};

// Load a row of queries, scale it by a power of two so that its largest element lies in
// [2^14, 2^15), store it as fp16 in a swizzled tile image.  Returns the exponent undone later.
template <int D>
__device__ __forceinline__ int store_query(const uint16_t* qp, bool valid, uint8_t* img, int r) {
  float mx = 0.f;
  uint32_t w[D / 2];
#pragma unroll
  for (int i = 0; i < D / 2; ++i) {
    w[i] = valid ? uint32_t(qp[2 * i]) | (uint32_t(qp[2 * i + 1]) << 16) : 0u;
    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
  }
  int e = 0;
  if (mx > 0.f && mx < INFINITY) {
    frexpf(mx, &e);
    e = 15 - e;
    e = e > 100 ? 100 : e;        // (tiny rows: the scores vanish either way)
  }
  const float up = ldexpf(1.f, e > 60 ? 60 : e), up2 = ldexpf(1.f, e > 60 ? e - 60 : 0);
#pragma unroll
  for (int c = 0; c < D / 8; ++c) {
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = w[4 * c + k];
      o[k] = pack_half2(__uint_as_float(x << 16) * up * up2, __uint_as_float(x & 0xffff0000u) * up * up2);
    }
    *reinterpret_cast<uint4*>(img + (c / 8) * (kRows * 128) + panel_offset(r, c % 8)) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
  return e;
}

// Two tiles of 128 query rows per CTA share every K and V tile.  Warps 0-3 and 4-7: softmax of
// tile 0 and 1, a thread per row; warp 8: copies; warp 9: products.  While one tile's softmax
// runs, the other's products do:  S_0 S_1 | P_0 V, S_0' | P_1 V, S_1' | ...
// The running maximum m is raised only when a tile exceeds it by 2^8 (O is rescaled in tensor
// memory then; P stays below 2^8); P overwrites S's columns.
// LSE: scores with K in two parts, no P and V; (m, l) per row and split are stored.
template <int D, bool LSE>
__global__ void __launch_bounds__(320, 1) attention_kernel(const __grid_constant__ AttnArgs a) {
  extern __shared__ uint8_t raw[];
  using L = AttnSmem<D>;
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  // barriers: K full/free [2], V full/free [2], S ready [2], P ready [2], Q ready, done
  const uint32_t bar0 = smem_u32(bars);
  auto kfull = [&](int s) { return bar0 + 8 * s; };
  auto kfree = [&](int s) { return bar0 + 8 * (2 + s); };
  auto vfull = [&](int s) { return bar0 + 8 * (4 + s); };
  auto vfree = [&](int s) { return bar0 + 8 * (6 + s); };
  auto sready = [&](int i) { return bar0 + 8 * (8 + i); };
  auto pready = [&](int i) { return bar0 + 8 * (10 + i); };
  const uint32_t qready = bar0 + 8 * 12, done = bar0 + 8 * 13;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 14);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
  const int split = blockIdx.x % a.n_splits;
  const int block = int(gridDim.x / a.n_splits) - 1 - int(blockIdx.x / a.n_splits);   // long rows first
  int n, ctx;
  // (one thread reads the error word: another CTA may be setting it)
  const bool flagged = __syncthreads_or(threadIdx.x == 0 && *reinterpret_cast<volatile unsigned*>(a.v.err) != 0u);
  const bool ok = lens_of(a.v, b, n, ctx) && !flagged;
  if (!ok) n = a.v.n_lens ? (n < 0 || n > a.v.n_new ? a.v.n_new : n) : a.v.n_new;
  const int first = LSE ? max(0, n - a.v.window) * a.v.heads : 0;   // first row of the unit's rows
  const int rows = n * a.v.heads - first;
  const int r0 = block * 2 * kRows;
  if (r0 >= rows) return;
  const bool two = r0 + kRows < rows;                               // the second tile has rows
  // key tiles of this split: of those up to the block's last row's own token
  const int j_last = (min(r0 + 2 * kRows, rows) - 1 + first) / a.v.heads;
  const int n_tiles = ok ? (ctx + j_last + kKeys) / kKeys : 0;
  const int kt0 = int(int64_t(split) * n_tiles / a.n_splits), kt1 = int(int64_t(split + 1) * n_tiles / a.n_splits);
  const int T = kt1 - kt0;

  if (warp == 9) tc_alloc(smem_u32(tslot), 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i) mbar_init(bar0 + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sready(i), 1);
      mbar_init(pready(i), kRows);
    }
    mbar_init(qready, 2 * kRows);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 384};
  bool failed = false;
  float m = -INFINITY, l = 0.f, c = 0.f;

  if (T > 0) {
    if (warp == 8) {
      if (lane == 0) {                                               // ---- copies
        const uint8_t* k = a.k + (unit * a.v.tiles + kt0) * L::kTileBytes;
        const uint8_t* v = (LSE ? a.klo : a.val) + (unit * a.v.tiles + kt0) * L::kTileBytes;
        int issued = 0;
        for (int j = 0; j < T; ++j, ++issued) {
          const int s = j & 1;
          if (j >= 2 && !(mbar_wait_bounded(kfree(s), ((j >> 1) - 1) & 1, kTcWaitLimitNs))) break;
          mbar_arrive_expect_tx(kfull(s), L::kTileBytes);
          bulk_g2s(smem_u32(smem + L::k + s * L::kTileBytes), k + int64_t(j) * L::kTileBytes, L::kTileBytes, kfull(s));
          if (j >= 2 && !(mbar_wait_bounded(vfree(s), ((j >> 1) - 1) & 1, kTcWaitLimitNs))) {
            mbar_wait_bounded(kfull(s), (j >> 1) & 1, kTcWaitLimitNs);
            break;
          }
          mbar_arrive_expect_tx(vfull(s), L::kTileBytes);
          bulk_g2s(smem_u32(smem + L::v + s * L::kTileBytes), v + int64_t(j) * L::kTileBytes, L::kTileBytes, vfull(s));
        }
        failed = issued < T;
        for (int j = max(0, issued - 2); j < issued; ++j) {          // no copy outlives the CTA
          failed |= !mbar_wait_bounded(kfull(j & 1), (j >> 1) & 1, kTcWaitLimitNs);
          failed |= !mbar_wait_bounded(vfull(j & 1), (j >> 1) & 1, kTcWaitLimitNs);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      if (lane == 0) {                                               // ---- products
        constexpr uint32_t ids = f16_idesc(kRows, kKeys), ido = f16_idesc(kRows, D);
        auto scores = [&](int i, int s) {
          const uint32_t q = smem_u32(smem + L::q + i * L::kTileBytes), k = smem_u32(smem + L::k + s * L::kTileBytes);
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            tc_mma(tS[i], panel_desc(q + (x / 4) * (kRows * 128) + (x % 4) * 32),
                   panel_desc(k + (x / 4) * (kKeys * 128) + (x % 4) * 32), ids, x > 0);
          if (LSE) {
            const uint32_t k2 = smem_u32(smem + L::v + s * L::kTileBytes);
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              tc_mma(tS[i], panel_desc(q + (x / 4) * (kRows * 128) + (x % 4) * 32),
                     panel_desc(k2 + (x / 4) * (kKeys * 128) + (x % 4) * 32), ids, true);
          }
          tc_commit(sready(i));
        };
        auto values = [&](int i, int s, bool add) {
          const uint32_t v = smem_u32(smem + L::v + s * L::kTileBytes);
#pragma unroll
          for (int x = 0; x < kKeys / 16; ++x)
            tc_mma_ta(tO[i], tS[i] + 8 * x, panel_desc(v + (x / 4) * (D * 128) + (x % 4) * 32), ido, add || x > 0);
        };
        const int I = two ? 2 : 1;
        bool good = mbar_wait_bounded(qready, 0, kTcWaitLimitNs) && mbar_wait_bounded(kfull(0), 0, kTcWaitLimitNs) &&
                    (!LSE || mbar_wait_bounded(vfull(0), 0, kTcWaitLimitNs));
        tc_fence_after();
        if (good) {
          for (int i = 0; i < I; ++i) scores(i, 0);
          tc_commit(kfree(0));
          if (LSE) tc_commit(vfree(0));
        }
        for (int j = 0; j < T && good; ++j) {
          const int s = j & 1;
          if (!LSE) good = mbar_wait_bounded(vfull(s), (j >> 1) & 1, kTcWaitLimitNs);
          for (int i = 0; i < I && good; ++i) {
            good = mbar_wait_bounded(pready(i), j & 1, kTcWaitLimitNs);
            if (!good) break;
            tc_fence_after();
            if (!LSE) values(i, s, j > 0);
            if (j + 1 < T) {
              const int s1 = s ^ 1;
              if (i == 0)
                good = mbar_wait_bounded(kfull(s1), ((j + 1) >> 1) & 1, kTcWaitLimitNs) &&
                       (!LSE || mbar_wait_bounded(vfull(s1), ((j + 1) >> 1) & 1, kTcWaitLimitNs));
              if (good) scores(i, s1);
            }
          }
          if (good && !LSE) tc_commit(vfree(s));
          if (good && j + 1 < T) {
            tc_commit(kfree(s ^ 1));
            if (LSE) tc_commit(vfree(s ^ 1));
          }
        }
        tc_commit(done);
        failed = !good;
        if (!good) mbar_wait_bounded(done, 0, kTcWaitLimitNs);       // nothing in flight
      }
      __syncwarp();
    } else {                                                         // ---- softmax
      const int i = warp >> 2, r = threadIdx.x & (kRows - 1);
      const int row = r0 + i * kRows + r;
      const bool valid = row < rows;
      const int arow = row + first, j = min(arow / a.v.heads, n - 1), g = arow % a.v.heads;
      const uint16_t* qp = a.q + b * a.qs0 + j * a.qs1 + (int64_t(h) * a.v.heads + g) * a.qs2;
      const int e = store_query<D>(qp, valid, smem + L::q + i * L::kTileBytes, r);
      c = ldexpf(a.scale_log2, -e);
      fence_async_smem();
      mbar_arrive(qready);
      const uint32_t lanes = uint32_t(warp & 3) << 21;               // this warp's tensor-memory lanes
      const int lim = ctx + j;                                       // last key the row sees
      const int j_first = min((r0 + i * kRows + first) / a.v.heads, n - 1);
      const int clear = ctx + j_first;                               // every row of the tile sees these
      if (i == 0 || two) {
        for (int jt = 0; jt < T; ++jt) {
          if (!mbar_wait_bounded(sready(i), jt & 1, kTcWaitLimitNs)) {
            failed = true;
            break;
          }
          tc_fence_after();
          uint32_t s[kKeys];
#pragma unroll
          for (int x = 0; x < 4; ++x) tc_ld32(tS[i] + lanes + 32 * x, s + 32 * x);
          tc_wait_ld();
          const int key0 = (kt0 + jt) * kKeys;
          if (key0 + kKeys - 1 > clear) {
            const int rel = lim - key0;
#pragma unroll
            for (int x = 0; x < kKeys; ++x)
              if (x > rel) s[x] = 0xff800000u;
          }
          float mx[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) mx[x] = __uint_as_float(s[x]);
#pragma unroll
          for (int x = 4; x < kKeys; ++x) mx[x & 3] = fmaxf(mx[x & 3], __uint_as_float(s[x]));
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          if (__any_sync(RQ_FULL_MASK, mt > m + kSlack)) {
            const float mn = mt > m + kSlack ? mt : m;
            const float f = m == -INFINITY ? 0.f : ex2(m - mn);
            l *= f;
            m = mn;
            if (!LSE && jt > 0) {
#pragma unroll
              for (int x = 0; x < D / 32; ++x) {
                uint32_t o[32];
                tc_ld32(tO[i] + lanes + 32 * x, o);
                tc_wait_ld();
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tc_st32(tO[i] + lanes + 32 * x, o);
              }
            }
          }
          const float ms = m == -INFINITY ? 0.f : -m;
          const uint64_t c2 = pack2(c, c), m2 = pack2(ms, ms);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t p[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int k = half * 64 + 2 * x;
              float p0, p1;
              unpack2(fma2(pack2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), c2, m2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[x & 1] = add2(sum[x & 1], pack2(p0, p1));
              if (!LSE) p[x] = pack_half2(p0, p1);
            }
            if (!LSE) tc_st32(tS[i] + lanes + 32 * half, p);
          }
          float s0, s1;
          unpack2(add2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          if (!LSE) tc_wait_st();
          tc_fence_before();
          mbar_arrive(pready(i));
        }
        if (!LSE && !failed) failed = !mbar_wait_bounded(done, 0, kTcWaitLimitNs);
      }
    }
  }
  const bool gave_up = __syncthreads_or(failed);
  if (gave_up && threadIdx.x == 0) atomicOr(a.v.err, 1u);
  if (warp < 8) {                                                    // ---- store
    const int i = warp >> 2;
    const int row = r0 + i * kRows + (threadIdx.x & (kRows - 1));
    const bool valid = row < rows;
    const uint32_t lanes = uint32_t(warp & 3) << 21;
    const float nan = __int_as_float(0x7fc00000);
    const int arow = row + first, j = arow / a.v.heads, g = arow % a.v.heads;
    const bool bad = !ok || gave_up || (valid && j >= a.v.first_bad[int64_t(b) * a.v.H + h]);
    if (LSE) {
      if (valid) a.stats[(unit * a.max_rows + row) * a.n_splits + split] = bad ? make_float2(nan, nan) : make_float2(m, l);
    } else if (i == 0 || two) {
      tc_fence_after();
      float* const part = a.part + ((unit * a.max_rows + row) * a.n_splits + split) * (4 + D);
      if (a.part && valid) *reinterpret_cast<float2*>(part) = bad ? make_float2(0.f, nan) : make_float2(m, l);
      const float inv = bad ? nan : 1.f / l;
      uint16_t* const o = a.out + ((int64_t(b) * a.v.n_new + j) * a.v.H * a.v.heads + h * a.v.heads + g) * D;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        uint32_t w[32];
        if (T > 0 && !gave_up) {
          tc_ld32(tO[i] + lanes + 32 * x, w);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) w[y] = 0u;
        }
        if (!valid) continue;
        if (a.part) {
#pragma unroll
          for (int y = 0; y < 32; y += 4)
            *reinterpret_cast<uint4*>(part + 4 + 32 * x + y) = make_uint4(w[y], w[y + 1], w[y + 2], w[y + 3]);
        } else {
#pragma unroll
          for (int y = 0; y < 32; y += 8) {
            uint32_t p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(__uint_as_float(w[y + 2 * k]) * inv,
                                                            __uint_as_float(w[y + 2 * k + 1]) * inv);
              p[k] = *reinterpret_cast<const uint32_t*>(&v);
            }
            if ((reinterpret_cast<uintptr_t>(o) & 15) == 0) {
              *reinterpret_cast<uint4*>(o + 32 * x + y) = make_uint4(p[0], p[1], p[2], p[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                o[32 * x + y + 2 * k] = uint16_t(p[k]);
                o[32 * x + y + 2 * k + 1] = uint16_t(p[k] >> 16);
              }
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tc_free(tmem, 512);
}

// One warp per row: merge the splits' (m, l, O).
template <int D>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int P = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  if (wid >= a.max_rows) return;
  const int row = int(wid), j = row / a.v.heads, g = row % a.v.heads;
  int n = a.v.n_lens ? a.v.n_lens[b] : a.v.n_new;
  if (n < 0 || n > a.v.n_new) n = a.v.n_new;
  if (j >= n) return;
  const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
  const float* part = a.part + (unit * a.max_rows + row) * a.n_splits * (4 + D);
  float M = -INFINITY, l = 0.f, o[P];
#pragma unroll
  for (int i = 0; i < P; ++i) o[i] = 0.f;
  for (int s = 0; s < a.n_splits; ++s) M = fmaxf(M, part[int64_t(s) * (4 + D)]);
  for (int s = 0; s < a.n_splits; ++s) {
    const float* p = part + int64_t(s) * (4 + D);
    const float ms = p[0], ls = p[1];
    if (ms == -INFINITY) continue;
    const float f = ex2(ms - M);
    l = fmaf(f, ls, l);
#pragma unroll
    for (int i = 0; i < P; ++i) o[i] = fmaf(f, p[4 + lane * P + i], o[i]);
  }
  uint16_t* out = a.out + ((int64_t(b) * a.v.n_new + j) * a.v.H * a.v.heads + h * a.v.heads + g) * D + lane * P;
  const float inv = *reinterpret_cast<volatile unsigned*>(a.v.err) ? __int_as_float(0x7fc00000) : 1.f / l;
#pragma unroll
  for (int i = 0; i < P; ++i) out[i] = float_to_bf16_bits(o[i] * inv);
}

// ---------------------------------------------------------------------------------- weights

struct WeightArgs {
  ChunkView v;
  const uint16_t* q;
  int64_t qs0, qs1, qs2;
  const uint8_t *k, *klo;
  uint8_t* qimg;           // [unit][row tile][image of 128 rows]
  float2* scale;           // [unit][row]: (score scale, -log2-sum-exp); (0, -inf): no row
  const float2* stats;     // [unit][row][split]
  float* weights;
  int n_splits, max_rows, q_tiles, cap;
  float scale_log2;
};

// Operand images of the window's queries, each row's score scale and log2-sum-exp.
template <int D>
__global__ void __launch_bounds__(128) window_rows_kernel(const __grid_constant__ WeightArgs a) {
  extern __shared__ __align__(1024) uint8_t img[];
  const int h = blockIdx.y, b = a.v.b0 + blockIdx.z;
  const int64_t unit = int64_t(blockIdx.z) * a.v.H + h;
  int n, ctx;
  if (!lens_of(a.v, b, n, ctx)) return;
  const int first = max(0, n - a.v.window) * a.v.heads, rows = n * a.v.heads - first;
  const int row = blockIdx.x * kRows + threadIdx.x;
  if (int(blockIdx.x) * kRows >= rows) return;
  const bool valid = row < rows;
  const int arow = valid ? row + first : first;
  const int j = arow / a.v.heads, g = arow % a.v.heads;
  const int e = store_query<D>(a.q + b * a.qs0 + j * a.qs1 + (int64_t(h) * a.v.heads + g) * a.qs2, valid, img,
                               threadIdx.x);
  float2 sc = make_float2(0.f, -INFINITY);
  if (valid) {
    const float2* st = a.stats + (unit * a.max_rows + row) * a.n_splits;
    float M = -INFINITY, l = 0.f;
    for (int s = 0; s < a.n_splits; ++s) M = fmaxf(M, st[s].x);
    for (int s = 0; s < a.n_splits; ++s) {
      const float2 x = st[s];
      if (x.x != -INFINITY) l = fmaf(ex2(x.x - M), x.y, l);
    }
    sc = make_float2(ldexpf(a.scale_log2, -e), -(M + log2f(l)));
  }
  a.scale[unit * (int64_t(a.q_tiles) * kRows) + row] = sc;
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(a.qimg + (unit * a.q_tiles + blockIdx.x) * (kRows * D * 2));
  for (int i = threadIdx.x; i < kRows * D * 2 / 16; i += 128) dst[i] = reinterpret_cast<const uint4*>(img)[i];
}

template <int D>
struct WeightSmem {
  static constexpr int kTileBytes = kKeys * D * 2;
  static constexpr int kStages = 3;
  static constexpr int kStage = kTileBytes + kRows * 8;   // queries, scales
  static constexpr int k = 0, q = 2 * kTileBytes, bars = q + kStages * kStage;
  static constexpr int total = bars + 256 + 1024;
};

// One CTA per 128 keys: S^T = K Q^T with the keys as rows, so a key's weights add up in its
// thread's registers, in row order.  Row tiles alternate between two tensor-memory buffers and the
// two softmax warpgroups.  Bound by the exponentials.
template <int D>
__global__ void __launch_bounds__(320, 1) weights_kernel(const __grid_constant__ WeightArgs a) {
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
    for (int i = 0; i < 3; ++i) {
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
        const int s = j % 3;
        if (j >= 3 && !mbar_wait_bounded(qfree(s), (j / 3 - 1) & 1, kTcWaitLimitNs)) break;
        const uint32_t dst = smem_u32(smem + L::q + s * L::kStage);
        mbar_arrive_expect_tx(qfull(s), L::kStage);
        bulk_g2s(dst, a.qimg + (unit * a.q_tiles + from + j) * L::kTileBytes, L::kTileBytes, qfull(s));
        bulk_g2s(dst + L::kTileBytes, a.scale + (unit * a.q_tiles + from + j) * kRows, kRows * 8, qfull(s));
      }
      failed = issued < T || !mbar_wait_bounded(kfull, 0, kTcWaitLimitNs);
      for (int j = max(0, issued - 3); j < issued; ++j)
        failed |= !mbar_wait_bounded(qfull(j % 3), (j / 3) & 1, kTcWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (lane == 0) {
      constexpr uint32_t id = f16_idesc(kKeys, kRows);
      bool good = mbar_wait_bounded(kfull, 0, kTcWaitLimitNs);
      for (int j = 0; j < T && good; ++j) {
        const int s = j % 3, i = j & 1;
        good = mbar_wait_bounded(qfull(s), (j / 3) & 1, kTcWaitLimitNs) &&
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
    for (int j = i; j < T; j += 2) {
      const int s = j % 3;
      if (!mbar_wait_bounded(sready(i), (j >> 1) & 1, kTcWaitLimitNs) ||
          !mbar_wait_bounded(qfull(s), (j / 3) & 1, kTcWaitLimitNs)) {
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
          const float p0 = ex2(fmaf(__uint_as_float(v[y]), f.x, f.y));
          const float p1 = ex2(fmaf(__uint_as_float(v[y + 1]), f.z, f.w));
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
  int tiles, rows, wrows, q_tiles, splits, wsplits;
  size_t first_bad, k, klo, val, part, stats, qimg, scale, total;
};

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

TcLayout tc_layout(const rq_shape& s, int n_new, int max_ctx, int window) {
  TcLayout l;
  const int heads = s.n_q_heads / s.n_kv_heads, D = s.head_dim;
  l.tiles = int((int64_t(max_ctx) + n_new + kKeys - 1) / kKeys);
  l.rows = n_new * heads;
  l.wrows = window * heads;
  l.q_tiles = (l.wrows + kRows - 1) / kRows;
  const size_t tile = size_t(kKeys) * D * 2;
  const size_t seq = size_t(s.n_kv_heads) * l.tiles * tile * (window ? 3 : 2);
  const size_t fit = kGroupBytes / (seq ? seq : 1);
  l.group = int(fit < 1 ? 1 : (fit > size_t(s.batch) ? size_t(s.batch) : fit));
  const size_t units = size_t(l.group) * s.n_kv_heads;
  const int64_t ctas = int64_t(units) * ((l.rows + 2 * kRows - 1) / (2 * kRows));
  l.splits = plan_tc_splits(ctas, l.tiles);
  l.wsplits = window ? plan_tc_splits(int64_t(units) * ((l.wrows + 2 * kRows - 1) / (2 * kRows)), l.tiles) : 1;
  size_t o = kWsHeaderBytes;
  l.first_bad = o;
  o = round1k(o + size_t(s.batch) * s.n_kv_heads * 4);
  l.k = o;
  o += units * l.tiles * tile;
  l.val = o;
  o += units * l.tiles * tile;
  l.klo = o;
  if (window) o += units * l.tiles * tile;
  l.part = o;
  if (l.splits > 1) o = round1k(o + units * l.rows * l.splits * (4 + size_t(D)) * 4);
  l.stats = o;
  o = round1k(o + units * l.wrows * l.wsplits * 8);
  l.qimg = o;
  o += units * l.q_tiles * (size_t(kRows) * D * 2);
  l.scale = o;
  o = round1k(o + units * l.q_tiles * kRows * 8);
  l.total = o;
  return l;
}

template <int D>
cudaError_t launch_tc(const rq_shape& s, const rq_cache& cache, const rq_paging* paging, const ChunkCall& c,
                      char* w, cudaStream_t stream) {
  const TcLayout l = tc_layout(s, c.n_new, c.max_ctx, c.window);
  cudaError_t e;
  using AS = AttnSmem<D>;
  using WS = WeightSmem<D>;
  if ((e = cudaFuncSetAttribute(rebuild_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, rebuild_smem<D>())) != cudaSuccess ||
      (e = cudaFuncSetAttribute(attention_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, AS::total)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(attention_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, AS::total)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(weights_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, WS::total)) != cudaSuccess ||
      (e = cudaMemsetAsync(w + l.first_bad, 0x7f, size_t(s.batch) * s.n_kv_heads * 4, stream)) != cudaSuccess)
    return e;
  ChunkView v;
  v.n_lens = c.n_lens;
  v.ctx_lens = c.ctx_lens;
  v.err = reinterpret_cast<unsigned*>(w);
  v.first_bad = reinterpret_cast<int*>(w + l.first_bad);
  v.H = s.n_kv_heads;
  v.heads = s.n_q_heads / s.n_kv_heads;
  v.n_new = c.n_new;
  v.max_ctx = c.max_ctx;
  v.window = c.window;
  v.tiles = l.tiles;
  const float scale = (s.softmax_scale > 0.f ? s.softmax_scale : 1.0f / sqrtf(float(s.head_dim))) * kLog2e;
  uint8_t* const wb = reinterpret_cast<uint8_t*>(w);
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
    rebuild_kernel<D><<<dim3(unsigned(l.tiles) * 2, H, nb), 128, rebuild_smem<D>(), stream>>>(r);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
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
    a.part = l.splits > 1 ? reinterpret_cast<float*>(w + l.part) : nullptr;
    a.stats = reinterpret_cast<float2*>(w + l.stats);
    a.n_splits = l.splits;
    a.max_rows = l.rows;
    a.scale_log2 = scale;
    const unsigned blocks = unsigned((l.rows + 2 * kRows - 1) / (2 * kRows));
    attention_kernel<D, false><<<dim3(blocks * l.splits, H, nb), 320, AS::total, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (l.splits > 1) {
      merge_kernel<D><<<dim3(unsigned((l.rows + 3) / 4), H, nb), 128, 0, stream>>>(a);
      if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (!c.window) continue;
    a.n_splits = l.wsplits;
    a.max_rows = l.wrows;
    const unsigned wblocks = unsigned((l.wrows + 2 * kRows - 1) / (2 * kRows));
    attention_kernel<D, true><<<dim3(wblocks * l.wsplits, H, nb), 320, AS::total, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
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
    x.max_rows = l.wrows;
    x.q_tiles = l.q_tiles;
    x.cap = s.capacity;
    x.scale_log2 = scale;
    window_rows_kernel<D><<<dim3(unsigned(l.q_tiles), H, nb), kRows, kRows * D * 2, stream>>>(x);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    weights_kernel<D><<<dim3(unsigned(l.tiles), H, nb), 320, WS::total, stream>>>(x);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t chunk_tc_workspace_bytes(const rq_shape& s, int n_new, int max_ctx, int window) {
  return tc_layout(s, n_new, max_ctx, window).total;
}

cudaError_t launch_chunk_tc(const rq_shape& s, const rq_cache& cache, const rq_paging* paging,
                            const ChunkCall& c, void* ws, cudaStream_t stream) {
  char* const w = static_cast<char*>(ws);
  return s.head_dim == 128 ? launch_tc<128>(s, cache, paging, c, w, stream)
                           : launch_tc<64>(s, cache, paging, c, w, stream);
}

}  // namespace rq
