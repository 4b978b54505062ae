// Attention over the 8-bit cache for few query rows (include/rq_q8.h): every tile that some row sees
// is read once per 32 rows, with the codes turned into exact fp16 operands in registers.
//
//   S[t, r] = q_r . K_t on mma.sync, M = a warp's 16 slots, N = 8 rows; one scale per warp and tile
//   (a block of 16 slots is a warp's share), so scores are S * scale_K * (softmax scale of the row).
//   w = 2^(S - m) scale_V 2^-h, fp16; O[ch, r] += V^T w on mma.sync, M = 16 channels, K = the slots.
// A warp keeps its own m, l, h (rows) and accumulators over its slots; the four warps are merged once per
// segment.  m is raised when a score exceeds it by more than 8.  h is one number E for all rows, 2^-3 of the
// first V scale, while V scales stay within 2^4 of that: weights then reach 2^-1 and stay below 2^15.  From
// the first other scale on every row has its own (`heights`), raised as w exceeds 2^15, to make it 2^7: what a
// row does not see, or gives no weight, takes nothing from its other weights' 11 bits.
//
// CTAs share the work by the line of rq_q8_line.cuh; q8_stream_join_kernel joins the partial results of
// divided units, and the queries' operands are made by the kernel before (q8_prepare_kernel): code for
// either in this kernel costs its loop registers (verification of 8 tokens: 121 us against 109).
//
// One row or a few: bound by HBM while it streams (16 x 16 heads: 7.3 TB/s from 8,192 to 16,384 slots), by
// launches, first tiles and joins at short contexts (4,096 slots in 55 us, 40 at a copy's rate).  32 rows: by
// the latency of each warp's scores, softmax and values, two warps a scheduler (8 x 8 heads after 16,384
// slots in 107 us).
#include <type_traits>

#include "rq_q8_line.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr float kTop = 8.f;
constexpr int kScaleBelow = 3, kScaleRange = 4;   // E: below the first V scale; how far others may be from that
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kMostCtas = 1024;

struct StreamArgs : Q8Line {
  uint8_t* queries;      // [B][Hkv][blocks] of StreamSmem::kQuery bytes
  float tame_ks;         // K scales up to which their products with rows' factors stay in fp32's range
};

template <int D, int NT>
struct StreamSmem {
  static constexpr int kCtas = NT == 1 ? 3 : 2, kThreads = NT > 1 ? 256 : 160;
  static constexpr int kCodes = 2 * kQ8Tile * D, kStage = kCodes + 128;   // (scales: 32 bytes)
  static constexpr int kRows = 8 * NT, kMergeRow = D + 4;
  static constexpr int kMerge = 4 * 8 * kMergeRow * 4;
  static constexpr int kFragments = NT * (D / 16) * 32 * 8;
  static constexpr int kQuery = kFragments + kRows * 8;     // of a unit: B fragments, factors, own slots
  static constexpr int kHeld = NT > 2 ? kQuery : kRows * 8;  // of it in shared memory
  static constexpr int kFixed = kMerge + kHeld + 4 * kRows * 12 + 768;
  static constexpr int kStages0 = (227 * 1024 / kCtas - 1024 - kFixed) / kStage;
  static constexpr int kStages = kStages0 > 8 ? 8 : kStages0;
  static constexpr int merge = kStages * kStage, query = merge + kMerge, stats = query + kHeld;
  static constexpr int heights = stats + 4 * kRows * 8, bars = heights + 4 * kRows * 4, misc = bars + 16 * kStages;
  static constexpr int cut = misc + 16, walk = cut + int(sizeof(OwnCut));
  static constexpr int total = walk + int(sizeof(Walk<8, kQ8Tile>)) + 128;
  static_assert(kStages >= 2 && cut % 8 == 0 && total <= 227 * 1024 / kCtas - 1024, "shared memory");
};

__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// CH channels of a unit's row y, times inv 2^unit (the unit last, in two steps: it brings back V's size).
template <int D, int CH>
__device__ __forceinline__ void store_row(const Q8Line& a, int b, int h, int r0, int y, int rows, int ch, const float (&o)[CH], float inv, float unit) {
  if (y >= rows) return;
  const int j = (r0 + y) / a.G, hq = h * a.G + (r0 + y) % a.G;
  uint16_t* const p = a.c.out + ((int64_t(b) * a.c.n_new + j) * a.Hq + hq) * D + ch;
  const bool vec = (reinterpret_cast<uintptr_t>(a.c.out) & 15) == 0;
  uint32_t u[CH / 2];
  const float up = ex2(0.5f * unit);
#pragma unroll
  for (int k = 0; k < CH / 2; ++k) {
    const __nv_bfloat162 z = __floats2bfloat162_rn(o[2 * k] * inv * up * up, o[2 * k + 1] * inv * up * up);
    u[k] = *reinterpret_cast<const uint32_t*>(&z);
  }
  if (vec && CH == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[CH / 2 - 2], u[CH / 2 - 1]);
  else if (vec)
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  else
#pragma unroll
    for (int k = 0; k < CH / 2; ++k) {
      p[2 * k] = uint16_t(u[k]);
      p[2 * k + 1] = uint16_t(u[k] >> 16);
    }
}

// The kernel before: clears the error word and what tells of divided units (or cuts the line), and makes
// the queries' operands, a CTA a unit: B fragments, (k-step, row) word pairs of the lanes that use them.
template <int D, int NT>
__global__ void __launch_bounds__(128) q8_prepare_kernel(const __grid_constant__ StreamArgs a) {
  grid_next();
  using L = StreamSmem<D, NT>;
  if (blockIdx.x == 0) {
    if (a.own_cut) {
      if (threadIdx.x == 0) *a.err = 0u;
      for (int i = threadIdx.x; i < a.n_ctas; i += 128) a.parted[i].rows = 0;
    } else {
      cut_line<8 * NT, kQ8Tile, 128>(a);
    }
    return;
  }
  constexpr int KS = D / 16, LPR = D / 8, AT = 128 / LPR;   // lanes per row, rows at a time
  const unsigned unit = blockIdx.x - 1;
  const int block = int(unit % unsigned(a.blocks)), bh = int(unit / unsigned(a.blocks)), b = bh / a.v.H, h = bh % a.v.H;
  const Rows x = rows_of<8 * NT, kQ8Tile>(a, b, block);
  if (x.rows <= 0 || !x.ok) return;
  uint8_t* const to = a.queries + int64_t(unit) * L::kQuery;
  uint2* const query = reinterpret_cast<uint2*>(to);
  float* const row_scale = reinterpret_cast<float*>(to + L::kFragments);
  int* const row_limit = reinterpret_cast<int*>(row_scale + L::kRows);         // a row's own slot
  const int r0 = block * L::kRows, qc = threadIdx.x % LPR, lane = threadIdx.x & 31;
#pragma unroll
  for (int y0 = 0; y0 < L::kRows; y0 += AT) {
    const int y = y0 + threadIdx.x / LPR, j = (r0 + y) / a.G, hq = h * a.G + (r0 + y) % a.G;
    const bool live = y < x.rows;
    uint4 raw = make_uint4(0u, 0u, 0u, 0u);
    if (live) raw = q8_load8(a.c.q + b * a.c.q_strides[0] + j * a.c.q_strides[1] + hq * a.c.q_strides[2] + 8 * qc, a.qvec);
    float f[8];
    bool lost = false;
    if (a.c.rope.table != nullptr) {
      int pos = -1;
      if (live) {
        pos = a.c.rope.positions ? a.c.rope.positions[int64_t(b) * a.c.n_new + j] : x.ctx + j;
        lost = pos < 0 || pos >= a.c.rope.n_pos;
        if (lost) pos = -1;
      }
      const Q8Angles angles = q8_angles<D>(a.c.rope, pos, lane);
      q8_floats(raw, f);
      q8_rotate<D>(f, a.c.rope, angles, lane);
    } else {
      q8_floats(raw, f);
    }
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(f[k]));
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(RQ_FULL_MASK, mx, o));
    // a power of two brings the row's largest element into [2^14, 2^15): bf16 values are exact
    const int ex = int(__float_as_uint(mx) >> 23);
    const int e = mx == 0.f || ex == 255 ? 0 : min(141 - ex, kMostUp);
    const float up = q8_pow2(e >> 1), up2 = q8_pow2(e - (e >> 1));
    if (y >= L::kRows) continue;
    const int nt = y >> 3, n = y & 7;
    const int cc = D == 128 ? qc >> 2 : qc >> 1, s = D == 128 ? 2 * (qc & 3) : 2 * (qc & 1);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      query[(nt * KS + s + k) * 32 + 4 * n + cc] =
          make_uint2(pack_half2(f[4 * k] * up * up2, f[4 * k + 1] * up * up2),
                     pack_half2(f[4 * k + 2] * up * up2, f[4 * k + 3] * up * up2));
    if (qc == 0) {
      row_scale[y] = lost ? __int_as_float(0x7fc00000) : a.scale_log2 * q8_pow2(-(e >> 1)) * q8_pow2(-(e - (e >> 1)));
      row_limit[y] = x.ctx + min(j, x.n - 1);
    }
  }
}

// The parts of a divided unit: two rows a CTA, 16 threads (CH channels each) a row and group; the groups of
// a row take every groups-th part, the loads of four at a time, and are joined in order.
template <int D, int NT>
__global__ void __launch_bounds__(256) q8_stream_join_kernel(const __grid_constant__ StreamArgs a) {
  grid_wait();
  const Parted u = a.parted[blockIdx.x];
  const int y0 = int(blockIdx.y) * 2;
  if (y0 >= u.rows) return;
  constexpr int CH = D / 16, kRows = 8 * NT, TOGETHER = 4, kRow = D + 4;
  __shared__ float buffer[16 * kRow];
  const int left = u.rows - y0, rows = min(left, 2), groups = 16 / rows;   // rows here; groups of a row
  const int group = threadIdx.x >> 4, ch = (threadIdx.x & 15) * CH, y = y0 + group % rows, mine = group / rows;
  auto place = [&](int k) { return (2 * int64_t(k) + (k == u.first)) * kRows + y; };
  Join x = Join::none();
  float o[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) o[k] = 0.f;
#pragma unroll 1
  for (int k = u.first + mine; y < u.rows && k <= u.last; k += TOGETHER * groups) {
    float4 st[TOGETHER];
    float4 v[TOGETHER][CH / 4];
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      const int ki = k + i * groups;
      st[i] = make_float4(kNoMax, 0.f, kNoScale, 0.f);
      if (ki > u.last) continue;
      st[i] = a.stats[place(ki)];
#pragma unroll
      for (int z = 0; z < CH / 4; ++z) v[i][z] = *(reinterpret_cast<const float4*>(a.part + place(ki) * D + ch) + z);
    }
    float to = x.M, f0 = 1.f;
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      to = fmaxf(to, st[i].x);
      f0 *= x.raise(st[i].x, st[i].z);
    }
    x.sum *= ex2(x.M - to);
    x.M = to;
#pragma unroll
    for (int z = 0; z < CH; ++z) o[z] *= f0;
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      if (k + i * groups > u.last) continue;
      const float f = x.factor(st[i].x, st[i].z);
      x.sum += ex2(st[i].x - x.M) * st[i].y;
#pragma unroll
      for (int z = 0; z < CH / 4; ++z) {
        o[4 * z] = fmaf(f, v[i][z].x, o[4 * z]);
        o[4 * z + 1] = fmaf(f, v[i][z].y, o[4 * z + 1]);
        o[4 * z + 2] = fmaf(f, v[i][z].z, o[4 * z + 2]);
        o[4 * z + 3] = fmaf(f, v[i][z].w, o[4 * z + 3]);
      }
    }
  }
  float* const at = buffer + group * kRow;
#pragma unroll
  for (int z = 0; z < CH; ++z) at[4 + ch + z] = o[z];
  if (ch == 0) {
    at[0] = x.M;
    at[1] = x.sum;
    at[2] = x.Mo;
    at[3] = x.h;
  }
  __syncthreads();
  if (mine != 0 || y >= u.rows) return;
  const int filled = min(groups, u.last - u.first + 1);     // (the others have no part)
  for (int i = 0; i < filled; ++i) {
    const float* const from = buffer + (group + i * rows) * kRow;
    x.M = fmaxf(x.M, from[0]);
    x.raise(from[2], from[3]);
  }
  x.sum = 0.f;
#pragma unroll
  for (int z = 0; z < CH; ++z) o[z] = 0.f;
  for (int i = 0; i < filled; ++i) {
    const float* const from = buffer + (group + i * rows) * kRow;
    const float f = x.factor(from[2], from[3]);
    x.sum += ex2(from[0] - x.M) * from[1];
#pragma unroll
    for (int z = 0; z < CH; ++z) o[z] = fmaf(f, from[4 + ch + z], o[z]);
  }
  store_row<D, CH>(a, u.b, u.h, u.r0, y, u.rows, ch, o, x.inverse(), x.unit());
}

// (more than 8 rows: accumulators take more registers than two CTAs of five warps leave, so three more
// warps are launched that give theirs away)
template <int D, int NT, int FMT>
__global__ void __launch_bounds__(StreamSmem<D, NT>::kThreads, StreamSmem<D, NT>::kCtas) q8_stream_kernel(const __grid_constant__ StreamArgs a) {
  grid_next();
  using L = StreamSmem<D, NT>;
  using StreamWalk = Walk<8 * NT, kQ8Tile>;
  constexpr int KS = D / 16;                                // k-steps of a score, 16-channel tiles of O
  const int me = int(blockIdx.x);
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = smem_u32(smem + L::bars);
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (L::kStages + s); };
  int* const misc = reinterpret_cast<int*>(smem + L::misc); // [0]: gave up
  OwnCut& cut = *reinterpret_cast<OwnCut*>(smem + L::cut);
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 4);
    }
    misc[0] = 0;
    fence_mbar_init();
  }
  if (a.own_cut) {
    const bool bad = own_cut<8 * NT, kQ8Tile, StreamSmem<D, NT>::kThreads>(a, cut, me);
    if (bad && me == 0 && threadIdx.x == 0) {
      grid_wait();
      atomicOr(a.err, 1u);
    }
  } else {
    grid_wait();
    if (threadIdx.x == 0) {
      cut.used = *a.used;
      cut.N = a.prefix[int64_t(a.B) * a.blocks];
      if (me < cut.used) {
        cut.from = a.cut[me];
        cut.to = a.cut[me + 1].pos;
        cut.rows = rows_of<8 * NT, kQ8Tile>(a, cut.from.b, cut.from.block);
      }
    }
    __syncthreads();
  }
  if (me >= cut.used) {
    grid_wait();                                            // (the kernel before is complete when this one is)
    return;
  }
  if (warp >= 4) {                                          // ---- copies
    if constexpr (NT > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp > 4) return;
    StreamWalk w;
    w.begin(cut);
    int g = 0;
    bool good = true;
    while (good && w.next(a)) {
      if (!w.x.ok) continue;
      for (int t0 = 0; t0 < w.T && good; t0 += 32) {
        int64_t rec = -1;
        if (t0 + lane < w.T) rec = a.v.record(w.b, w.h, w.x.tile(w.x.step(w.kt0 + t0 + lane)));
        const int m = min(32, w.T - t0);
        for (int t = 0; t < m && good; ++t, ++g) {
          const int64_t r = __shfl_sync(RQ_FULL_MASK, rec, t);
          const int s = g % L::kStages, n = g / L::kStages;
          if (n > 0) good = mbar_wait_bounded(empty(s), (n - 1) & 1, kWaitNs);
          good = __all_sync(RQ_FULL_MASK, good);
          if (!good) break;
          uint8_t* const stage = smem + s * L::kStage;
          if (r < 0) {                                      // no page: zeros under scales that are not numbers
            for (int k = lane; k < L::kCodes / 16; k += 32) reinterpret_cast<uint4*>(stage)[k] = make_uint4(0u, 0u, 0u, 0u);
            if (lane < 8) reinterpret_cast<float*>(stage + L::kCodes)[lane] = __int_as_float(0x7fc00000);
            fence_async_smem();                             // (a later copy writes there)
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(full(s));
              grid_wait();
              atomicOr(a.err, 1u);
            }
          } else if (lane == 0) {
            mbar_arrive_expect_tx(full(s), L::kCodes + 32);
            bulk_g2s(smem_u32(stage), a.v.codes + r * a.v.rec_codes, L::kCodes, full(s));
            bulk_g2s(smem_u32(stage + L::kCodes), a.v.scales + r * a.v.rec_scales, 32, full(s));
          }
          __syncwarp();
        }
      }
    }
    if (!good) {                                            // copies in flight land before the CTA leaves
      for (int k = max(0, g - L::kStages); k < g; ++k) mbar_wait_bounded(full(k % L::kStages), (k / L::kStages) & 1, kWaitNs);
      if (lane == 0) {
        atomicExch(&misc[0], 1);
        grid_wait();
        atomicOr(a.err, 1u);
      }
    }
  } else {                                                  // ---- products
    if constexpr (NT > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int r = lane >> 2, c = lane & 3;
    float* const merge = reinterpret_cast<float*>(smem + L::merge);
    float2* const stats = reinterpret_cast<float2*>(smem + L::stats);          // [warp][row]
    float* const heights = reinterpret_cast<float*>(smem + L::heights) + warp * L::kRows;   // h of this warp's rows
    uint8_t* const held = smem + L::query;                  // what is held of the unit's queries: all, or factors and own slots
    const uint2* const query = reinterpret_cast<const uint2*>(held);
    const float* const row_scale = reinterpret_cast<const float*>(held + L::kHeld - L::kRows * 8);
    const int* const row_limit = reinterpret_cast<const int*>(row_scale + L::kRows);   // a row's own slot
    constexpr int CH = D / 16;                              // channels of a thread that stores
    StreamWalk& w = *reinterpret_cast<StreamWalk*>(smem + L::walk);            // thread 0 walks
    if (threadIdx.x == 0) w.begin(cut);
    int g = 0;
    bool dead = false;
    for (;;) {
      if (threadIdx.x == 0) w.next(a);
      consumers_sync();
      if (!w.more) break;
      const Rows& x = w.x;
      const int r0 = w.block * L::kRows;
      const uint8_t* const queries = a.queries + ((int64_t(w.b) * a.v.H + w.h) * a.blocks + w.block) * L::kQuery;
      grid_wait();                                          // (the queries are there)
      if (x.ok)
        for (int k = threadIdx.x; k < L::kHeld / 8; k += 128)
          reinterpret_cast<uint2*>(held)[k] = __ldcg(reinterpret_cast<const uint2*>(queries + L::kQuery - L::kHeld) + k);
      uint2 qf[NT <= 2 ? NT * KS : 1];                      // (more rows: read again for every tile)
      if (NT <= 2)
#pragma unroll
        for (int k = 0; k < NT * KS; ++k) qf[k] = x.ok ? __ldcg(reinterpret_cast<const uint2*>(queries) + k * 32 + lane) : make_uint2(0u, 0u);
      consumers_sync();

      float acc[NT][KS][4], m[NT][2], l[NT][2], cs[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          m[t][k] = kNoMax;
          l[t][k] = 0.f;
          cs[t][k] = row_scale[8 * t + 2 * c + k];
        }
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[t][i][k] = 0.f;
      }
      int E = kNoScale, t = 0;
      // Tiles from t on; without APART up to one whose V scale is out of E's range, or whose K scale is huge.  (Two loops: as one, with
      // the rows' h behind a branch, verification of 8 tokens took 121 us, now 112.)
      auto tiles = [&](auto apart) {
      constexpr bool APART = decltype(apart)::value;
      for (; x.ok && t < w.T; ++t, ++g) {
        const int s = g % L::kStages;
        if (!dead) dead = !__all_sync(RQ_FULL_MASK, mbar_wait_bounded(full(s), (g / L::kStages) & 1, kWaitNs));
        if (dead) continue;                                 // (the copies' warp gives up in its turn)
        const uint8_t* const stage = smem + s * L::kStage;
        const int slot0 = x.tile(x.step(w.kt0 + t)) * kQ8Tile + 16 * warp;
        const int oldest = a.c.window > 0 ? x.ctx + x.j0 + 1 - a.c.window : 0;   // the first row's window
        if (slot0 < x.hi && (slot0 + 15 >= oldest || slot0 < a.c.n_sink)) {
          const float* const scales = reinterpret_cast<const float*>(stage + L::kCodes);
          const float ks = scales[warp], vs = scales[4 + warp];
          // ---- scores
          float sc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[n][k] = 0.f;
          {
            const uint8_t* const k0 = stage + (16 * warp + r) * D;     // rows r and r + 8: the same swizzle
            const int sw = q8_swizzle<D>(r);
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              const int at = ((D / 64 * c + half) ^ sw) << 4;
              const uint4 u = *reinterpret_cast<const uint4*>(k0 + at), v = *reinterpret_cast<const uint4*>(k0 + 8 * D + at);
              const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t x0 = q8_word<FMT>(uw[k]), x1 = q8_word<FMT>(vw[k]);
                const uint32_t a0 = q8_pair<FMT, 0>(x0), a1 = q8_pair<FMT, 0>(x1);
                const uint32_t a2 = q8_pair<FMT, 1>(x0), a3 = q8_pair<FMT, 1>(x1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  const int at_q = n * KS + 4 * half + k;
                  const uint2 q = NT <= 2 ? qf[NT <= 2 ? at_q : 0] : query[at_q * 32 + lane];
                  mma_f16(sc[n], a0, a1, a2, a3, q.x, q.y);
                }
              }
            }
          }
          // ---- softmax weights
          const bool clear = slot0 + 15 <= x.ctx + x.j0 &&
                             (a.c.window <= 0 || slot0 > x.ctx + x.j1 - a.c.window || slot0 + 15 < a.c.n_sink);
          float ksc[NT][2];
          bool over = false;
          uint32_t hidden = 0u;                             // bit 4 n + k: element not seen by its row
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) ksc[n][k] = cs[n][k] * ks;
          if (APART && ks > a.tame_ks) {                    // (both factors huge: one by one, so that 0 stays 0)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (ksc[n][k] == INFINITY) {
                  sc[n][k] *= cs[n][k];
                  sc[n][k + 2] *= cs[n][k];
                  ksc[n][k] = ks;
                }
          }
          if (!clear) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int slot = slot0 + r + 8 * (k >> 1), own = row_limit[8 * n + 2 * c + (k & 1)];
                const bool seen = slot <= own && (a.c.window <= 0 || slot > own - a.c.window || slot < a.c.n_sink);
                if (!seen) {
                  hidden |= 1u << (4 * n + k);
                  sc[n][k] = -INFINITY;
                }
              }
            // (a scale of 0 or less does not occur; NaN stays with the rows that see the block)
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              sc[n][k] = hidden >> (4 * n + k) & 1u ? -INFINITY : sc[n][k] * ksc[n][k & 1];
              over |= sc[n][k] > m[n][k & 1] + kTop;
            }
          const int ev = q8_exponent(vs);
          const bool lost = ev > 127, far = !APART && (unsigned(ev - E - kScaleBelow + kScaleRange) > 2u * kScaleRange || ks > a.tame_ks);
          const float evf = lost ? vs : float(ev);          // (NaN where the scale is)
          if (APART)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                over |= (sc[n][k] - m[n][k & 1]) + (evf - heights[8 * n + 2 * c + (k & 1)]) > kWeightTop;
          if (__any_sync(RQ_FULL_MASK, over) || far) {
            if (far && !lost) {
              if (E != kNoScale || ks > a.tame_ks) return;  // (here and not before the scores, which need not wait for it)
              E = ev - kScaleBelow;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const float h = APART ? heights[8 * n + 2 * c + k] : 0.f;
                if (APART) __syncwarp();                    // (read before one lane of the row's writes)
                float v = fmaxf(sc[n][k], sc[n][k + 2]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(RQ_FULL_MASK, v, o));
                const float to = v > m[n][k] + kTop ? v : m[n][k];
                const float f = ex2(m[n][k] - to);
                float fa = f;                               // of the accumulators, whose unit is 2^(m + h)
                if (APART && (v > m[n][k] + kTop || (v - m[n][k]) + (evf - h) > kWeightTop)) {
                  const float hn = fmaxf(h + (m[n][k] - to), evf + (v - to) - kWeightHead);   // (evf NaN: the first)
                  fa = ex2((m[n][k] - to) + (h - hn));
                  if (r == 0) heights[8 * n + 2 * c + k] = hn;
                }
                m[n][k] = to;
                l[n][k] *= f;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                  acc[n][i][k] *= fa;
                  acc[n][i][k + 2] *= fa;
                }
              }
            if (APART) __syncwarp();
          }
          uint32_t b0[NT], b1[NT];
          const float vsc = APART ? 1.f : vs * q8_pow2(-E);   // (E == kNoScale: vs is not a number)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float z = sc[n][k] - m[n][k & 1];
              p[k] = ex2(z);
              l[n][k & 1] += p[k];
              p[k] = APART ? ex2(z + (evf - heights[8 * n + 2 * c + (k & 1)])) : p[k] * vsc;
              if (hidden >> (4 * n + k) & 1u) p[k] = 0.f;
            }
            b0[n] = transposed(pack_half2(p[0], p[1]));
            b1[n] = transposed(pack_half2(p[2], p[3]));
          }
          // ---- values
          {
            constexpr int W = D / 32;                       // words of a lane's channels of one row
            uint32_t v[4][W];                               // slots 2c, 2c + 1, 2c + 8, 2c + 9
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int row = 16 * warp + 2 * c + (k & 1) + 8 * (k >> 1);
              const uint8_t* const p = stage + kQ8Tile * D + row * D;
              if (D == 128) {
                const uint4 u = *reinterpret_cast<const uint4*>(p + ((r ^ q8_swizzle<D>(row)) << 4));
                v[k][0] = u.x;
                v[k][1] = u.y;
                v[k][W - 2] = u.z;
                v[k][W - 1] = u.w;
              } else {
                const uint2 u = *reinterpret_cast<const uint2*>(p + (((r >> 1) ^ q8_swizzle<D>(row)) << 4) + (r & 1) * 8);
                v[k][0] = u.x;
                v[k][1] = u.y;
              }
              // slots that no row sees may hold anything (a code that is not a number, too)
              const int slot = slot0 - 16 * warp + row;
              if (!clear && (slot >= x.hi || (slot < oldest && slot >= a.c.n_sink)))
#pragma unroll
                for (int i = 0; i < W; ++i) v[k][i] = 0u;
#pragma unroll
              for (int i = 0; i < W; ++i) v[k][i] = q8_word<FMT>(v[k][i]);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              const uint32_t lo = __byte_perm(v[0][i / 2], v[1][i / 2], i & 1 ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(v[2][i / 2], v[3][i / 2], i & 1 ? 0x7362 : 0x5140);
              const uint32_t a0 = q8_pair<FMT, 0>(lo), a1 = q8_pair<FMT, 1>(lo);
              const uint32_t a2 = q8_pair<FMT, 0>(hi), a3 = q8_pair<FMT, 1>(hi);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16(acc[n][i], a0, a1, a2, a3, b0[n], b1[n]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(s));
      }
      };
      tiles(std::false_type{});
      if (lane < L::kRows) heights[lane] = float(E);        // (E == kNoScale: acc is 0)
      __syncwarp();
      tiles(std::true_type{});

      // ---- the four warps' results joined, eight rows at a time
      if (dead && lane == 0) atomicExch(&misc[0], 1);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[n][k] += __shfl_xor_sync(RQ_FULL_MASK, l[n][k], o);
          if (r == 0) stats[warp * L::kRows + 8 * n + 2 * c + k] = make_float2(m[n][k], l[n][k]);
        }
      const bool whole = w.kt0 == 0 && w.T == x.V;
      const int slot = 2 * me + (w.kt0 == 0 ? 1 : 0);
      const float* const all_heights = reinterpret_cast<const float*>(smem + L::heights);
      const int mr = threadIdx.x >> 4, ch = (threadIdx.x & 15) * CH;   // row, channels of a thread
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        consumers_sync();
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<float2*>(merge + (warp * 8 + 2 * c + k) * L::kMergeRow + KS * 2 * r + 2 * i) =
                make_float2(acc[n][i][k], acc[n][i][k + 2]);
        consumers_sync();
        const int y = 8 * n + mr;
        float M = kNoMax, sum = 0.f, H = -INFINITY, z4[4], o[CH];   // z4: a warp's unit against 2^M
#pragma unroll
        for (int k = 0; k < CH; ++k) o[k] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) M = fmaxf(M, stats[k * L::kRows + y].x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 st = stats[k * L::kRows + y];
          sum += ex2(st.x - M) * st.y;
          z4[k] = (st.x - M) + all_heights[k * L::kRows + y];
          H = fmaxf(H, z4[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float fe = ex2(z4[k] - H);
          const float* const p = merge + (k * 8 + mr) * L::kMergeRow + ch;
#pragma unroll
          for (int z = 0; z < CH; ++z) o[z] = fmaf(fe, p[z], o[z]);
        }
        if (!x.ok || *reinterpret_cast<volatile int*>(&misc[0]) != 0) sum = __int_as_float(0x7fc00000);
        if (whole) {
          store_row<D, CH>(a, w.b, w.h, r0, y, x.rows, ch, o, sum == 0.f ? 0.f : 1.f / sum, H);
        } else {
          float* const p = a.part + (int64_t(slot) * L::kRows + y) * D + ch;
#pragma unroll
          for (int z = 0; z < CH; z += 4) *reinterpret_cast<float4*>(p + z) = make_float4(o[z], o[z + 1], o[z + 2], o[z + 3]);
          if (ch == 0) a.stats[int64_t(slot) * L::kRows + y] = make_float4(M, sum, H, 0.f);
        }
      }
      if (!whole && w.kt0 == 0 && threadIdx.x == 0) {       // (told by the CTA where the unit begins)
        int first, last;
        w.sharers(cut.N, cut.used, first, last);
        a.parted[me] = {w.b, w.h, r0, x.rows, first, last};
      }
      consumers_sync();                                     // (the next segment overwrites what was read)
    }
    grid_wait();
    if (dead && lane == 0) atomicOr(a.err, 1u);
  }
}

// ------------------------------------------------------------------------------------- host

int tiles_of_rows(int64_t rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

Q8Layout stream_layout(const rq_q8_shape& s, int n_new, int max_ctx, int nt) {
  return q8_layout(s, n_new, max_ctx, 8 * nt, kQ8Tile, std::min(device_sm_count() * (nt == 1 ? 3 : 2), kMostCtas));
}

size_t query_bytes(const rq_q8_shape& s, int n_new, int nt) {
  const int64_t rows = int64_t(n_new) * (s.n_q_heads / s.n_kv_heads), blocks = (rows + 8 * nt - 1) / (8 * nt);
  return size_t(s.batch) * s.n_kv_heads * blocks * (size_t(nt) * (s.head_dim / 16) * 256 + size_t(8 * nt) * 8);
}

template <int D, int NT, int FMT>
cudaError_t launch(const StreamArgs& a, cudaStream_t stream) {
  using L = StreamSmem<D, NT>;
  static OncePerDevice once;
  cudaError_t e = once([] {
    return cudaFuncSetAttribute(q8_stream_kernel<D, NT, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
  });
  if (e != cudaSuccess) return e;
  q8_prepare_kernel<D, NT><<<1 + unsigned(a.B) * a.v.H * a.blocks, 128, 0, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_after(true, q8_stream_kernel<D, NT, FMT>, dim3(unsigned(a.n_ctas)), L::kThreads, L::total, stream, a)) != cudaSuccess) return e;
  if (a.whole) return cudaSuccess;                          // (nothing to join)
  const int rows = int(std::min<int64_t>(8 * NT, int64_t(a.c.n_new) * a.G));
  return launch_after(true, q8_stream_join_kernel<D, NT>, dim3(unsigned(a.n_ctas), unsigned((rows + 1) / 2)), 256, 0, stream, a);
}

// Whether units stay whole, which saves the launch that joins their parts.  That launch costs what about
// four more tiles on a CTA cost, a fourth of it where few units leave most CTAs idle; and no more than
// eight tiles, as one long sequence among short ones is then a CTA's.  After 250 slots, 16 heads each:
// 16 sequences 16.1 -> 12.4 us, 8 14.1 -> 11.9; 32 sequences of 8 heads with 16 rows each 24.9 -> 15.3.
// Against the rule: 8 heads after 500 slots 9.3 -> 12.0, 512 heads 22.6 -> 25.7.
bool whole_units(const StreamArgs& a) {
  int64_t tiles = (std::min<int64_t>(int64_t(a.c.max_ctx) + a.c.n_new, a.cap) + kQ8Tile - 1) / kQ8Tile;
  if (a.c.window > 0) {
    const int64_t sinks = (int64_t(a.c.n_sink) + kQ8Tile - 1) / kQ8Tile;
    tiles = std::min(tiles, sinks + (int64_t(a.c.window) + a.c.n_new + kQ8Tile - 1) / kQ8Tile + 1);
  }
  const int64_t units = int64_t(a.B) * a.v.H * a.blocks, ctas = a.n_ctas;
  const int64_t whole = (units + ctas - 1) / ctas * tiles, divided = (units * tiles + ctas - 1) / ctas;
  return tiles <= 8 && whole - divided <= (4 * units >= ctas ? 4 : 1);
}

}  // namespace

size_t q8_stream_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx) {
  const int nt = tiles_of_rows(int64_t(n_new) * (s.n_q_heads / s.n_kv_heads));
  return stream_layout(s, n_new, max_ctx, nt).total + query_bytes(s, n_new, nt);
}

cudaError_t launch_q8_stream(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                             const Q8Call& c, void* ws, cudaStream_t stream) {
  const int nt = tiles_of_rows(int64_t(c.n_new) * (s.n_q_heads / s.n_kv_heads));
  StreamArgs a = {};
  static_cast<Q8Line&>(a) = q8_line(s, cache, paging, c, 8 * nt);
  const Q8Layout x = stream_layout(s, c.n_new, c.max_ctx, nt);
  q8_place(a, x, ws);
  a.queries = static_cast<uint8_t*>(ws) + x.total;
  a.tame_ks = a.scale_log2 <= 64.f ? 256.f : 0.f;           // (factors: 2^113 scale_log2 at most)
  a.own_cut = int64_t(a.B) * a.blocks <= kOwnCutPairs;
  a.whole = a.own_cut && whole_units(a);
  const bool i8 = s.format == RQ_Q8_INT8, wide = s.head_dim == 128;
  switch (nt) {
    case 1:
      return wide ? (i8 ? launch<128, 1, RQ_Q8_INT8>(a, stream) : launch<128, 1, RQ_Q8_E4M3>(a, stream))
                  : (i8 ? launch<64, 1, RQ_Q8_INT8>(a, stream) : launch<64, 1, RQ_Q8_E4M3>(a, stream));
    case 2:
      return wide ? (i8 ? launch<128, 2, RQ_Q8_INT8>(a, stream) : launch<128, 2, RQ_Q8_E4M3>(a, stream))
                  : (i8 ? launch<64, 2, RQ_Q8_INT8>(a, stream) : launch<64, 2, RQ_Q8_E4M3>(a, stream));
    default:
      return wide ? (i8 ? launch<128, 4, RQ_Q8_INT8>(a, stream) : launch<128, 4, RQ_Q8_E4M3>(a, stream))
                  : (i8 ? launch<64, 4, RQ_Q8_INT8>(a, stream) : launch<64, 4, RQ_Q8_E4M3>(a, stream));
  }
}

}  // namespace rq
