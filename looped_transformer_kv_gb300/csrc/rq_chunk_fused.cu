// Chunk attention of up to 128 rows per kv-head over the packed cache on the 5th-generation tensor
// cores (sm_103a): the codes are turned into fp16 operands in shared memory and never leave it.
//
// For a row's query q and a cached token t (rit.work summary, "How each pass's KV cache is
// reconstructed": reference and residuals rebuilt inside attention)
//   S = [q | R q] . [a (s^r c^r + z^r) | s^e c^e + z^e]
//   O_ref += P a (s^r c^r + z^r),   O_res += P (s^e c^e + z^e)        (rotated domain)
// so one product with K = 2 d gives the scores and one with N = 2 d both accumulators; the
// combine kernel undoes the rotation once.  Tiles are the cache's 64-token records.
//
// Warps 0-3: softmax, a thread per row; 4-11: K codes -> operand images; 12-19: V's; 20: products;
// 21: copies.  Tensor memory: queries (A operand) 128 columns, two score tiles of 64 (the softmax
// weights overwrite them), accumulators 256.  Shared memory: 4 raw records, two K and two V images.
//
// A code pair sits 16 bits apart in its word, so an image's channels are permuted: inside 8
// channels (4-bit codes) position 2 i + e holds channel i + 4 e, inside 16 (2-bit codes) channel
// i + 8 e.  The queries are stored in the same order and the accumulators are put back in order
// when they leave.
// The queries are fp16 (q exactly, R q rounded once, both times the row's power of two); a level
// s c + z is rounded once to fp16, a reference level once more by a; weights once; sums are fp32.
// 8 tokens x 4 heads after 16,384 (8 sequences, 8 kv-heads, 2-bit residuals): 118 us, 2.3 TB/s, 1,600
// cycles per record and about 7 us per CTA to begin and end.  No one part bounds it: issue slots are 53 %
// used, the tensor pipe 50 % (1,250 cycles of a 128-row tile whatever the rows), shared memory's data
// banks 15 % each way; what does is the chain of a record through its parts, two deep.  The copies
// alone take 69 us, conversions with the copies 92, products and softmax with them 110.  More raw
// records, records prefetched to L2, a warp each for scores' and values' products, conflict-free
// stores of the images and weights through shared memory did not shorten it.
#include "rq_common.cuh"
#include "rq_kernels.h"
#include "rq_launch.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

constexpr uint64_t kFuWaitLimitNs = 2000000000ull;
constexpr int kFuRows = 128;
constexpr int kRawStages = 4;

struct FusedArgs {
  const uint8_t* data;
  int64_t rec_bytes;
  const int32_t* bt;
  int max_pages, n_pages, cap, sec_off;
  const uint16_t* q;
  int64_t qs0, qs1, qs2;
  const int8_t* ksigns;
  uint4* qimg;               // [unit][row][2 D] fp16 (q | R q), scaled per row
  float* qscale;             // [unit][row]: score scale (log2 units)
  const int32_t* n_lens;
  const int32_t* ctx_lens;
  float* part;               // [unit][row][split][4 + 2 D]
  unsigned* err;
  int H, heads, n_new, max_ctx, n_splits, rows;
  float scale_log2;
};

// Position of channel c in an image of BITS-bit codes (the order above).
template <int BITS>
__host__ __device__ constexpr int image_position(int c) {
  constexpr int N = 16 / BITS;            // codes of 16 bits
  return c / (2 * N) * (2 * N) + 2 * (c % N) + c / N % 2;
}

// One warp per row: the row's fp16 queries and its scale.  Clears the call's error word first (it
// runs before anything that sets it).
template <int D, int RES>
__global__ void __launch_bounds__(128) fused_rows_kernel(const __grid_constant__ FusedArgs a, int n_rows) {
  grid_next();
  constexpr int P = D / 32;
  if (blockIdx.x == 0 && threadIdx.x < kWsHeaderBytes / 4) a.err[threadIdx.x] = 0u;
  const int lane = threadIdx.x & 31;
  const int64_t wid = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (wid >= n_rows) return;
  const int row = int(wid % a.rows), h = int(wid / a.rows % a.H), b = int(wid / a.rows / a.H);
  const int j = row / a.heads, g = row % a.heads;
  const int n = a.n_lens ? a.n_lens[b] : a.n_new;
  float v[P], mx = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    v[i] = j < n ? bf16_bits_to_float(a.q[b * a.qs0 + j * a.qs1 + (int64_t(h) * a.heads + g) * a.qs2 + lane * P + i]) : 0.f;
    mx = fmaxf(mx, fabsf(v[i]));
  }
  mx = warp_max(mx);
  // largest element to [2^10, 2^11): |R q| stays below sqrt(128) times that, inside fp16
  const int x = int(__float_as_uint(mx) >> 23);
  const int e = x == 0 || x == 255 ? 0 : min(137 - x, 100);
  const float up = ldexpf(1.f, e >> 1), up2 = ldexpf(1.f, e - (e >> 1));
  __half* const o = reinterpret_cast<__half*>(a.qimg) + wid * (RES ? 2 * D : D);
  float r[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    v[i] = v[i] * up * up2;
    o[image_position<4>(lane * P + i)] = __float2half_rn(v[i]);
    if (RES) r[i] = v[i] * float(a.ksigns[int64_t(h) * D + lane * P + i]);
  }
  if (RES) {
    warp_fwht<P>(r, lane);
    const float inv_sqrt_d = (D == 128) ? 0.08838834764831845f : 0.125f;
#pragma unroll
    for (int i = 0; i < P; ++i) o[D + image_position<RES ? RES : 4>(lane * P + i)] = __float2half_rn(r[i] * inv_sqrt_d);
  }
  if (lane == 0) a.qscale[wid] = ldexpf(a.scale_log2, -e);
}

// B operand with N contiguous (V rows): panels of 64 tokens x 64 channels, the token rows 128 bytes,
// swizzled as the K-major panels; `panel` bytes from one 64-channel panel to the next.
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr, uint32_t panel) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(panel >> 4) << 16) | (uint64_t(64) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
constexpr uint32_t kMnB = 1u << 16;   // instruction descriptor: B's N index is contiguous

// The levels s c + z of a word's codes as 16-byte chunks of the image (4-bit codes: one, 2-bit: two),
// each rounded once, whatever the step's size: code_pair_at gives the code itself, not its multiple by
// the power of two of its bit position, which would leave its inverse to a step that fp16 holds exactly
// only above 2^-8 (2-bit codes; states of 0.001 then had errors of 0.2 %).
struct Steps {
  __half2 s, z;
  __device__ __forceinline__ explicit Steps(uint32_t meta) {
    const __half2 m = *reinterpret_cast<const __half2*>(&meta);
    s = __low2half2(m);
    z = __high2half2(m);
  }
};
template <int BITS>
__device__ __forceinline__ void levels(uint32_t w, const Steps& st, uint32_t* o) {
  constexpr uint32_t MASK = BITS == 2 ? 0x00030003u : 0x000F000Fu;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t x = e ? w >> 8 : w;
#pragma unroll
    for (int i = 0; i < 8 / BITS; ++i) {
      const uint32_t c = code_pair_at(x, MASK, BITS * i);
      const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&c), st.s, st.z);
      o[e * (8 / BITS) + i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
}
__device__ __forceinline__ uint32_t times(uint32_t x, __half2 a) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&x), a);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D, int RES>
struct FusedSmem {
  static constexpr int NG = D / 32, NP = (D / 64) * (RES ? 2 : 1);       // 64-wide panels of an image
  static constexpr int kRef = kTile * (D + 8 * NG);
  static constexpr int kRes = RES ? kTile * (2 * (D * RES / 8) + 8 * NG + 4) : 0;
  static constexpr int kRaw = kRef + kRes, kPanel = kTile * 128, kImg = NP * kPanel;
  static constexpr int k = 0, v = 2 * kImg, raw = 4 * kImg;
  static constexpr int bars = raw + kRawStages * kRaw, total = bars + 256 + 1024;
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
};

template <int D, int RES>
__global__ void __launch_bounds__(768, 1) fused_kernel(const __grid_constant__ FusedArgs a) {
  grid_wait();
  grid_next();
  using L = FusedSmem<D, RES>;
  constexpr int NG = L::NG, KD = 64 * L::NP;                 // scores' K, accumulators' N
  constexpr int SIDE = kTile * (D / 2 + 4 * NG);             // K (or V) part of the reference section
  constexpr int RROW = D * RES / 8, RSIDE = kTile * (RROW + 4 * NG + 2);
  extern __shared__ uint8_t raw_smem[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  const uint32_t bar0 = smem_u32(bars);
  auto rawfull = [&](int s) { return bar0 + 8 * s; };
  auto rawfree = [&](int s) { return bar0 + 8 * (4 + s); };
  auto kfull = [&](int s) { return bar0 + 8 * (8 + s); };
  auto kfree = [&](int s) { return bar0 + 8 * (10 + s); };
  auto vfull = [&](int s) { return bar0 + 8 * (12 + s); };
  auto vfree = [&](int s) { return bar0 + 8 * (14 + s); };
  auto sready = [&](int s) { return bar0 + 8 * (16 + s); };
  auto pready = [&](int s) { return bar0 + 8 * (18 + s); };
  const uint32_t qready = bar0 + 8 * 20, done = bar0 + 8 * 21;
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 22);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t unit = int64_t(b) * a.H + h;
  const int n = a.n_lens ? a.n_lens[b] : a.n_new, ctx = a.ctx_lens[b];
  if (n < 0 || n > a.n_new || ctx < 0 || ctx > a.max_ctx) {
    if (threadIdx.x == 0) atomicOr(a.err, 1u);
    return;
  }
  const int rows = n * a.heads;
  if (rows == 0) return;
  const int n_tiles = (ctx + kTile - 1) / kTile;
  const int kt0 = int(int64_t(split) * n_tiles / a.n_splits), T = int(int64_t(split + 1) * n_tiles / a.n_splits) - kt0;
  const int active = (rows + 31) / 32;                       // softmax warps with rows

  if (warp == 20) tc_alloc(smem_u32(tslot), 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(rawfull(i), 1);
      mbar_init(rawfree(i), 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(kfull(i), 8);
      mbar_init(kfree(i), 1);
      mbar_init(vfull(i), 8);
      mbar_init(vfree(i), 1);
      mbar_init(sready(i), 1);
      mbar_init(pready(i), active);
    }
    mbar_init(qready, active);
    mbar_init(done, 1);
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tQ = tmem, tS = tmem + 128, tO = tmem + 256;
  bool failed = false;

  if (warp >= 20) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    const bool leader = elect_one();
    if (warp == 21 && leader) {                             // ---- copies
      int issued = 0;
      for (; issued < T; ++issued) {
        const int s = issued % kRawStages, use = issued / kRawStages;
        if (use > 0 && !mbar_wait_bounded(rawfree(s), (use - 1) & 1, kFuWaitLimitNs)) break;
        int64_t rec;
        if (a.bt) {
          int pg = a.bt[int64_t(b) * a.max_pages + kt0 + issued];
          if (pg < 0 || pg >= a.n_pages) {
            atomicOr(a.err, 1u);
            pg = 0;
          }
          rec = int64_t(pg) * a.H + h;
        } else {
          rec = unit * (a.cap / kTile) + kt0 + issued;
        }
        const uint8_t* src = a.data + rec * a.rec_bytes;
        const uint32_t dst = smem_u32(smem + L::raw + s * L::kRaw);
        mbar_arrive_expect_tx(rawfull(s), L::kRaw);
        bulk_g2s(dst, src, L::kRef, rawfull(s));
        if (RES) bulk_g2s(dst + L::kRef, src + a.sec_off, L::kRes, rawfull(s));
      }
      failed = issued < T;
      for (int j = max(0, issued - kRawStages); j < issued; ++j)     // no copy outlives the CTA
        failed |= !mbar_wait_bounded(rawfull(j % kRawStages), (j / kRawStages) & 1, kFuWaitLimitNs);
    }
    if (warp == 20 && leader && T > 0) {                     // ---- products
      constexpr uint32_t ids = f16_idesc(kFuRows, kTile), ido = f16_idesc(kFuRows, KD) | kMnB;
      auto scores = [&](int s) {
        const uint32_t k = smem_u32(smem + L::k + s * L::kImg);
#pragma unroll
        for (int x = 0; x < KD / 16; ++x)
          tc_mma_ta(tS + 64 * s, tQ + 8 * x, panel_desc(k + (x / 4) * L::kPanel + (x % 4) * 32), ids, x > 0);
        tc_commit(sready(s));
        tc_commit(kfree(s));
      };
      bool good = mbar_wait_bounded(qready, 0, kFuWaitLimitNs);
      for (int j = 0; j <= T && good; ++j) {
        if (j < T) {
          good = mbar_wait_bounded(kfull(j & 1), (j >> 1) & 1, kFuWaitLimitNs);
          if (!good) break;
          tc_fence_after();
          scores(j & 1);
        }
        if (j > 0) {
          const int i = j - 1, s = i & 1;
          good = mbar_wait_bounded(pready(s), (i >> 1) & 1, kFuWaitLimitNs) &&
                 mbar_wait_bounded(vfull(s), (i >> 1) & 1, kFuWaitLimitNs);
          if (!good) break;
          tc_fence_after();
          const uint32_t v = smem_u32(smem + L::v + s * L::kImg);
#pragma unroll
          for (int x = 0; x < kTile / 16; ++x)
            tc_mma_ta(tO, tS + 64 * s + 8 * x, mn_desc(v + x * 2048, L::kPanel), ido, i > 0 || x > 0);
          tc_commit(vfree(s));
        }
      }
      tc_commit(done);
      failed = !mbar_wait_bounded(done, 0, kFuWaitLimitNs) || !good;
      for (int j = max(0, T - 2); j < T && !failed; ++j)     // no arrival outstanding when the CTA leaves
        failed = !mbar_wait_bounded(kfree(j & 1), (j >> 1) & 1, kFuWaitLimitNs) ||
                 !mbar_wait_bounded(vfree(j & 1), (j >> 1) & 1, kFuWaitLimitNs);
    }
    __syncwarp();
  } else if (warp >= 12) {                                   // ---- V codes -> operand images
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // a thread per pair of tokens and 4 (2-bit residuals: 2) 16-bit units of both
    const int tid = threadIdx.x - 384;
    constexpr int CH = D / 16;                               // 16-byte chunks of a pair's reference words
    const int p = tid / CH, u0 = (4 * (tid % CH)) ^ v_unit_swizzle(p, D / 4), g = u0 / 8;
    const bool has_ref = D == 128 || tid < 32 * CH;
    constexpr int W = RES == 2 ? 2 : 4, PR = RES ? D * RES / 16 / W : 1;   // residual words per thread, threads per pair
    const int rp = tid / PR, rc = tid % PR, ru0 = (W * rc) ^ v_unit_swizzle(rp, RROW / 2), rg = RES ? ru0 * 16 / (RES ? RES : 1) / 32 : 0;
    const bool has_res = RES && tid < 32 * PR;
    for (int j = 0; j < T; ++j) {
      const int st = j % kRawStages, s = j & 1;
      const uint8_t* const rec = smem + L::raw + st * L::kRaw;
      const uint8_t* const res = rec + L::kRef + RSIDE;      // V's part of the residual section
      const uint8_t* const vr = rec + SIDE;
      const int live = min(kTile, ctx - (kt0 + j) * kTile);  // cached tokens of the record
      bool good = mbar_wait_bounded(rawfull(st), (j / kRawStages) & 1, kFuWaitLimitNs);
      if (good && j >= 2) good = mbar_wait_bounded(vfree(s), ((j >> 1) - 1) & 1, kFuWaitLimitNs);
      if (__any_sync(RQ_FULL_MASK, !good)) {
        failed = true;
        break;
      }
      uint8_t* const img = smem + L::v + s * L::kImg;
      if (has_ref) {
        const uint4 w = *reinterpret_cast<const uint4*>(vr + p * D + (tid % CH) * 16);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 2 * p + e;
          const bool on = row < live;                        // (rows behind the context: zeros)
          uint32_t al = 0x3C003C00u;
          if (RES) al = *reinterpret_cast<const uint16_t*>(res + kTile * (RROW + 4 * NG) + row * 2) * 0x10001u;
          al = on ? al : 0u;
          const __half2 a2 = *reinterpret_cast<const __half2*>(&al);
          const Steps steps(on ? *reinterpret_cast<const uint32_t*>(vr + kTile * D / 2 + (row * NG + g) * 4) : 0u);
#pragma unroll
          for (int k = 0; k < 2; ++k) {                      // units u0 + 2 k, + 1: 8 channels
            uint32_t o[4];
            levels<4>(k ? __byte_perm(w.z, w.w, e ? 0x7632 : 0x5410) : __byte_perm(w.x, w.y, e ? 0x7632 : 0x5410), steps, o);
            const int chunk = u0 / 2 + k;
            *reinterpret_cast<uint4*>(img + (chunk / 8) * L::kPanel + panel_offset(row, chunk % 8)) =
                RES ? make_uint4(times(o[0], a2), times(o[1], a2), times(o[2], a2), times(o[3], a2))
                    : make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
      }
      if constexpr (RES != 0) {
        if (has_res) {
          uint32_t w[W];
          if constexpr (W == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(res + rp * 2 * RROW + rc * 8);
            w[0] = x.x, w[1] = x.y;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(res + rp * 2 * RROW + rc * 16);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = 2 * rp + e;
            const Steps steps(row < live ? *reinterpret_cast<const uint32_t*>(res + kTile * RROW + (row * NG + rg) * 4) : 0u);
#pragma unroll
            for (int k = 0; k < W / 2; ++k) {                // a token's word of two units
              uint32_t o[16 / RES];
              levels<RES>(__byte_perm(w[2 * k], w[2 * k + 1], e ? 0x7632 : 0x5410), steps, o);
#pragma unroll
              for (int q = 0; q < 4 / RES; ++q) {
                const int chunk = (ru0 + 2 * k) * (16 / RES) / 8 + q;
                *reinterpret_cast<uint4*>(img + (D / 64 + chunk / 8) * L::kPanel + panel_offset(row, chunk % 8)) =
                    make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
              }
            }
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(vfull(s));
        mbar_arrive(rawfree(st));
      }
    }
  } else if (warp >= 4) {                                    // ---- K codes -> operand images
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    // a thread per row and 32 codes of each section
    const int tid = threadIdx.x - 128;
    const int row = D == 128 ? tid >> 2 : tid >> 1, part = D == 128 ? tid & 3 : tid & 1;
    const bool has_ref = D == 128 || tid < 128;
    constexpr int W = RES == 2 ? 2 : 4, PR = RES ? NG * RES / W : 1;       // residual words per thread, threads per row
    const int rrow = tid / PR, rpart = tid % PR;
    const bool has_res = RES && tid < kTile * PR;
    for (int j = 0; j < T; ++j) {
      const int st = j % kRawStages, s = j & 1;
      const uint8_t* const rec = smem + L::raw + st * L::kRaw;
      const uint8_t* const res = rec + L::kRef;
      bool good = mbar_wait_bounded(rawfull(st), (j / kRawStages) & 1, kFuWaitLimitNs);
      if (good && j >= 2) good = mbar_wait_bounded(kfree(s), ((j >> 1) - 1) & 1, kFuWaitLimitNs);
      if (__any_sync(RQ_FULL_MASK, !good)) {
        failed = true;
        break;
      }
      uint8_t* const img = smem + L::k + s * L::kImg;
      if (has_ref) {
        // words `part` (d 64: 2 part, 2 part + 1) of every group
        const uint4 w = *reinterpret_cast<const uint4*>(rec + row * (D / 2) + part * 16);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        uint32_t al = 0x3C003C00u;
        if (RES) al = *reinterpret_cast<const uint16_t*>(res + kTile * (RROW + 4 * NG) + row * 2) * 0x10001u;
        const __half2 a2 = *reinterpret_cast<const __half2*>(&al);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int g = D == 128 ? i : i % 2, jj = D == 128 ? part : 2 * part + i / 2;
          const Steps steps(*reinterpret_cast<const uint32_t*>(rec + kTile * D / 2 + (row * NG + g) * 4));
          uint32_t o[4];
          levels<4>(ws[i], steps, o);
          *reinterpret_cast<uint4*>(img + (g / 2) * L::kPanel + panel_offset(row, (g % 2) * 4 + jj)) =
              RES ? make_uint4(times(o[0], a2), times(o[1], a2), times(o[2], a2), times(o[3], a2))
                  : make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      if constexpr (RES != 0) {
        if (has_res) {
          uint32_t ws[W];
          if constexpr (W == 2) {
            const uint2 w = *reinterpret_cast<const uint2*>(res + rrow * RROW + rpart * 8);
            ws[0] = w.x, ws[1] = w.y;
          } else {
            const uint4 w = *reinterpret_cast<const uint4*>(res + rrow * RROW + rpart * 16);
            ws[0] = w.x, ws[1] = w.y, ws[2] = w.z, ws[3] = w.w;
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const int word = rpart * W + i, g = word % NG, jj = word / NG;
            const Steps steps(*reinterpret_cast<const uint32_t*>(res + kTile * RROW + (rrow * NG + g) * 4));
            uint32_t o[16 / RES];
            levels<RES>(ws[i], steps, o);
#pragma unroll
            for (int c = 0; c < 4 / RES; ++c)
              *reinterpret_cast<uint4*>(img + (D / 64 + g / 2) * L::kPanel +
                                        panel_offset(rrow, (g % 2) * 4 + jj * (4 / RES) + c)) =
                  make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(kfull(s));
        mbar_arrive(rawfree(st));
      }
    }
  } else {                                                   // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    const int row = threadIdx.x;
    const uint32_t lanes = uint32_t(warp) << 21;
    float m = -INFINITY, l = 0.f, c = 1.f;
    if (warp < active) {
      const bool valid = row < rows;
      {   // queries -> tensor memory
        const uint4* const q = a.qimg + (unit * a.rows + min(row, rows - 1)) * (KD / 8);
#pragma unroll 1
        for (int x = 0; x < KD / 64; ++x) {
          uint32_t w[32];
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const uint4 v = q[8 * x + y];
            w[4 * y] = v.x, w[4 * y + 1] = v.y, w[4 * y + 2] = v.z, w[4 * y + 3] = v.w;
          }
          tc_st32(tQ + lanes + 32 * x, w);
        }
        c = a.qscale[unit * a.rows + min(row, rows - 1)];
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready);
      }
      for (int j = 0; j < T; ++j) {
        const int s = j & 1;
        const bool good = mbar_wait_bounded(sready(s), (j >> 1) & 1, kFuWaitLimitNs);
        if (__any_sync(RQ_FULL_MASK, !good)) {
          failed = true;
          break;
        }
        tc_fence_after();
        uint32_t v[kTile];
        tc_ld32(tS + 64 * s + lanes, v);
        tc_ld32(tS + 64 * s + lanes + 32, v + 32);
        tc_wait_ld();
        const int live = ctx - (kt0 + j) * kTile;
        if (live < kTile) {
#pragma unroll
          for (int x = 0; x < kTile; ++x)
            if (x >= live) v[x] = 0xff800000u;
        }
        float mx[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) mx[x] = __uint_as_float(v[x]);
#pragma unroll
        for (int x = 4; x < kTile; ++x) mx[x & 3] = fmaxf(mx[x & 3], __uint_as_float(v[x]));
        const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        if (__any_sync(RQ_FULL_MASK, mt > m + kWeightTop)) {
          const float mn = mt > m + kWeightTop ? mt - kWeightHead : m;
          const float f = m == -INFINITY ? 0.f : ex2(m - mn);
          l *= f;
          m = mn;
          if (j > 0) {                                       // rescale O (its last product is done)
            const bool fin = mbar_wait_bounded(vfree(s ^ 1), ((j - 1) >> 1) & 1, kFuWaitLimitNs);
            if (__any_sync(RQ_FULL_MASK, !fin)) {
              failed = true;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < KD / 16; ++x) {
              uint32_t o[16];
              tc_ld16(tO + lanes + 16 * x, o);
              tc_wait_ld();
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tc_st16(tO + lanes + 16 * x, o);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.f : -m;
        const uint64_t c2 = pack2(c, c), m2 = pack2(ms, ms);
        uint64_t sum = 0ull;
        uint32_t p[32];
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float p0, p1;
          unpack2(fma2(pack2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), c2, m2), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          sum = add2(sum, pack2(p0, p1));
          p[x] = pack_half2(p0, p1);
        }
        tc_st32(tS + 64 * s + lanes, p);
        float s0, s1;
        unpack2(sum, s0, s1);
        l += s0 + s1;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pready(s));
      }
      if (T > 0 && !failed) failed = !mbar_wait_bounded(done, 0, kFuWaitLimitNs);
      // partial record: m, l, pad, O_ref, O_res
      failed = __any_sync(RQ_FULL_MASK, failed);
      tc_fence_after();
      float* const part = a.part + ((unit * a.rows + min(row, rows - 1)) * a.n_splits + split) * (4 + 2 * D);
      if (valid) *reinterpret_cast<float2*>(part) = make_float2(m, l);
      auto store = [&](int x, auto order) {                  // 32 columns, channels in order
        uint32_t w[32];
        if (T > 0) {
          tc_ld32(tO + lanes + 32 * x, w);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) w[y] = 0u;
        }
        if (valid) {
#pragma unroll
          for (int y = 0; y < 32; y += 4)
            *reinterpret_cast<uint4*>(part + 4 + 32 * x + y) =
                make_uint4(w[order.at(y)], w[order.at(y + 1)], w[order.at(y + 2)], w[order.at(y + 3)]);
        }
      };
      struct Four { __device__ static constexpr int at(int c) { return image_position<4>(c); } };
      struct Residual { __device__ static constexpr int at(int c) { return image_position<RES ? RES : 4>(c); } };
#pragma unroll 1
      for (int x = 0; x < D / 32; ++x) store(x, Four());
#pragma unroll 1
      for (int x = D / 32; x < KD / 32; ++x) store(x, Residual());
      tc_fence_before();
    }
  }
  if (__syncthreads_or(failed) && threadIdx.x == 0) atomicOr(a.err, 1u);
  tc_fence_after();
  if (warp == 20) tc_free(tmem, 512);
}

size_t round1k(size_t n) { return (n + 1023) / 1024 * 1024; }

int plan_fused_splits(const rq_shape& s, int max_ctx) {
  const int tiles = (max_ctx + kTile - 1) / kTile;
  const int64_t units = int64_t(s.batch) * s.n_kv_heads, sms = device_sm_count();
  double best = 1e300;
  int found = 1;
  for (int k = 1; k <= tiles && k <= 64; ++k) {   // waves x (tiles + set-up, worth about six tiles)
    const double cost = double((units * k + sms - 1) / sms) * ((tiles + k - 1) / k + 6.0);
    if (cost < best - 1e-9) {
      best = cost;
      found = k;
    }
  }
  return found;
}

struct FusedLayout {
  int splits;
  size_t part, qimg, qscale, total;
};

FusedLayout fused_layout(const rq_shape& s, int loop, int n_new, int max_ctx, size_t budget) {
  FusedLayout l;
  const size_t rows = size_t(s.batch) * s.n_q_heads * n_new;
  const int kd = s.head_dim * (loop < s.n_loops - 1 ? 2 : 1);
  for (l.splits = plan_fused_splits(s, max_ctx);; --l.splits) {
    size_t o = kWsHeaderBytes;
    l.part = o;
    o = round1k(o + rows * l.splits * partial_floats(s) * 4);
    l.qimg = o;
    o = round1k(o + rows * kd * 2);
    l.qscale = o;
    o = round1k(o + rows * 4);
    l.total = o;
    if (o <= budget || l.splits == 1) return l;
  }
}

template <int D, int RES>
cudaError_t launch_fused(const FusedArgs& a, int batch, cudaStream_t stream) {
  using L = FusedSmem<D, RES>;
  static OncePerDevice once;
  cudaError_t e = once([] {
    return cudaFuncSetAttribute(fused_kernel<D, RES>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::total);
  });
  if (e != cudaSuccess) return e;
  const int64_t n_rows = int64_t(batch) * a.H * a.rows;
  fused_rows_kernel<D, RES><<<unsigned((n_rows + 3) / 4), 128, 0, stream>>>(a, int(n_rows));
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_after(true, fused_kernel<D, RES>, dim3(unsigned(a.n_splits), unsigned(a.H), unsigned(batch)), 768,
                      L::total, stream, a);
}

}  // namespace

size_t chunk_fused_workspace_bytes(const rq_shape& s, int loop, int n_new, int max_ctx, size_t budget) {
  return fused_layout(s, loop, n_new, max_ctx, budget).total;
}

cudaError_t launch_chunk_fused(const rq_shape& s, const rq_cache& cache, const rq_paging* paging,
                               const ChunkCall& c, void* ws, size_t ws_bytes, const float** part,
                               int* n_splits, cudaStream_t stream) {
  const FusedLayout l = fused_layout(s, c.loop, c.n_new, c.max_ctx, ws_bytes);
  char* const w = static_cast<char*>(ws);
  FusedArgs a;
  a.data = cache.data;
  a.rec_bytes = record_bytes(s);
  a.bt = paging ? paging->block_table : nullptr;
  a.max_pages = paging ? paging->max_pages : 0;
  a.n_pages = paging ? paging->n_pages : 0;
  a.cap = s.capacity;
  a.sec_off = loop_section_offset(s.head_dim, s.res_bits, c.loop);
  a.q = c.q;
  a.qs0 = c.q_strides[0];
  a.qs1 = c.q_strides[1];
  a.qs2 = c.q_strides[2];
  a.ksigns = cache.rot_signs[0];
  a.qimg = reinterpret_cast<uint4*>(w + l.qimg);
  a.qscale = reinterpret_cast<float*>(w + l.qscale);
  a.n_lens = c.n_lens;
  a.ctx_lens = c.ctx_lens;
  a.part = reinterpret_cast<float*>(w + l.part);
  a.err = reinterpret_cast<unsigned*>(w);
  a.H = s.n_kv_heads;
  a.heads = s.n_q_heads / s.n_kv_heads;
  a.n_new = c.n_new;
  a.max_ctx = c.max_ctx;
  a.n_splits = l.splits;
  a.rows = a.heads * c.n_new;
  a.scale_log2 = (s.softmax_scale > 0.f ? s.softmax_scale : 1.0f / sqrtf(float(s.head_dim))) * kLog2e;
  *part = a.part;
  *n_splits = l.splits;
  const int bits = c.loop < s.n_loops - 1 ? s.res_bits[c.loop] : 0;
  if (s.head_dim == 128)
    return bits == 0 ? launch_fused<128, 0>(a, s.batch, stream)
                     : bits == 2 ? launch_fused<128, 2>(a, s.batch, stream) : launch_fused<128, 4>(a, s.batch, stream);
  return bits == 0 ? launch_fused<64, 0>(a, s.batch, stream)
                   : bits == 2 ? launch_fused<64, 2>(a, s.batch, stream) : launch_fused<64, 4>(a, s.batch, stream);
}

}  // namespace rq
