// Appending to the 8-bit cache (include/rq_q8.h): two warps (d = 64: one) take one block of 16 slots of one
// (sequence, loop, kv-head, K or V); D / 8 lanes hold a row, 8 channels each.  The new rows are loaded and
// rotated, their largest magnitude gives the scale, and the codes follow from registers.
//
// Bound by instructions and occupancy (issue slots 73 % used): 1,024 tokens of 4 x 16 heads and 4 loops in 41 us
// without rotation, 4.9 TB/s, 57 us rotated.  A whole block a warp took 110 registers and 51 us (75 rotated);
// blocks of 256 threads, whose warps end together, 46 (77).  Head dim 64 takes a whole block a warp and spills
// some 25 registers for it.
#include <algorithm>

#include "rq_kernels.h"
#include "rq_q8.cuh"

namespace rq {
namespace {

struct AppendArgs {
  Q8View v;              // of loop_begin
  const uint16_t* kv;
  int64_t s0, s1, s2, s3, s4;
  const int32_t* n_lens;
  const int32_t* ctx_lens;
  Q8Rope rope;
  int32_t n_new, loops, blocks, cap;   // blocks: of 16 slots that n_new tokens touch at most
  int64_t units;
  int32_t vec;           // rows allow 16-byte loads
};

// Codes of 8 values under a scale whose inverse is `inv`.
template <int FMT>
__device__ __forceinline__ uint2 codes_of(const float (&f)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (FMT == RQ_Q8_INT8) {
      // under 2^23 + 2^22 a unit is worth 1: the sum's rounding is the code's, its low byte the code (a
      // magnitude is at most 127.25 here)
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __float_as_uint(fmaf(f[4 * k + i], inv, 12582912.f));
      w[k] = __byte_perm(__byte_perm(x[0], x[1], 0x0040), __byte_perm(x[2], x[3], 0x0040), 0x5410);
    } else {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k] * inv, f[4 * k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * k + 2] * inv, f[4 * k + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[k] = lo | (hi << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

// 8 codes as numbers.
template <int FMT>
__device__ __forceinline__ void values_of(uint2 w, float (&f)[8]) {
  const uint32_t x[2] = {q8_word<FMT>(w.x), q8_word<FMT>(w.y)};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t lo = q8_pair<FMT, 0>(x[k]), hi = q8_pair<FMT, 1>(x[k]);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[4 * k] = a.x;
    f[4 * k + 1] = a.y;
    f[4 * k + 2] = b.x;
    f[4 * k + 3] = b.y;
  }
}

// The larger magnitude (of any sign); not a number if either is none.
__device__ __forceinline__ float larger(float m, float x) {
  float y;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(m), "f"(x));
  return y;
}

template <int D, int FMT>
__global__ void __launch_bounds__(64, 16) q8_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int SPLIT = D / 64, LPR = D / 8, RPI = 32 / LPR, IT = kQ8Block / SPLIT / RPI;   // warps per block, lanes per row, rows at a time
  __shared__ uint32_t halves[2];                                     // largest magnitude of a warp's rows
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % LPR, half = warp % SPLIT;
  const int sub = lane / LPR + half * (kQ8Block / 2);
  int64_t u = int64_t(blockIdx.x) * (2 / SPLIT) + warp / SPLIT;
  if (u >= a.units) return;
  const int h = int(u % a.v.H);
  u /= a.v.H;
  const int kv = int(u & 1);
  u >>= 1;
  const int l = int(u % a.loops);
  u /= a.loops;
  const int blk = int(u % a.blocks), b = int(u / a.blocks);

  const int ctx = a.ctx_lens[b];
  int n = a.n_lens ? a.n_lens[b] : a.n_new;
  if (ctx < 0 || ctx >= a.cap || n < 0 || n > a.n_new) return;
  n = min(n, a.cap - ctx);
  const int k0 = (ctx / kQ8Block + blk) * kQ8Block;                  // the block's first slot
  const int t0 = max(ctx, k0), t1 = min(ctx + n, k0 + kQ8Block);     // slots of new tokens
  if (t0 >= t1) return;
  const int tile = k0 / kQ8Tile, part = k0 % kQ8Tile / kQ8Block;
  const int64_t rec = a.v.record(b, h, tile);
  if (rec < 0) return;
  uint8_t* const rows = a.v.codes + rec * a.v.rec_codes + int64_t(l * 2 + kv) * (kQ8Tile * D);
  float* const scale = a.v.scales + rec * a.v.rec_scales + (l * 2 + kv) * 4 + part;
  const float was = k0 < ctx ? *scale : 0.f;

  const uint16_t* const src = a.kv + b * a.s0 + kv * a.s2 + l * a.s3 + h * a.s4 + 8 * c;
  float f[IT][8];
  float largest = 0.f;
  uint4 raw[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = k0 + i * RPI + sub;
    raw[i] = t >= t0 && t < t1 ? q8_load8(src + (t - ctx) * a.s1, a.vec) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (kv == 0 && a.rope.table != nullptr) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int t = k0 + i * RPI + sub;
      int pos = -1;
      if (t >= t0 && t < t1) {
        pos = a.rope.positions ? a.rope.positions[int64_t(b) * a.n_new + t - ctx] : t;
        if (pos < 0 || pos >= a.rope.n_pos) {
          pos = -1;
          largest = __int_as_float(0x7fc00000);                      // as a row that is not finite
        }
      }
      const Q8Angles angles = q8_angles<D>(a.rope, pos, lane);
      q8_floats(raw[i], f[i]);
      q8_rotate<D>(f[i], a.rope, angles, lane);
    }
  } else {
#pragma unroll
    for (int i = 0; i < IT; ++i) q8_floats(raw[i], f[i]);
  }
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) largest = larger(largest, f[i][k]);
  // (a NaN's bits, without the sign, are above every number's)
  uint32_t most = __reduce_max_sync(RQ_FULL_MASK, __float_as_uint(largest) & 0x7fffffffu);
  if (SPLIT == 2) {
    if (lane == 0) halves[warp] = most;
    __syncthreads();
    most = max(most, halves[warp ^ 1]);
  }

  // the least exponent that holds them; bf16 bits: exponent field, 7 bits of the significand
  const uint32_t m16 = most < 0x7f800000u ? float_to_bf16_bits(__uint_as_float(most)) : 0x7f80u;
  constexpr int TOP = FMT == RQ_Q8_INT8 ? 126 : 96, K = FMT == RQ_Q8_INT8 ? 6 : 8;   // 127 = 2^6 (1 + 126/128), 448 = 2^8 (1 + 96/128)
  int e = kQ8LeastExp;
  if (m16 >= 0x80u) e = max(e, int(m16 >> 7) - 127 - K + (int(m16 & 127u) > TOP ? 1 : 0));
  const int e_old = k0 < ctx ? q8_exponent(was) : kQ8LeastExp;
  const bool bad = m16 >= 0x7f80u || e_old > 127;
  e = max(e, e_old);
  if (lane == 0 && half == 0 && (k0 >= ctx || bad || e > e_old)) *scale = bad ? __int_as_float(0x7fc00000) : q8_pow2(e);
  const float inv = bad ? 0.f : q8_pow2(-e);

  auto at = [&](int t) {
    const int r = t % kQ8Tile;
    return rows + r * D + (((c >> 1) ^ q8_swizzle<D>(r)) << 4) + (c & 1) * 8;
  };
  if (k0 < ctx && e > e_old && !bad) {                               // older rows under the new scale
    const float down = q8_pow2(-min(e - e_old, 60));                 // (2^-60 of any code is 0)
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int t = k0 + i * RPI + sub;
      if (t < ctx) {
        float g[8];
        values_of<FMT>(*reinterpret_cast<const uint2*>(at(t)), g);
        *reinterpret_cast<uint2*>(at(t)) = codes_of<FMT>(g, down);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = k0 + i * RPI + sub;
    if (t >= t0 && t < t1) *reinterpret_cast<uint2*>(at(t)) = bad ? make_uint2(0u, 0u) : codes_of<FMT>(f[i], inv);
  }
}

}  // namespace

cudaError_t launch_q8_append(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                             const uint16_t* kv_new, const int64_t strides[5], int loop_begin,
                             int loop_count, const int32_t* n_lens, int n_new, const int32_t* ctx_lens,
                             const Q8Rope& rope, cudaStream_t stream) {
  AppendArgs a = {};
  a.v = q8_view(s, cache, paging, loop_begin);
  a.kv = kv_new;
  a.s0 = strides[0];
  a.s1 = strides[1];
  a.s2 = strides[2];
  a.s3 = strides[3];
  a.s4 = strides[4];
  a.n_lens = n_lens;
  a.ctx_lens = ctx_lens;
  a.rope = rope;
  a.n_new = n_new;
  a.loops = loop_count;
  a.cap = s.capacity;
  // (no more tokens than slots are stored)
  a.blocks = (std::min(n_new, s.capacity) + 2 * kQ8Block - 2) / kQ8Block;
  a.units = int64_t(s.batch) * a.blocks * loop_count * 2 * s.n_kv_heads;
  bool vec = (reinterpret_cast<uintptr_t>(kv_new) & 15) == 0;
  for (int i = 0; i < 5; ++i) vec = vec && strides[i] % 8 == 0;
  a.vec = vec;
  const int each = 128 / s.head_dim;                                 // units of a CTA
  const unsigned grid = unsigned((a.units + each - 1) / each);
  if (s.head_dim == 128) {
    if (s.format == RQ_Q8_INT8)
      q8_append_kernel<128, RQ_Q8_INT8><<<grid, 64, 0, stream>>>(a);
    else
      q8_append_kernel<128, RQ_Q8_E4M3><<<grid, 64, 0, stream>>>(a);
  } else {
    if (s.format == RQ_Q8_INT8)
      q8_append_kernel<64, RQ_Q8_INT8><<<grid, 64, 0, stream>>>(a);
    else
      q8_append_kernel<64, RQ_Q8_E4M3><<<grid, 64, 0, stream>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace rq
