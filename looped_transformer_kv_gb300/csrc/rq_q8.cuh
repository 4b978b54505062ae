// The 8-bit cache (include/rq_q8.h): what its kernels share.
#pragma once

#include <cuda_fp8.h>

#include "../../include/rq_q8.h"
#include "rq_common.cuh"
#include "rq_ptx.cuh"

namespace rq {

constexpr int kQ8Tile = 64, kQ8Block = 16;
constexpr int kQ8LeastExp = -100;   // exponent of the smallest scale
constexpr int kMostUp = 110;        // exponent of what brings queries into fp16's range, at most

struct Q8View {          // one loop's part of a cache
  uint8_t* codes;        // + loop * 2 * 64 * d
  float* scales;         // + loop * 8
  int64_t rec_codes;     // bytes, floats from one record to the next
  int32_t rec_scales;
  const int32_t* bt;     // block table, or null
  int32_t max_pages, n_pages;
  int32_t H, tiles;      // tiles of a sequence

  // Record of a tile of (b, h); -1: a block-table entry that is no page.
  __device__ __forceinline__ int64_t record(int b, int h, int tile) const {
    if (bt == nullptr) return (int64_t(b) * H + h) * tiles + tile;
    const int page = bt[int64_t(b) * max_pages + tile];
    return page < 0 || page >= n_pages ? -1 : int64_t(page) * H + h;
  }
};

struct Q8Rope {
  const float* table;         // null: no rotation
  const int32_t* positions;
  int32_t n_pos, rot, interleaved;
};

// XOR of a row's 16-byte chunk index.
template <int D>
__host__ __device__ __forceinline__ constexpr int q8_swizzle(int t) {
  return D == 128 ? (t & 7) : ((t >> 1) & 3);
}

// 8 channels of a bf16 row.
__device__ __forceinline__ uint4 q8_load8(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = uint32_t(p[2 * k]) | (uint32_t(p[2 * k + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint2 q8_load4(const uint16_t* p, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p);
  return make_uint2(uint32_t(p[0]) | (uint32_t(p[1]) << 16), uint32_t(p[2]) | (uint32_t(p[3]) << 16));
}
__device__ __forceinline__ void q8_floats(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}

// The angles of a lane's 8 channels at a position, of a row held by D / 8 neighbouring lanes; below 0
// (the same in a row's lanes): none.
struct Q8Angles {
  float4 a[4];           // (interleaved: two)
  bool turned;
};
template <int D>
__device__ __forceinline__ Q8Angles q8_angles(const Q8Rope& rope, int pos, int lane) {
  Q8Angles r;
  const int c = lane % (D / 8), half = rope.rot / 16;      // half: lanes of the first channels of the pairs
  r.turned = pos >= 0 && 8 * c < rope.rot;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.a[k] = make_float4(1.f, 0.f, 1.f, 0.f);
  if (!r.turned) return r;
  const float* const row = rope.table + int64_t(pos) * rope.rot + (rope.interleaved ? 8 * c : 16 * (c >= half ? c - half : c));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < 2 || !rope.interleaved) r.a[k] = *reinterpret_cast<const float4*>(row + 4 * k);
  return r;
}

// Rotates a pair; each product and sum is rounded.
__device__ __forceinline__ void q8_turn(float& x, float& y, float c, float s) {
  const float x0 = x, y0 = y;
  x = __fsub_rn(__fmul_rn(x0, c), __fmul_rn(y0, s));
  y = __fadd_rn(__fmul_rn(y0, c), __fmul_rn(x0, s));
}

// Rotates the row.  Every lane of the warp calls it.
template <int D>
__device__ __forceinline__ void q8_rotate(float (&f)[8], const Q8Rope& rope, const Q8Angles& r, int lane) {
  if (rope.interleaved) {
    if (r.turned) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        q8_turn(f[4 * k], f[4 * k + 1], r.a[k].x, r.a[k].y);
        q8_turn(f[4 * k + 2], f[4 * k + 3], r.a[k].z, r.a[k].w);
      }
    }
    return;
  }
  const int c = lane % (D / 8), half = rope.rot / 16;
  const bool second = c >= half;
  const float sign = second ? 1.f : -1.f;
  const int partner = lane - c + (8 * c < rope.rot ? (second ? c - half : c + half) : c);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float o0 = __shfl_sync(RQ_FULL_MASK, f[2 * k], partner);
    const float o1 = __shfl_sync(RQ_FULL_MASK, f[2 * k + 1], partner);
    if (r.turned) {
      const float4 a = r.a[k];
      // (a product with 1 or -1 is exact: the sum's is the only rounding of the last step)
      f[2 * k] = __fmaf_rn(__fmul_rn(o0, a.y), sign, __fmul_rn(f[2 * k], a.x));
      f[2 * k + 1] = __fmaf_rn(__fmul_rn(o1, a.w), sign, __fmul_rn(f[2 * k + 1], a.z));
    }
  }
}

// The power of two 2^e, -126 <= e <= 127.
__device__ __forceinline__ float q8_pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

// Exponent of a scale (a power of two, or not a number: 128).
__device__ __forceinline__ int q8_exponent(float scale) { return int(__float_as_uint(scale) >> 23 & 255) - 127; }

// The lower or upper two codes of a word as fp16 numbers, exact.  int8: `w` is the word with every
// sign bit flipped (q8_word), so that a byte under 1024's exponent is 1024 + 128 + code.
template <int FMT>
__device__ __forceinline__ uint32_t q8_word(uint32_t w) {
  return FMT == RQ_Q8_INT8 ? w ^ 0x80808080u : w;
}
template <int FMT, int HALF>
__device__ __forceinline__ uint32_t q8_pair(uint32_t w) {
  uint32_t out;
  if (FMT == RQ_Q8_INT8) {
    const uint32_t t = __byte_perm(w, 0x64646464u, HALF ? 0x4342 : 0x4140);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(out) : "r"(t), "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, %2;\n\t}"
        : "=r"(out) : "r"(w), "h"(uint16_t(HALF ? w >> 16 : w)));
  }
  return out;
}

struct Q8Call {          // an attention call, arguments as in include/rq_q8.h
  const uint16_t* q;
  int64_t q_strides[3];
  int loop;
  const int32_t* n_lens;
  int n_new;
  const int32_t* ctx_lens;
  int max_ctx, window, n_sink;
  Q8Rope rope;
  uint16_t* out;
};

size_t q8_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx, int window, int n_sink);
cudaError_t launch_q8_attention(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                                const Q8Call& c, void* ws, cudaStream_t stream);
// Few rows a kv-head (rq_q8_stream.cu), many (rq_q8_rows.cu); their workspaces.
size_t q8_stream_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx);
cudaError_t launch_q8_stream(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                             const Q8Call& c, void* ws, cudaStream_t stream);
size_t q8_rows_workspace_bytes(const rq_q8_shape& s, int n_new, int max_ctx, int window, int n_sink);
cudaError_t launch_q8_rows(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                           const Q8Call& c, void* ws, cudaStream_t stream);
cudaError_t launch_q8_append(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging,
                             const uint16_t* kv_new, const int64_t strides[5], int loop_begin,
                             int loop_count, const int32_t* n_lens, int n_new, const int32_t* ctx_lens,
                             const Q8Rope& rope, cudaStream_t stream);

inline Q8View q8_view(const rq_q8_shape& s, const rq_q8_cache& cache, const rq_paging* paging, int loop) {
  Q8View v = {};
  v.codes = cache.codes + int64_t(loop) * 2 * kQ8Tile * s.head_dim;
  v.scales = cache.scales + loop * 8;
  v.rec_codes = int64_t(s.n_loops) * 2 * kQ8Tile * s.head_dim;
  v.rec_scales = s.n_loops * 8;
  v.bt = paging ? paging->block_table : nullptr;
  v.max_pages = paging ? paging->max_pages : 0;
  v.n_pages = paging ? paging->n_pages : 0;
  v.H = s.n_kv_heads;
  v.tiles = s.capacity / kQ8Tile;
  return v;
}

}  // namespace rq
