// Argument checks that the C entry points share (host code).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/rq.h"

namespace rq {

inline rq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? RQ_OK : RQ_ERR_CUDA; }

// Strides of an input: non-negative, and every element's offset in 63 bits.
inline bool strides_ok(const int64_t* strides, const int64_t* extents, int n) {
  int64_t last = 0;
  for (int i = 0; i < n; ++i) {
    if (strides[i] < 0) return false;
    const int64_t steps = extents[i] > 0 ? extents[i] - 1 : 0;
    if (steps > 0 && strides[i] > (INT64_MAX / 4 - last) / steps) return false;
    last += steps * strides[i];
  }
  return true;
}

// Does the span of bf16 rows of `d` elements at these (checked) strides meet [begin, end)?
inline bool overlaps(const uint16_t* p, const int64_t* strides, const int64_t* extents, int n, int d,
              uintptr_t begin, uintptr_t end) {
  int64_t last = d;
  for (int i = 0; i < n; ++i) last += (extents[i] - 1) * strides[i];
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(p), a1 = a0 + uintptr_t(last) * 2;
  return a0 < end && begin < a1;
}

}  // namespace rq
