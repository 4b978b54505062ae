// Decode-kernel variants of the chunk calls over a contiguous cache (the kernel template is in
// rq_decode_mma.cuh).
#include "rq_decode_mma.cuh"

namespace rq {

KernelFn pick_chunk(int D, bool res4, int nr, int pk) {
  if (pk == 2) return pick_chunk_pk<false, 2>(D, res4, nr);
  return pk == 1 ? pick_chunk_pk<false, 1>(D, res4, nr) : pick_chunk_pk<false, 0>(D, res4, nr);
}

}  // namespace rq
