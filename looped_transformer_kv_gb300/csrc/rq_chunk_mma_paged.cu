// Decode-kernel variants of the chunk calls over a paged cache (the kernel template is in
// rq_decode_mma.cuh).
#include "rq_decode_mma.cuh"

namespace rq {

KernelFn pick_chunk_paged(int D, bool res4, int nr, int pk) {
  if (pk == 2) return pick_chunk_pk<true, 2>(D, res4, nr);
  return pk == 1 ? pick_chunk_pk<true, 1>(D, res4, nr) : pick_chunk_pk<true, 0>(D, res4, nr);
}

}  // namespace rq
