// Chunk attention over a cache of this type.

#include "chunk.cuh"

namespace specv_chunk {

template <>
cudaError_t run<F16>(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  return run_any<F16>(P, k_map, v_map, stream);
}

}  // namespace specv_chunk
