// Chunk attention over a cache of this type.

#include "chunk.cuh"
#include "single.cuh"

namespace specv_chunk {

template <>
cudaError_t run<F16>(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  if (singles(P))
    return P.cache.head_dim <= 64 ? launch_single<F16, 64>(P, stream) : launch_single<F16, 128>(P, stream);
  return run_any<F16>(P, k_map, v_map, stream);
}

}  // namespace specv_chunk
