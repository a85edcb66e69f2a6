// Chunk attention over a cache of this type.

#include "chunk.cuh"
#include "single.cuh"

namespace specv_chunk {

template <>
cudaError_t run<Bf16>(const Params& P, const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream) {
  if (singles(P))
    return P.cache.head_dim <= 64 ? launch_single<Bf16, 64>(P, stream) : launch_single<Bf16, 128>(P, stream);
  return run_any<Bf16>(P, k_map, v_map, stream);
}

}  // namespace specv_chunk
