// The dense attention of new tokens (chunk_kernel.cuh) where groups of requests
// begin with common rows: units of a prefix, of a request's own keys, and of
// requests alone in one launch, then their join (chunk_merge.cu).
//
// What sharing saves is tiles.  A unit reads its rows from the L2 cache either
// way; with 16 heads a request of one token fills half of a unit's 32 columns,
// with 8 a quarter, and packed rows fill them all.  The work is bound as that of
// the dense attention: us of a tile of 32 columns about those of one of 16.
#include "chunk_kernel.cuh"

namespace dsa {

bool launch_prefix_attn(const ChunkWork& work, cudaStream_t stream) {
  ChunkWork w = work;
  ChunkMaps maps{};
  return prepare(w, maps) && launch_nc<32, true>(w, maps, stream);
}

}  // namespace dsa
