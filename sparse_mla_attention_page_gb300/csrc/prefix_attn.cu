// The dense attention of new tokens (chunk_kernel.cuh) where groups of requests
// begin with common rows: units of a prefix, of a request's own keys, and of
// requests alone in one launch, then their join (chunk_merge.cu).
//
// What sharing saves is tiles, not bytes: a unit reads its rows from the L2 cache
// whoever read them before.  With 16 heads a request of one token fills half of a
// unit's 32 columns, with 8 a quarter; packed rows fill them all, and a tile of 32
// columns takes 1.1 to 1.3 times one of 16.  So it is bound as the dense attention
// is (shared-memory banks over raw rows, the way of a row block through the ring
// over the others), after a plan and before a join that take some 3 and 5 us more.
// us with / without sharing: 64 single tokens of 16 heads behind 8192 raw rows
// 42 / 50, behind 32768 90 / 145, of 8 heads behind 8192 33 / 50; 96 requests of 2
// tokens and 8 heads behind four prefixes of up to 6000 rows of 656 bytes 61 / 69;
// 128 single tokens of 8 heads behind 32768 rows of 656 bytes 162 / 376, of 416
// 233 / 692.  (Multiples of 32 heads fill the units by themselves: nothing is shared.)
#include "chunk_kernel.cuh"

namespace dsa {

bool launch_prefix_attn(const ChunkWork& work, cudaStream_t stream) {
  ChunkWork w = work;
  ChunkMaps maps{};
  return prepare(w, maps) && launch_nc<32, true>(w, maps, stream);
}

}  // namespace dsa
