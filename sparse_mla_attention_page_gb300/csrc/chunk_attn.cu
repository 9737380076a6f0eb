// The dense attention of new tokens (chunk_kernel.cuh) over each request's rows.
#include "chunk_kernel.cuh"

namespace dsa {

// 16 rows where the average request has no more, else 32: half the columns
// need less of everything but the rows' bytes, two units of 16 read the rows
// twice.  us with 16 / 32, 64 requests of up to 8192 rows: 16 heads, raw 40.6 /
// 43.4, rope 52.4 / 58.8; 24 heads, raw 57.3 / 45.9, rope 81.9 / 61.1; one of
// 131072: 16 heads, raw 21.7 / 23.3; 32 heads 29.3 / 23.8.
int chunk_columns(int T, int H, int B) {
  const int64_t rows = ((int64_t)T * H + B - 1) / B;     // of an average request
  return rows <= kFewestRows ? kFewestRows : 32;
}

bool launch_chunk_attn(const ChunkWork& work, cudaStream_t stream) {
  ChunkWork w = work;
  ChunkMaps maps{};
  if (!prepare(w, maps)) return false;
  return w.nc == 16 ? launch_nc<16, false>(w, maps, stream) : launch_nc<32, false>(w, maps, stream);
}

}  // namespace dsa
