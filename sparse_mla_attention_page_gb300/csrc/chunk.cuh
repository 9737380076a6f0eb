// Work list of the dense attention of new tokens, shared by its plan, its
// attention kernel and the merge of split units (chunk_plan.cu, chunk_attn.cu).
//
// A unit is a group of up to NC consecutive query rows of one request (row =
// token x head, tokens outermost) and takes the 128-key tiles up to the last
// key that its last row sees.  The units' tiles, one after another, are the
// global tile list; CTA c of the persistent grid owns the tiles
// [c n / grid, (c + 1) n / grid), so a unit may be spread over CTAs.  Lengths
// live on the GPU: a plan kernel writes the list into the workspace.
#pragma once
#include <cstdint>

#include "dense.h"

namespace dsa {

constexpr int kChunkTile = 128;      // keys of a tile

struct __align__(16) ChunkUnit {
  int64_t tile0;     // first global tile
  int64_t row0;      // first query row, counted over the whole batch (token * H + head)
  int32_t b;         // request
  int32_t cols;      // query rows, 1 .. NC
  int32_t r0;        // first row within the request
  int32_t vis0;      // keys that the request's first token sees (may be negative); all keys when not causal
  int32_t tiles;     // at least 1
  int32_t kv;        // the request's keys
  int32_t pad[2];
};

// A unit spread over CTAs c0 .. c1; its parts lie in the slots slot0, 2 (c0 + 1), 2 (c0 + 2), ...
struct ChunkSplit {
  int32_t unit, c0, c1, slot0;
};

struct ChunkHeader {
  int64_t n_tiles;
  int32_t n_units, n_splits;
};

// Everything a call needs; the pointers from hdr on lie in the workspace.
struct ChunkWork {
  ChunkArgs a;
  int nc;                  // query rows of a unit
  int64_t max_units;
  int grid;                // CTAs of the attention grid
  uint64_t wait_ns;
  ChunkHeader* hdr;
  ChunkUnit* units;
  int32_t* cta_unit;       // [grid] the unit of each CTA's first tile
  ChunkSplit* splits;      // [grid]
  float* part_lse;         // [2 grid][nc]
  float* part_o;           // [2 grid][nc][512] normalised
};

__host__ __device__ __forceinline__ int64_t chunk_tile_begin(int64_t c, int64_t n_tiles, int grid) {
  return c * n_tiles / grid;
}

// Keys that row r of a unit's request sees.
__device__ __forceinline__ int chunk_visible(const ChunkArgs& a, const ChunkUnit& u, int col) {
  if (!a.causal) return u.kv;
  const int64_t v = (int64_t)u.vis0 + (u.r0 + col) / a.H;
  return v < 0 ? 0 : v > u.kv ? u.kv : (int)v;
}

void launch_chunk_plan(const ChunkWork& w, cudaStream_t stream);
bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream);

}  // namespace dsa
