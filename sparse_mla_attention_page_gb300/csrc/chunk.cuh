// Work list of the dense attention of new tokens, shared by the attention
// kernel, its plan and the merge of split units (chunk_attn.cu,
// chunk_plan.cuh, chunk_merge.cu).
//
// A unit is a group of up to NC consecutive query rows of one request (row =
// token x head, tokens outermost) and takes the 128-key tiles up to the last
// key that its last row sees.  The units' tiles, one after another, are the
// global tile list; CTA c of the persistent grid owns a range of it, so a unit
// may be spread over CTAs.  The ranges are cut evenly by cost: a unit counts
// chunk_unit_cost more than its tiles, for its query operand and its output.
// Lengths live on the GPU: every CTA of the attention kernel forms the list's
// prefix sums for itself.
#pragma once
#include <cstdint>

#include "dense.h"

namespace dsa {

constexpr int kChunkTile = 128;      // keys of a tile

// Costs of a tile, and of a unit beside its tiles'.  us of five prompts of up to
// 2047 tokens and 16 heads, units of 1 to 16 tiles, for a unit cost of 3 / 4 / 5 / 6 / 7:
//   rows by TMA       raw 242 / 218 / 202 / 199 / 204   scaled 310 / 284 / 287 / 294 / 295   rope 373 / 353 / 361 / 365 / 371
//   rows one by one   raw 277 / 250 / 235 / 239 / 245   scaled 321 / 302 / 311 / 315 / 325   rope 377 / 380 / 388 / 397 / 403
constexpr int kTileCost = 2;
constexpr int chunk_unit_cost(int layout) { return layout == DSA_KV_RAW512 ? 5 : 4; }

struct __align__(16) ChunkUnit {
  int64_t tile0;     // first global tile
  int64_t row0;      // first query row, counted over the whole batch (token * H + head)
  int32_t b;         // request
  int32_t cols;      // query rows, 1 .. NC
  int32_t r0;        // first row within the request
  int32_t vis0;      // keys that the request's first token sees (may be negative); all keys when not causal
  int32_t tiles;     // at least 1
  int32_t kv;        // the request's keys
  int32_t last;      // keys that the unit's last row sees
  int32_t pad;
};

// A unit spread over CTAs c0 ..: its parts lie in the slots slot0, 2 (c0 + 1), 2 (c0 + 2), ...
struct __align__(16) ChunkSplit {
  int64_t row0;      // as of the unit
  int32_t cols;
  int32_t parts;     // 0: no split unit begins in this CTA
  int32_t slot0, next;
  int32_t pad[2];
};
constexpr int kFewParts = 8;         // split units of up to so many parts are merged a thread for each 4 dims
constexpr int kMaxCtas = 1024;       // of the attention grid (one per SM); parts of a unit

// Everything a call needs; the pointers from hdr on lie in the workspace.
struct ChunkWork {
  ChunkArgs a;
  int nc;                  // query rows of a unit
  int64_t max_units;
  int grid;                // CTAs of the attention grid
  int box_shift;           // log2 of the rows of a TMA box; 0: rows are copied one by one
  int unit_cost;
  uint64_t wait_ns;
  ChunkUnit* units;        // [max_units + 1]; those that begin inside a CTA's range
  ChunkSplit* splits;      // [grid] by the CTA in which the unit begins
  float* part_lse;         // [2 grid][nc]
  float* part_o;           // [2 grid][nc][512] normalised
};

// Keys that row r of a unit's request sees.
__device__ __forceinline__ int chunk_visible(const ChunkArgs& a, const ChunkUnit& u, int col) {
  if (!a.causal) return u.kv;
  const int64_t v = (int64_t)u.vis0 + (u.r0 + col) / a.H;
  return v < 0 ? 0 : v > u.kv ? u.kv : (int)v;
}

bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream);

}  // namespace dsa
