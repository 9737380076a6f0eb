// Work list of the dense attention of new tokens, shared by the attention
// kernel, its plan and the merge of split units (chunk_kernel.cuh,
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
//
// Shared prefixes.  The requests of a group begin with common rows.  Where that
// takes fewer tiles, their query rows are packed into units of the prefix alone,
// and each request keeps units over its own keys; the two results of a row are
// joined as those of split units are.
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
enum ChunkSide { kAlone = 0, kPrefix = 1, kOwn = 2 };   // all of a row's keys; those it shares; the others
struct __align__(16) SharedUnit : ChunkUnit {
  int32_t key0;      // the request's key that the unit's first one is
  int32_t mate;      // of a kOwn unit: the unit that holds its first row's part over the prefix,
  uint8_t side;      // ChunkSide
  uint8_t mate_col;  // and that row's column there
  int16_t pad2;
  int16_t slot0;     // parts > 0: spread over CTAs, its parts in the slots slot0, then as of ChunkSplit
  int16_t parts;
};
static_assert(sizeof(ChunkUnit) == 48 && sizeof(SharedUnit) == 64, "whole 16-byte words");
// The kernels with groups of requests (kShared) are built apart from those
// without: these ran up to 6 % slower with the other's code in them.
template <bool kShared>
struct UnitOf {
  using type = ChunkUnit;
};
template <>
struct UnitOf<true> {
  using type = SharedUnit;
};
template <bool kShared>
using Unit = typename UnitOf<kShared>::type;

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
  void* units;             // Unit<kShared>[max_units + 1]; those that begin inside a CTA's range
  ChunkSplit* splits;      // [grid] by the CTA in which the unit begins
  float* part_lse;         // [2 grid][nc]
  float* part_o;           // [2 grid][nc][512] normalised
  // With shared prefixes (a.G > 0) the parts are followed by rows of kPrefix and
  // kOwn units that are not spread over CTAs: part joined0 + (side - 1) T H + row.
  int64_t joined0;
  int32_t* n_units;        // all of them; those of requests, which come first
};
// Sharing is for batches of few query rows a request; at most so many on average
// (eight units each: packing rows could save one of them at most).
constexpr int kSharedRows = 256;
// What all groups together could save, a CTA, for a call to go to the shared
// kernel and the join: about four tiles.  us there / on the dense path, 16 heads over raw rows, by the tiles saved: 64 single
// tokens behind 2048 (2.9) 31.0 / 28.7, 4096 (6.2) 33.2 / 35.2, 8192 (13) 43.4 /
// 51.5, 32768 (54) 90.6 / 144.9; four behind 32768 (3.4) 26.9 / 25.0.
constexpr int kJoinCost = 4 * kTileCost;
// Whether they could: packing rows saves less than a unit a request, of
// the tiles that the page table has room for.
inline bool sharing_possible(const ChunkArgs& a, int ctas) {
  return (int64_t)a.T * a.H <= (int64_t)a.B * kSharedRows &&
         (int64_t)(a.B - 1) * ((int64_t)a.max_pages * a.page_size / kChunkTile) * kTileCost >= (int64_t)ctas * kJoinCost;
}

template <bool kShared>
__device__ __forceinline__ Unit<kShared>* units_of(const ChunkWork& w) {
  return static_cast<Unit<kShared>*>(w.units);
}

// Keys that row r of a unit's request sees.
template <class U>
__device__ __forceinline__ int chunk_visible(const ChunkArgs& a, const U& u, int col) {
  if (!a.causal) return u.kv;
  if constexpr (sizeof(U) == sizeof(SharedUnit)) {
    if (u.side == kPrefix) return u.kv;
  }
  const int64_t v = (int64_t)u.vis0 + (u.r0 + col) / a.H;
  return v < 0 ? 0 : v > u.kv ? u.kv : (int)v;
}

bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream);
bool launch_prefix_merge(const ChunkWork& w, cudaStream_t stream);

}  // namespace dsa
