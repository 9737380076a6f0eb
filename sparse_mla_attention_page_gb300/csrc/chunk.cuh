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
constexpr int kLoopParts = 24;       // rows of up to so many parts over prefix and own keys are joined so, kFewParts at a time
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
// kernel and the join: three tiles.  us there / on the dense path of single tokens,
// by the tiles that they save a CTA, about 2 / 3 / 4 / 6:
//   64 of 4 heads    raw 18.7 / 15.8  19.3 / 18.1  19.5 / 19.3  20.6 / 21.6   656 bytes 23.4 / 19.6  23.2 / 22.2  22.1 / 22.9  25.0 / 27.0
//   64 of 16 heads   raw 23.6 / 19.8  24.9 / 22.0  26.3 / 24.4  28.8 / 28.9   416 bytes 34.0 / 32.4  38.3 / 38.5  42.0 / 44.7  50.1 / 57.0
//   16 of 8 heads    raw 19.4 / 20.9  23.5 / 22.1  23.7 / 23.3  24.9 / 26.7   656 bytes 23.1 / 23.7  27.3 / 25.8  27.3 / 27.5  29.6 / 32.8
//   16 of 40 heads   raw 23.8 / 24.5  26.3 / 27.1  29.5 / 30.5  33.8 / 36.7   656 bytes 31.4 / 32.2  35.4 / 38.2  41.9 / 43.6  48.8 / 57.9
//   64 of 48 heads   raw 37.9 / 24.3  41.6 / 30.2  44.2 / 40.0  52.3 / 50.0   416 bytes 62.3 / 52.4  75.2 / 71.6  86.9 / 86.6  109 / 116
// (the last have a unit a CTA on the dense path, nothing spread).
constexpr int kJoinCost = 3 * kTileCost;
// Whether they could, by the sizes alone.  A request's rows are a multiple of
// gcd(H, 32), so its last unit has at most 32 less that many columns to spare, and
// packing saves no more than the units that the spare columns of all make up: none
// where the heads are a multiple of 32.  Beside that: where the dense path spreads
// long units over so many CTAs that its merge goes by slices, but the join takes the
// parts in a loop, the join alone makes up for the rest, whatever is shared.  us there /
// on the dense path, behind 12 / 24 / 80 tiles:
//   16 of 32 heads   raw 18.3 / 19.2  20.4 / 32.8  28.2 / 40.4   656 bytes 22.8 / 31.2  25.8 / 37.6  42.0 / 53.0
//   4 of 64 heads    raw 18.7 / 23.7  20.8 / 24.0  24.8 / 27.6   416 bytes 25.1 / 30.0  27.2 / 30.3  38.5 / 40.7
//   16 of 16 heads   raw 18.7 / 15.5  19.8 / 24.8  24.9 / 31.6   656 bytes 22.4 / 22.9  23.6 / 27.7  33.1 / 37.9
//   16 of 8 heads    raw 17.2 / 14.1  19.3 / 20.4  24.8 / 27.2   656 bytes 21.3 / 19.5  23.0 / 23.2  29.8 / 33.3
//   10 of 16 heads   raw 17.9 / 19.7  19.8 / 20.8  24.4 / 25.1   656 bytes 21.4 / 21.9  23.9 / 23.3  29.6 / 29.9
// (64 of 32 heads, of two parts each, behind 32 and 64 raw tiles 38.9 / 36.6, 54.7 / 52.1.)
inline bool sharing_possible(const ChunkArgs& a, int ctas) {
  const int64_t rows = (int64_t)a.T * a.H, tiles = (int64_t)a.max_pages * a.page_size / kChunkTile;
  if (rows > (int64_t)a.B * kSharedRows) return false;
  const int spare = 32 - (a.H % 32 == 0 ? 32 : a.H & -a.H);
  if ((int64_t)a.B * spare / 32 * tiles * kTileCost >= (int64_t)ctas * kJoinCost) return true;
  const int nc = chunk_columns(a.T, a.H, a.B);
  const int64_t units = a.B * (((rows + a.B - 1) / a.B + nc - 1) / nc);
  return units * kFewParts < ctas && units * kLoopParts >= ctas && tiles >= kLoopParts;
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
