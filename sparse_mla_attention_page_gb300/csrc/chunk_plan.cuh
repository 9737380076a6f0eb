// The plan of the dense attention of new tokens: each CTA's range of the tile
// list (chunk.cuh), found by every CTA for itself at its start.
//
// Two prefix sums over the block's threads (units of each request, tiles of
// each unit); the thread whose units hold the range's border fills in the
// start, and the units that begin inside the range go to the workspace, for
// the producers.  (A plan kernel of one block in front, whose list every CTA
// read back, cost a launch and two trips to memory more: 12.9 us against 10.1
// for one token over 101 rows, 45 against 40 for 64 requests of up to 8192 raw
// rows, 39 against 35 for one request of 131072 scaled rows.  The sums over
// the thousands of units of a long chunk are below a percent of its time.)
#pragma once
#include "chunk.cuh"
#include "dsa_common.cuh"
#include "scan.cuh"

namespace dsa {

struct Request {
  int t0, n, kv, err;
};

// Query rows [t0, t0 + n) and keys of request b, made safe.
__device__ __forceinline__ Request request_of(const ChunkArgs& a, int b) {
  Request r;
  r.t0 = __ldg(a.cu_q + b);
  const int t1 = __ldg(a.cu_q + b + 1);
  r.kv = __ldg(a.kv_lens + b);
  const int room = a.max_pages * a.page_size;
  r.err = 0;
  r.n = t1 - r.t0;
  if (r.t0 < 0 || t1 < r.t0 || t1 > a.T) {
    r.err = DSA_DEV_ERR_LENGTH;
    r.t0 = r.n = 0;
  }
  if (r.kv < 0 || r.kv > room) {
    r.err = DSA_DEV_ERR_LENGTH;
    r.kv = r.kv < 0 ? 0 : room;
  }
  return r;
}

__device__ __forceinline__ int units_of(const ChunkArgs& a, const Request& r, int nc) {
  return (int)(((int64_t)r.n * a.H + nc - 1) / nc);
}

// Entry of the i-th unit of request b (tile0 is filled in later).
__device__ __forceinline__ ChunkUnit unit_of(const ChunkArgs& a, const Request& r, int b, int i, int nc) {
  ChunkUnit u;
  const int64_t rows = (int64_t)r.n * a.H, r0 = (int64_t)i * nc;
  u.tile0 = 0;
  u.row0 = (int64_t)r.t0 * a.H + r0;
  u.b = b;
  u.cols = (int)(rows - r0 < nc ? rows - r0 : nc);
  u.r0 = (int)r0;
  u.vis0 = a.causal ? r.kv - r.n + 1 : r.kv;
  u.kv = r.kv;
  u.last = chunk_visible(a, u, u.cols - 1);
  u.tiles = u.last <= kChunkTile ? 1 : (u.last - 1) / kChunkTile + 1;
  u.pad = 0;
  return u;
}

// A CTA's part of the tile list.
struct ChunkRange {
  int64_t t0, t1;    // global tiles
  int unit;          // that the first one belongs to
};

// Few short units, a CTA each: taken where no unit has more tiles than a CTA
// would get of split ones and this many.  us with / without, two tiles more:
// 2 x 20 tokens of 32 heads over 300, raw 13.7 / 18.6, rope 18.1 / 21.8; 30
// single tokens over up to 300, raw 12.5 / 13.9; 300 tokens of 8 heads, raw
// 13.8 / 19.0; three tiles more (16 single tokens over up to 500): raw 13.5 /
// 13.7, rope 16.2 / 16.4.
constexpr int kWholeTiles = 2;

constexpr int kPlanScratch = DSA_MAX_REQUESTS * 4 + 256;   // bytes of shared memory

// By all THREADS threads; mine and start (the range's first unit) lie in
// shared memory and hold after the caller's next barrier.
template <int THREADS>
__device__ __forceinline__ void chunk_plan(const ChunkWork& w, uint8_t* scratch, ChunkRange& mine, ChunkUnit& start) {
  int32_t* first_unit = reinterpret_cast<int32_t*>(scratch);                             // [B]
  int64_t* sums = reinterpret_cast<int64_t*>(scratch + DSA_MAX_REQUESTS * 4);
  const ChunkArgs& a = w.a;
  const int tid = threadIdx.x, cta = blockIdx.x;
  int err = 0;
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t here = 0;
  int last_units = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    err |= r.err;
    last_units = units_of(a, r, w.nc);
    here += last_units;
  }
  int64_t total;
  int64_t at = block_scan<THREADS>(here, &total, sums);
  if (total > w.max_units) {     // only when the requests' ranges overlap: the list has no room
    err = DSA_DEV_ERR_LENGTH;
    total = 0;
  }
  if (err && cta == 0) set_err(a.err, err);
  const int n_units = (int)total;
  for (int b = b0; b < b1; ++b) {
    first_unit[b] = (int)min(at, (int64_t)INT32_MAX);
    at += b + 1 == b1 ? last_units : units_of(a, request_of(a, b), w.nc);
  }
  __syncthreads();

  // thread -> a run of consecutive units
  const int uper = (n_units + THREADS - 1) / THREADS;
  const int u0 = (int)min((int64_t)tid * uper, (int64_t)n_units), u1 = min(u0 + uper, n_units);
  const int first_b = u0 < u1 ? scan_owner(first_unit, a.B, u0) : 0;
  int64_t tiles = 0;
  ChunkUnit only{};              // of a thread that has one unit: worked out once
  auto walk = [&](auto&& visit) {
    if (u1 - u0 == 1 && tiles > 0) return visit(u0, only);
    int b = first_b;
    Request r{};
    bool have = false;
    for (int u = u0; u < u1; ++u) {
      while (b + 1 < a.B && first_unit[b + 1] <= u) {
        ++b;
        have = false;
      }
      if (!have) r = request_of(a, b);
      have = true;
      visit(u, unit_of(a, r, b, u - first_unit[b], w.nc));
    }
  };
  walk([&](int, const ChunkUnit& e) {
    tiles += e.tiles;
    only = e;
  });
  int64_t n_tiles;
  int64_t tile0 = block_scan<THREADS>(tiles, &n_tiles, sums);
  if (n_units <= min(w.grid, THREADS)) {
    const int fair = (int)((n_tiles + w.grid - 1) / w.grid);       // tiles of a CTA where units are split
    if (!__syncthreads_or(u1 > u0 && only.tiles > fair + kWholeTiles)) {
      if (tid == 0) {
        w.splits[cta].parts = 0;
        if (cta >= n_units) mine.t0 = mine.t1 = 0;
      }
      if (u1 > u0 && u0 == cta) {
        start = only;
        start.tile0 = tile0;
        mine.unit = u0;
        mine.t0 = tile0;
        mine.t1 = tile0 + only.tiles;
      }
      return;
    }
  }
  // cost: position v of the list, of length V, is tile (v - body) / kTileCost of
  // the unit whose tiles begin at body, or its first; CTA c begins at floor(c V / grid)
  const int64_t V = n_tiles * kTileCost + (int64_t)n_units * w.unit_cost;
  const int grid = (int)(n_tiles < w.grid ? n_tiles : w.grid);
  const bool idle = cta >= grid, ends = cta + 1 >= grid;     // nothing to do; the last range
  if (tid == 0) {
    if (idle) mine.t0 = mine.t1 = 0;
    else if (ends) mine.t1 = n_tiles;
    if (ends) w.splits[cta].parts = 0;
  }
  if (idle) return;
  const int64_t va = cta * V / grid, vb = (cta + 1) * V / grid;
  int64_t v0 = tile0 * kTileCost + (int64_t)u0 * w.unit_cost;
  walk([&](int u, ChunkUnit e) {
    e.tile0 = tile0;
    const int64_t body = v0 + w.unit_cost, end = body + (int64_t)e.tiles * kTileCost;
    auto tile_at = [&](int64_t v) { return v < body ? 0 : (v - body) / kTileCost; };
    if (v0 > va && v0 < vb) w.units[u] = e;
    if (va >= v0 && va < end) {
      start = e;
      mine.unit = u;
      mine.t0 = tile0 + tile_at(va);
    }
    if (!ends && vb >= v0 && vb < end) {
      mine.t1 = tile0 + tile_at(vb);
      // Does the unit end in a later CTA, and begin in this one?  Its parts lie
      // in CTAs cta .. ceil(end grid / V) - 1: in slot 0 of a CTA whose range
      // starts with the unit, in slot 1 where another one is in front.
      ChunkSplit sp{};
      if (tile_at(vb) > 0 && tile_at(va) == 0) {
        sp.row0 = e.row0;
        sp.cols = e.cols;
        sp.parts = (int)min((end * grid + V - 1) / V, (int64_t)grid) - cta;
        sp.slot0 = 2 * cta + (va < v0 ? 1 : 0);
        sp.next = 2 * (cta + 1);
      }
      w.splits[cta] = sp;
    }
    tile0 += e.tiles;
    v0 = end;
  });
}

}  // namespace dsa
