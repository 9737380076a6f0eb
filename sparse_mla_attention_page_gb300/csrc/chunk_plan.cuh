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

__device__ __forceinline__ int unit_count(const ChunkArgs& a, int n, int nc) { return (int)(((int64_t)n * a.H + nc - 1) / nc); }

// Keys that the first new token of a request sees.
__device__ __forceinline__ int first_visible(const ChunkArgs& a, const Request& r) { return a.causal ? r.kv - r.n + 1 : r.kv; }

// Rows and keys that units are cut from: a request, its own keys, or a group's
// rows over their prefix.
struct Part {
  int t0, n, kv, vis0, key0, b, side;
  int64_t group_row0;      // kOwn: the group's first query row and first unit
  int group_unit;
};

// Entry of the i-th unit of a part (tile0 is filled in later).
template <bool kShared>
__device__ __forceinline__ Unit<kShared> unit_of(const ChunkArgs& a, const Part& r, int i, int nc) {
  Unit<kShared> u{};
  const int64_t rows = (int64_t)r.n * a.H, r0 = (int64_t)i * nc;
  u.row0 = (int64_t)r.t0 * a.H + r0;
  u.b = r.b;
  u.cols = (int)(rows - r0 < nc ? rows - r0 : nc);
  u.r0 = (int)r0;
  u.vis0 = r.vis0;
  u.kv = r.kv;
  if constexpr (kShared) {
    u.key0 = r.key0;
    u.side = (uint8_t)r.side;
    if (r.side == kOwn) {
      const int64_t at = u.row0 - r.group_row0;
      u.mate = r.group_unit + (int)(at / nc);
      u.mate_col = (uint8_t)(at % nc);
    }
  }
  u.last = chunk_visible(a, u, u.cols - 1);
  u.tiles = u.last <= kChunkTile ? 1 : (u.last - 1) / kChunkTile + 1;
  return u;
}

// The groups of requests, in shared memory.
struct Groups {
  const int32_t* cu;       // [G + 1]
  int32_t* keys;           // [G] shared keys (while they are found: what every row sees)
  int32_t* first;          // [G] the first request with new tokens
  int32_t* units;          // [G] units of the requests
};

// A group shares a whole number of tiles of its prefix, at most what its first
// tokens all see, and only where packing its rows takes less than each request
// reading those tiles for itself (the cost of a unit counted as the ranges do).
// However little that is: with a call in this kernel the rows are joined anyway,
// and not sharing (each request's keys in units of 32 rows) only takes longer.
// us with sharing / without, 64 single tokens of 16 heads behind 512 keys: raw
// 24.6 / 26.7, 656-byte rows 30.8 / 31.9, 416-byte rows 36.9 / 36.9; behind 2048:
// 28.8 / 32.7, 39.0 / 43.0, 47.2 / 53.7.  (At 256 keys of 416-byte rows and 8
// heads 32.8 / 30.8, the one of 36 such cases that loses more than the noise.)
// Requests with lengths out of range end the sharing of their group, offsets out
// of order that of all.
template <int THREADS>
__device__ __forceinline__ Groups find_groups(const ChunkWork& w, int32_t* scratch) {
  const ChunkArgs& a = w.a;
  const int tid = threadIdx.x, G = a.G;
  int32_t* cu = scratch;
  const Groups g{cu, cu + G + 1, cu + 2 * G + 1, cu + 3 * G + 1};
  bool bad = false;
  Request r{};
  if (tid < a.B) r = request_of(a, tid);         // (on its way beside the groups)
  for (int i = tid; i <= G; i += THREADS) {
    const int x = __ldg(a.group_cu + i);
    bad |= x < 0 || x > a.B || (i < G && (x > __ldg(a.group_cu + i + 1) || __ldg(a.prefix_lens + i) < 0));
    cu[i] = x;
    if (i == G) break;
    g.keys[i] = INT32_MAX;
    g.first[i] = INT32_MAX;
    g.units[i] = 0;
  }
  bad = __syncthreads_or(bad) != 0;
  if (bad) {
    if (blockIdx.x == 0 && tid == 0) set_err(a.err, DSA_DEV_ERR_LENGTH);
    for (int i = tid; i <= G; i += THREADS) cu[i] = 0;      // nobody belongs to a group
    __syncthreads();
  } else {
    for (int b = tid; b < cu[G]; b += THREADS) {
      if (b != tid) r = request_of(a, b);
      if (b < cu[0]) continue;
      const int i = scan_owner(cu, G, b);
      if (r.err) atomicMin(g.keys + i, 0);
      if (r.n <= 0) continue;
      atomicMin(g.keys + i, max(first_visible(a, r), 0));
      atomicMin(g.first + i, b);
      atomicAdd(g.units + i, unit_count(a, r.n, w.nc));
    }
    __syncthreads();
  }
  for (int i = tid; i < G; i += THREADS) {
    const int tiles = g.first[i] == INT32_MAX ? 0 : min(g.keys[i], __ldg(a.prefix_lens + i)) / kChunkTile;
    int keys = 0;
    if (tiles > 0) {
      const int n = __ldg(a.cu_q + cu[i + 1]) - __ldg(a.cu_q + cu[i]);
      const int64_t apart = (int64_t)g.units[i] * tiles * kTileCost;
      const int64_t packed = (int64_t)unit_count(a, n, w.nc) * (tiles * kTileCost + w.unit_cost);
      if (packed < apart) keys = tiles * kChunkTile;
    }
    g.keys[i] = keys;
  }
  __syncthreads();
  return g;
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

// Bytes of shared memory: 32-bit words of the requests, or of the requests and
// five of each group, and the scans' sums.
constexpr int plan_words(bool shared) { return shared ? 6 * DSA_MAX_PREFIX_REQUESTS + 2 : DSA_MAX_REQUESTS; }
constexpr int plan_scratch(bool shared) { return plan_words(shared) * 4 + 256; }

// By all THREADS threads; mine and start (the range's first unit) lie in
// shared memory and hold after the caller's next barrier.
template <int THREADS, bool kShared>
__device__ __forceinline__ void chunk_plan(const ChunkWork& w, uint8_t* scratch, ChunkRange& mine, Unit<kShared>& start) {
  int64_t* sums = reinterpret_cast<int64_t*>(scratch + plan_words(kShared) * 4);
  int32_t* first_unit = reinterpret_cast<int32_t*>(scratch);                             // [N]
  const ChunkArgs& a = w.a;
  const int tid = threadIdx.x, cta = blockIdx.x;
  Unit<kShared>* units = units_of<kShared>(w);
  const int N = kShared ? a.B + a.G : a.B;         // parts: the requests, then the groups' prefixes
  Groups groups{};
  if constexpr (kShared) groups = find_groups<THREADS>(w, first_unit + N);
  int err = 0;
  auto part = [&](int p) -> Part {
    Part x{};
    if (kShared && p >= a.B) {
      const int g = p - a.B;
      x.side = kPrefix;
      x.kv = x.vis0 = groups.keys[g];
      if (x.kv > 0) {
        x.b = groups.first[g];
        x.t0 = __ldg(a.cu_q + groups.cu[g]);
        x.n = __ldg(a.cu_q + groups.cu[g + 1]) - x.t0;
      }
      return x;
    }
    const Request r = request_of(a, p);
    err |= r.err;
    x.t0 = r.t0;
    x.n = r.n;
    x.b = p;
    x.kv = r.kv;
    x.vis0 = first_visible(a, r);
    if (kShared && r.n > 0 && p >= groups.cu[0] && p < groups.cu[a.G]) {
      const int g = scan_owner(groups.cu, a.G, p);
      if (groups.keys[g] > 0) {
        x.side = kOwn;
        x.key0 = groups.keys[g];
        x.kv -= x.key0;
        x.vis0 -= x.key0;
        x.group_row0 = (int64_t)__ldg(a.cu_q + groups.cu[g]) * a.H;
        x.group_unit = first_unit[a.B + g];      // (once the sums are there)
      }
    }
    return x;
  };
  const int per = (N + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, N), b1 = min(b0 + per, N);
  int64_t here = 0;
  int last_units = 0;
  for (int b = b0; b < b1; ++b) {
    last_units = unit_count(a, part(b).n, w.nc);
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
    at += b + 1 == b1 ? last_units : unit_count(a, part(b).n, w.nc);
  }
  __syncthreads();
  if (kShared && cta == 0 && tid == 0) {
    w.n_units[0] = n_units;
    w.n_units[1] = min(first_unit[a.B], n_units);
  }

  // thread -> a run of consecutive units
  const int uper = (n_units + THREADS - 1) / THREADS;
  const int u0 = (int)min((int64_t)tid * uper, (int64_t)n_units), u1 = min(u0 + uper, n_units);
  const int first_b = u0 < u1 ? scan_owner(first_unit, N, u0) : 0;
  int64_t tiles = 0;
  Unit<kShared> only{};          // of a thread that has one unit: worked out once
  auto walk = [&](auto&& visit) {
    if (u1 - u0 == 1 && tiles > 0) return visit(u0, only);
    int b = first_b;
    Part r{};
    bool have = false;
    for (int u = u0; u < u1; ++u) {
      while (b + 1 < N && first_unit[b + 1] <= u) {
        ++b;
        have = false;
      }
      if (!have) r = part(b);
      have = true;
      visit(u, unit_of<kShared>(a, r, u - first_unit[b], w.nc));
    }
  };
  walk([&](int, const Unit<kShared>& e) {
    tiles += e.tiles;
    only = e;
  });
  int64_t n_tiles;
  int64_t tile0 = block_scan<THREADS>(tiles, &n_tiles, sums);
  if (n_units <= min(w.grid, THREADS)) {
    const int fair = (int)((n_tiles + w.grid - 1) / w.grid);       // tiles of a CTA where units are split
    if (!__syncthreads_or(u1 > u0 && only.tiles > fair + kWholeTiles)) {
      if (tid == 0) {
        if (!kShared) w.splits[cta].parts = 0;
        if (cta >= n_units) mine.t0 = mine.t1 = 0;
      }
      if (u1 > u0 && u0 == cta) {
        start = only;
        start.tile0 = tile0;
        if constexpr (kShared) units[u0] = start;
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
    if (!kShared && ends) w.splits[cta].parts = 0;
  }
  if (idle) return;
  const int64_t va = cta * V / grid, vb = (cta + 1) * V / grid;
  int64_t v0 = tile0 * kTileCost + (int64_t)u0 * w.unit_cost;
  walk([&](int u, Unit<kShared> e) {
    e.tile0 = tile0;
    const int64_t body = v0 + w.unit_cost, end = body + (int64_t)e.tiles * kTileCost;
    auto tile_at = [&](int64_t v) { return v < body ? 0 : (v - body) / kTileCost; };
    // with shared prefixes: the unit's first tile lies in this range (a border may lie in front of it, in the
    // unit's own cost), so that each entry is written once, with its parts
    const bool begins = kShared && v0 < vb && va < end && tile_at(va) == 0 && (ends || vb >= end || tile_at(vb) > 0);
    if (!kShared && v0 > va && v0 < vb) units[u] = e;
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
      if constexpr (kShared) {
        e.slot0 = (int16_t)sp.slot0;
        e.parts = (int16_t)sp.parts;
      } else {
        w.splits[cta] = sp;
      }
    }
    if constexpr (kShared) {
      if (begins) units[u] = e;
    }
    tile0 += e.tiles;
    v0 = end;
  });
}

}  // namespace dsa
