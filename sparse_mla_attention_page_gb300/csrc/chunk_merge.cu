// The merge of the units that the attention of new tokens spread over CTAs.
//
// A split unit's parts are normalised (O_c, LSE_c) of its query rows
// over disjoint keys: LSE = log sum_c exp(LSE_c), O = sum_c exp(LSE_c - LSE) O_c.
// Units of few parts (nearly all): a thread for each 4 dims of a row, all
// parts' loads in flight at once.  Units of many parts (a long context over
// most SMs): a block for each eighth of a row's dims, the weights of all parts
// (one a thread) while the first parts' loads are in flight, 32 part lanes of
// 8 threads.  Both are chains of a few trips to the L2 cache, so what counts is
// that no load waits for another and that the blocks are resident at once:
// 32.3 us for one request of 131072 scaled rows (150 parts) with 256 slices in
// flight, 34.6 with 128 whose loads came after the weights; 81.8 us for 32
// requests of 4096 rows and two tokens of 128 heads with four blocks of rows a
// unit, 85 with sixteen.
#include <cstddef>
#include <cuda_bf16.h>

#include "chunk.cuh"
#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kFewThreads = kD / 4;                       // few parts: threads of a row, 4 dims each
constexpr int kFewRows = kMergeThreads / kFewThreads;
constexpr int kFewBlocks = 4;                             // blocks of a unit (all resident: four fit an SM)
constexpr int kSlices = 8;                                // many parts: blocks of a row
constexpr int kSlice4 = kD / 4 / kSlices;                 // float4 of a slice
constexpr int kVec = 2;                                   // float4 of a thread
constexpr int kDimThreads = kSlice4 / kVec;
constexpr int kLanes = kMergeThreads / kDimThreads;       // part lanes
constexpr int kBatch = 5;                                 // parts of a lane whose loads are issued together (160 at once)

__device__ __forceinline__ void fold(float4& acc, float w, const float4& v) {
  acc.x = fmaf(w, v.x, acc.x);
  acc.y = fmaf(w, v.y, acc.y);
  acc.z = fmaf(w, v.z, acc.z);
  acc.w = fmaf(w, v.w, acc.w);
}

__device__ __forceinline__ void store_row(const ChunkArgs& a, int64_t row, int d4, const float4& o, float inv) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 packed;
  packed.x = *reinterpret_cast<const uint32_t*>(&lo);
  packed.y = *reinterpret_cast<const uint32_t*>(&hi);
  reinterpret_cast<uint2*>(a.o + row * kD)[d4] = packed;
}

__device__ __forceinline__ ChunkSplit split_of(const ChunkSplit* s) {
  union {
    ChunkSplit s;
    int4 v[2];
  } x;
  x.v[0] = __ldcg(reinterpret_cast<const int4*>(s));
  x.v[1] = __ldcg(reinterpret_cast<const int4*>(s) + 1);
  return x.s;
}

// One slice of a row of many parts, part p of which lies at `slot(p)`, by the
// whole block.
template <class Slot>
__device__ __forceinline__ void merge_many(const ChunkWork& w, int parts, int64_t row, int slice, Slot&& slot) {
  __shared__ float wt[2 * kMaxCtas];
  __shared__ float red[kMergeThreads / 32], red2[kMergeThreads / 32];
  __shared__ float4 acc_s[kLanes][kSlice4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pl = tid / kDimThreads, dt = tid % kDimThreads;
  float4 v[kBatch][kVec];
  auto load = [&](int p0) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int p = p0 + q * kLanes;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[q][i] = p < parts ? __ldcg(reinterpret_cast<const float4*>(w.part_o + slot(p) * kD) + slice * kSlice4 + dt + i * kDimThreads)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(pl);
  float m = -INFINITY;
  bool nan = false;
  for (int p = tid; p < parts; p += kMergeThreads) {
    const float x = __ldcg(w.part_lse + slot(p));
    wt[p] = x;
    m = fmaxf(m, x);
    nan |= x != x;
  }
  m = warp_max(m);
  if (lane == 0) red[warp] = m;
  nan = __syncthreads_or(nan) != 0;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) m = fmaxf(m, red[i]);
  float sum = 0.f;
  for (int p = tid; p < parts; p += kMergeThreads) {
    wt[p] = nan ? __int_as_float(0x7FC00000) : m == -INFINITY ? 0.f : expf(wt[p] - m);
    sum += wt[p];
  }
  sum = warp_sum(sum);
  if (lane == 0) red2[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMergeThreads / 32; ++i) sum += red2[i];
  float4 acc[kVec] = {};
  for (int p0 = pl; p0 < parts; p0 += kLanes * kBatch) {
    if (p0 != pl) load(p0);
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int p = p0 + q * kLanes;
      if (p >= parts) break;
#pragma unroll
      for (int i = 0; i < kVec; ++i) fold(acc[i], wt[p], v[q][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) acc_s[pl][dt + i * kDimThreads] = acc[i];
  __syncthreads();
  if (tid < kSlice4) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kLanes; ++i) fold(o, 1.f, acc_s[i][tid]);
    store_row(w.a, row, slice * kSlice4 + tid, o, sum == 0.f ? 0.f : 1.f / sum);
    if (tid == 0 && slice == 0) w.a.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
  __syncthreads();   // acc_s, wt and the sums are free for the next row
}

__global__ void __launch_bounds__(kMergeThreads, 4) chunk_merge_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");               // every part is written
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // The units of many parts: a bit for each CTA that one begins in, and its
  // entry (they begin more than kFewParts CTAs apart).
  __shared__ uint32_t many[kMaxCtas / 32];
  __shared__ ChunkSplit big[kMaxCtas / kFewParts];
  for (int c0 = threadIdx.x & ~31; c0 < w.grid; c0 += kMergeThreads) {
    const int c = c0 + (threadIdx.x & 31);
    ChunkSplit s{};
    if (c < w.grid) s = split_of(w.splits + c);
    if (s.parts > kFewParts) big[c / kFewParts] = s;
    const uint32_t bits = __ballot_sync(0xffffffffu, s.parts > kFewParts);
    if ((threadIdx.x & 31) == 0) many[c0 / 32] = bits;
  }
  const ChunkSplit sp = split_of(w.splits + blockIdx.x);           // blockIdx.y: every fourth pair of rows
  const int d4 = threadIdx.x % kFewThreads;
  for (int col = blockIdx.y * kFewRows + threadIdx.x / kFewThreads; sp.parts > 0 && sp.parts <= kFewParts && col < sp.cols; col += gridDim.y * kFewRows) {
    float ls[kFewParts];
    float4 v[kFewParts];
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) {
      const int64_t at = (int64_t)(p == 0 ? sp.slot0 : sp.next + 2 * (p - 1)) * w.nc + col;
      ls[p] = p < sp.parts ? __ldcg(w.part_lse + at) : -INFINITY;
      v[p] = p < sp.parts ? __ldcg(reinterpret_cast<const float4*>(w.part_o + at * kD) + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m = ls[0], sum = 0.f;
#pragma unroll
    for (int p = 1; p < kFewParts; ++p) m = fmaxf(m, ls[p]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int p = 0; p < kFewParts; ++p) {
      if (ls[p] == -INFINITY) continue;                            // a part without a visible key
      const float e = expf(ls[p] - m);                             // (NaN where one of them is: fmaxf passes it over)
      sum += e;
      fold(acc, e, v[p]);
    }
    store_row(w.a, sp.row0 + col, d4, acc, sum == 0.f ? 0.f : 1.f / sum);
    if (d4 == 0) w.a.lse[sp.row0 + col] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
  __syncthreads();
  // the slices of those units' rows, over all blocks
  const int blocks = gridDim.x * gridDim.y;
  int item = blockIdx.y * gridDim.x + blockIdx.x;                  // from the unit's first on
  for (int i = 0; i < (w.grid + 31) / 32; ++i)
    for (uint32_t bits = many[i]; bits != 0; bits &= bits - 1) {
      const ChunkSplit& u = big[(32 * i + __ffs(bits) - 1) / kFewParts];
      for (; item < kSlices * u.cols; item += blocks) {
        const int col = item / kSlices;
        merge_many(w, u.parts, u.row0 + col, item % kSlices,
                   [&](int p) { return (int64_t)(p == 0 ? u.slot0 : u.next + 2 * (p - 1)) * w.nc + col; });
      }
      item -= kSlices * u.cols;
    }
}

// ---- rows that share a prefix

// Rows of up to kLoopParts parts are joined by a thread for each 4 dims, kFewParts
// parts at a time; with more, which only few rows have, by slices.

// A unit of a request, and where its rows' parts over the prefix lie: those of
// its first rows, and from column brk on those of the prefix's next unit.
struct Join {
  int64_t row0;
  int cols, brk, col0;                 // col0: column of the first row in the prefix's unit
  int16_t own_slot, own_parts;         // parts 0: one part, behind joined0
  int16_t slot[2], parts[2];           // -1: no prefix
  int kind;                            // 0: nothing to do, 1: up to kLoopParts parts, 2: more
};

// The words of a unit's entry that a join needs.
struct JoinUnit {
  int64_t row0;
  int cols;
  int4 last;      // key0; mate; side and mate_col; slot0 and parts
  __device__ __forceinline__ void fetch(const SharedUnit* u) {
    row0 = __ldcg(reinterpret_cast<const long long*>(&u->row0));
    cols = __ldcg(&u->cols);
    last = __ldcg(reinterpret_cast<const int4*>(&u->key0));
  }
};
static_assert(offsetof(SharedUnit, key0) == 48 && offsetof(SharedUnit, mate) == 52 && offsetof(SharedUnit, side) == 56 &&
              offsetof(SharedUnit, mate_col) == 57 && offsetof(SharedUnit, slot0) == 60 && offsetof(SharedUnit, parts) == 62,
              "entry");

// parts_of(m): the word of unit m that holds its slot0 and parts.
template <class PartsOf>
__device__ __forceinline__ Join join_of(const ChunkWork& w, const JoinUnit& u, int n_units, PartsOf&& parts_of) {
  Join j{};
  j.row0 = u.row0;
  j.cols = j.brk = u.cols;
  j.own_slot = (int16_t)u.last.w;
  j.own_parts = (int16_t)(u.last.w >> 16);
  j.parts[0] = -1;
  if ((u.last.z & 0xFF) == kAlone) {
    j.kind = j.own_parts == 0 ? 0 : j.own_parts <= kLoopParts ? 1 : 2;
    return j;
  }
  const int m0 = parts_of(u.last.y), m1 = parts_of(min(u.last.y + 1, n_units - 1));
  j.col0 = u.last.z >> 8 & 0xFF;
  j.brk = min(j.cols, w.nc - j.col0);
  j.slot[0] = (int16_t)m0;
  j.parts[0] = (int16_t)(m0 >> 16);
  j.slot[1] = (int16_t)m1;
  j.parts[1] = (int16_t)(m1 >> 16);
  const int most = max((int)j.parts[0], j.brk < j.cols ? (int)j.parts[1] : 0);
  j.kind = max((int)j.own_parts, 1) + max(most, 1) <= kLoopParts ? 1 : 2;
  return j;
}

// The parts of one row: its own keys' first, then the prefix's.
struct RowParts {
  int64_t row;
  int own, n;                          // parts over its own keys, all
  int own0, own1, pre0, pre1, step;    // where the first ones lie, and (but for the step) the others
  __device__ __forceinline__ RowParts(const ChunkWork& w, const Join& j, int c) : row(j.row0 + c), step(2 * w.nc) {
    const int64_t rows = (int64_t)w.a.T * w.a.H;
    auto others = [&](int slot, int col) { return (slot / 2 * 2) * w.nc + col; };   // the k-th part: + k step
    own = max((int)j.own_parts, 1);
    own0 = j.own_parts == 0 ? (int)(w.joined0 + rows + row) : j.own_slot * w.nc + c;
    own1 = others(j.own_slot, c);
    const bool second = c >= j.brk;
    const int parts = second ? j.parts[1] : j.parts[0], slot = second ? j.slot[1] : j.slot[0];
    const int col = second ? c - j.brk : j.col0 + c;
    n = own + (parts < 0 ? 0 : max(parts, 1));
    pre0 = parts == 0 ? (int)(w.joined0 + row) : slot * w.nc + col;
    pre1 = others(slot, col);
  }
  __device__ __forceinline__ int64_t at(int p) const {
    const bool mine = p < own;
    const int q = mine ? p : p - own;
    return q == 0 ? (mine ? own0 : pre0) : (mine ? own1 : pre1) + q * step;
  }
};

// d4: the thread's four dims.
__device__ __forceinline__ void join_few(const ChunkWork& w, const RowParts& rp, int d4) {
  float m = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int p0 = 0; p0 < rp.n; p0 += kFewParts) {
    float ls[kFewParts];
    float4 v[kFewParts];
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) {
      const bool there = p0 + k < rp.n;
      const int64_t at = there ? rp.at(p0 + k) : 0;
      ls[k] = there ? __ldcg(w.part_lse + at) : -INFINITY;
      v[k] = there ? __ldcg(reinterpret_cast<const float4*>(w.part_o + at * kD) + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) top = fmaxf(top, ls[k]);
    if (p0 > 0 && top != m) {
      const float f = expf(m - top);
      sum *= f;
      acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    }
    m = top;
#pragma unroll
    for (int k = 0; k < kFewParts; ++k) {
      if (ls[k] == -INFINITY) continue;            // no such part, or one without a visible key
      const float e = expf(ls[k] - m);             // (NaN where one of them is: fmaxf passes it over)
      sum += e;
      fold(acc, e, v[k]);
    }
  }
  store_row(w.a, rp.row, d4, acc, sum == 0.f ? 0.f : 1.f / sum);
  if (d4 == 0) w.a.lse[rp.row] = sum == 0.f ? -INFINITY : m + logf(sum);
}

constexpr int kJoinAll = 512;                      // units of requests up to which every block looks at all of them
constexpr int kJoinRun = 8;

// Up to kJoinAll units of requests, whose rows may have many parts: every block
// knows all units and takes its share of the rows of few parts (a pair at a time)
// and of the slices of those of many.  More units: a block takes runs of them.
__global__ void __launch_bounds__(kMergeThreads, 3) prefix_merge_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");               // every part is written
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Join joins[kMergeThreads];
  __shared__ int near[kMergeThreads];              // slot0 and parts of the first units
  const int tid = threadIdx.x, blocks = gridDim.x;
  const SharedUnit* units = units_of<true>(w);
  JoinUnit u{};
  if (tid < w.max_units) u.fetch(units + tid);                    // (while the counts are on their way)
  const int n_units = __ldcg(w.n_units), n = __ldcg(w.n_units + 1);
  near[tid] = u.last.w;
  const bool all = n <= kJoinAll;
  const int run = all ? kMergeThreads : kJoinRun;
  const int pairs = w.nc / kFewRows;
  for (int u0 = all ? 0 : blockIdx.x * run; u0 < n; u0 += all ? run : run * blocks) {
    const int here = min(run, n - u0);
    __syncthreads();                               // the entries before are done with
    bool many = false;
    if (tid < here) {
      if (u0 > 0) u.fetch(units + u0 + tid);
      const Join j = join_of(w, u, n_units, [&](int m) {
        return m < kMergeThreads ? near[m] : __ldcg(reinterpret_cast<const int*>(&units[m].slot0));
      });
      many = j.kind == 2;
      joins[tid] = j;
    }
    many = __syncthreads_or(many) != 0;
    // rows of few parts; units first, as units may have fewer rows than others
    for (int item = all ? blockIdx.x : 0; item < here * pairs; item += all ? blocks : 1) {
      const Join& j = joins[item % here];
      const int col = item / here * kFewRows + tid / kFewThreads;
      if (j.kind == 0 || (j.kind == 2 && all) || col >= j.cols) continue;
      join_few(w, RowParts(w, j, col), tid % kFewThreads);
    }
    if (!all || !many) continue;
    int item = blockIdx.x;                         // from the unit's first row on
    for (int i = 0; i < here; ++i) {
      const Join& j = joins[i];
      if (j.kind != 2) continue;
      for (; item < kSlices * j.cols; item += blocks) {
        const RowParts rp(w, j, item / kSlices);
        merge_many(w, rp.n, rp.row, item % kSlices, [&](int p) { return rp.at(p); });
      }
      item -= kSlices * j.cols;
    }
  }
}

template <class Kernel>
bool launch_merge(Kernel kernel, dim3 grid, const ChunkWork& w, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, w) == cudaSuccess;
}

}  // namespace

bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream) {
  return launch_merge(chunk_merge_kernel, dim3(w.grid, kFewBlocks), w, stream);
}

bool launch_prefix_merge(const ChunkWork& w, cudaStream_t stream) {
  return launch_merge(prefix_merge_kernel, dim3(w.grid * 3), w, stream);
}

}  // namespace dsa
