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

// One slice of one row of a unit of many parts, by the whole block.
__device__ __forceinline__ void merge_many(const ChunkWork& w, const ChunkSplit& sp, int col, int slice) {
  __shared__ float wt[kMaxCtas];
  __shared__ float red[kMergeThreads / 32], red2[kMergeThreads / 32];
  __shared__ float4 acc_s[kLanes][kSlice4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto slot = [&](int p) { return (int64_t)(p == 0 ? sp.slot0 : sp.next + 2 * (p - 1)) * w.nc + col; };
  const int pl = tid / kDimThreads, dt = tid % kDimThreads;
  float4 v[kBatch][kVec];
  auto load = [&](int p0) {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int p = p0 + q * kLanes;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[q][i] = p < sp.parts ? __ldcg(reinterpret_cast<const float4*>(w.part_o + slot(p) * kD) + slice * kSlice4 + dt + i * kDimThreads)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  load(pl);
  float m = -INFINITY;
  bool nan = false;
  for (int p = tid; p < sp.parts; p += kMergeThreads) {
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
  for (int p = tid; p < sp.parts; p += kMergeThreads) {
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
  for (int p0 = pl; p0 < sp.parts; p0 += kLanes * kBatch) {
    if (p0 != pl) load(p0);
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int p = p0 + q * kLanes;
      if (p >= sp.parts) break;
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
    store_row(w.a, sp.row0 + col, slice * kSlice4 + tid, o, sum == 0.f ? 0.f : 1.f / sum);
    if (tid == 0 && slice == 0) w.a.lse[sp.row0 + col] = sum == 0.f ? -INFINITY : m + logf(sum);
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
      for (; item < kSlices * u.cols; item += blocks) merge_many(w, u, item / kSlices, item % kSlices);
      item -= kSlices * u.cols;
    }
}

// ---- rows that share a prefix

// Where the parts of a unit's rows over the prefix lie: those of its first rows,
// and from column brk on those of the next unit of the prefix.
struct Join {
  int64_t row0;
  int cols, own_slot, own_parts;       // parts 0: one part, in row_o
  int brk, col0, slot[2], parts[2];    // column of its first row there
  int kind;                            // 0: nothing to do, 1: up to kFewParts parts, 2: more
};

__device__ __forceinline__ Join join_of(const ChunkWork& w, int u) {
  union {
    ChunkUnit u;
    int4 v[4];
  } x;
  auto fetch = [&](int i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x.v[k] = __ldcg(reinterpret_cast<const int4*>(w.units + i) + k);
  };
  fetch(u);
  Join j{};
  if (x.u.side == kPrefix || (x.u.side == kAlone && x.u.parts == 0)) return j;
  j.row0 = x.u.row0;
  j.cols = x.u.cols;
  j.own_slot = x.u.slot0;
  j.own_parts = x.u.parts;
  j.brk = j.cols;
  int parts = max(j.own_parts, 1);
  if (x.u.side == kOwn) {
    const int mate = x.u.mate;
    j.col0 = x.u.mate_col;
    j.brk = min(j.cols, w.nc - j.col0);
    fetch(mate);
    j.slot[0] = x.u.slot0;
    j.parts[0] = max((int)x.u.parts, 0);
    int most = max(j.parts[0], 1);
    if (j.brk < j.cols) {
      fetch(mate + 1);
      j.slot[1] = x.u.slot0;
      j.parts[1] = max((int)x.u.parts, 0);
      most = max(most, j.parts[1]);
    }
    parts += most;
  } else {
    j.parts[0] = -1;                   // no prefix
  }
  j.kind = parts <= kFewParts ? 1 : 2;
  return j;
}

// The parts of one row: its own keys' first, then the prefix's.
struct RowParts {
  const ChunkWork& w;
  int64_t row, own_at, pre_at;         // rows of part_o (or of row_o, where there is one part)
  int own, pre;                        // parts
  bool own_whole, pre_whole;
  int own_next, pre_next, col, pre_col;
  __device__ __forceinline__ RowParts(const ChunkWork& work, const Join& j, int c) : w(work), row(j.row0 + c), col(c) {
    own_whole = j.own_parts == 0;
    own = own_whole ? 1 : j.own_parts;
    own_at = own_whole ? w.rows + row : (int64_t)j.own_slot * w.nc + c;
    own_next = (j.own_slot / 2 + 1) * 2;
    const int second = c >= j.brk;
    const int n = second ? j.parts[1] : j.parts[0], slot = second ? j.slot[1] : j.slot[0];
    pre_col = (j.col0 + c) % w.nc;
    pre_whole = n == 0;
    pre = n < 0 ? 0 : pre_whole ? 1 : n;
    pre_at = pre_whole ? row : (int64_t)slot * w.nc + pre_col;
    pre_next = (slot / 2 + 1) * 2;
  }
  __device__ __forceinline__ int count() const { return own + pre; }
  // part p's LSE and row of 512
  __device__ __forceinline__ void at(int p, const float*& lse, const float4*& o) const {
    const bool mine = p < own;
    const int q = mine ? p : p - own;
    const bool whole = mine ? own_whole : pre_whole;
    const int64_t r = q == 0 ? (mine ? own_at : pre_at)
                             : (int64_t)((mine ? own_next : pre_next) + 2 * (q - 1)) * w.nc + (mine ? col : pre_col);
    lse = (whole ? w.row_lse : w.part_lse) + r;
    o = reinterpret_cast<const float4*>((whole ? w.row_o : w.part_o) + r * kD);
  }
};

// Parts p0, p0 + step, ... of a row, kInFlight of them at once: running maximum,
// sum and V float4 of the dims, d4 + 32 i for i < V.
template <int V, int kInFlight>
__device__ __forceinline__ void fold_parts(const RowParts& rp, int p0, int step, int d4, float& m, float& sum, float4 (&acc)[V]) {
  const int n = rp.count();
  m = -INFINITY;
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (; p0 < n; p0 += step * kInFlight) {
    float ls[kInFlight];
    float4 v[kInFlight][V];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int p = p0 + k * step;
      ls[k] = -INFINITY;
      if (p >= n) continue;
      const float* lse;
      const float4* o;
      rp.at(p, lse, o);
      ls[k] = __ldcg(lse);
#pragma unroll
      for (int i = 0; i < V; ++i) v[k][i] = __ldcg(o + d4 + 32 * i);
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) top = fmaxf(top, ls[k]);
    if (top != m && m != -INFINITY) {
      const float f = expf(m - top);
      sum *= f;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f);
    }
    m = top;
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (ls[k] == -INFINITY) continue;            // no such part, or one without a visible key
      const float e = expf(ls[k] - m);             // (NaN where it is: fmaxf passes it over)
      sum += e;
#pragma unroll
      for (int i = 0; i < V; ++i) fold(acc[i], e, v[k][i]);
    }
  }
}

constexpr int kJoinLanes = kMergeThreads / 32;     // many parts: a warp for every eighth part of a row
constexpr int kJoinAll = 1024;                     // units up to which every block looks at all of them

// Few units (and so perhaps many parts): every block knows all of them, takes
// its share of the rows of few parts, a pair at a time, and of those of many,
// one at a time.  Many units: a block takes runs of 32 for itself.
__global__ void __launch_bounds__(kMergeThreads, 4) prefix_merge_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");               // every part is written
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ Join joins[kMergeThreads];
  __shared__ float lane_m[kJoinLanes], lane_sum[kJoinLanes];
  __shared__ float4 lane_o[kJoinLanes][kD / 4];
  const int tid = threadIdx.x, n_units = __ldcg(w.n_units);
  const bool all = n_units <= kJoinAll;
  const int run = all ? kMergeThreads : 32;
  const int pairs = w.nc / kFewRows;
  for (int u0 = all ? 0 : blockIdx.x * run; u0 < n_units; u0 += all ? run : run * (int)gridDim.x) {
    const int here = min(run, n_units - u0);
    __syncthreads();                               // the entries before are done with
    if (tid < here) joins[tid] = join_of(w, u0 + tid);
    __syncthreads();
    for (int item = all ? blockIdx.x : 0; item < here * pairs; item += all ? gridDim.x : 1) {
      const Join& j = joins[item / pairs];
      const int col = item % pairs * kFewRows + tid / kFewThreads, d4 = tid % kFewThreads;
      if ((j.kind == 0 || (j.kind == 2 && all)) || col >= j.cols) continue;
      const RowParts rp(w, j, col);
      float m, sum;
      float4 acc[1];
      fold_parts<1, 4>(rp, 0, 1, d4, m, sum, acc);
      store_row(w.a, rp.row, d4, acc[0], sum == 0.f ? 0.f : 1.f / sum);
      if (d4 == 0) w.a.lse[rp.row] = sum == 0.f ? -INFINITY : m + logf(sum);
    }
    if (!all) continue;
    int item = blockIdx.x;                         // from the unit's first row on
    for (int i = 0; i < here; ++i) {
      const Join& j = joins[i];
      if (j.kind != 2) continue;
      for (; item < j.cols; item += gridDim.x) {
        const RowParts rp(w, j, item);
        const int lane = tid & 31, warp = tid >> 5;
        float m, sum;
        float4 acc[4];
        fold_parts<4, 2>(rp, warp, kJoinLanes, lane, m, sum, acc);
        if (lane == 0) {
          lane_m[warp] = m;
          lane_sum[warp] = sum;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) lane_o[warp][lane + 32 * k] = acc[k];
        __syncthreads();
        if (tid < kD / 4) {
          float top = -INFINITY, total = 0.f;
#pragma unroll
          for (int k = 0; k < kJoinLanes; ++k) top = fmaxf(top, lane_m[k]);
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kJoinLanes; ++k) {
            if (lane_sum[k] == 0.f) continue;      // none of its parts has a visible key
            const float e = expf(lane_m[k] - top);
            total = fmaf(e, lane_sum[k], total);
            fold(o, e, lane_o[k][tid]);
          }
          store_row(w.a, rp.row, tid, o, total == 0.f ? 0.f : 1.f / total);
          if (tid == 0) w.a.lse[rp.row] = total == 0.f ? -INFINITY : top + logf(total);
        }
        __syncthreads();
      }
      item -= j.cols;
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
  return launch_merge(prefix_merge_kernel, dim3(w.grid * 4), w, stream);
}

}  // namespace dsa
