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

}  // namespace

bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.grid, kFewBlocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel, w) == cudaSuccess;
}

}  // namespace dsa
