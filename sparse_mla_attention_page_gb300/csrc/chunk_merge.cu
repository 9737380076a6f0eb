// The merge of the units that the attention of new tokens spread over CTAs.
//
// A split unit's parts are normalised (O_c, LSE_c) of its query rows
// over disjoint keys: LSE = log sum_c exp(LSE_c), O = sum_c exp(LSE_c - LSE) O_c.
// Units of few parts (nearly all): a thread for each 8 dims of a row folds the
// parts four at a time.  Units of many parts (a long context over most SMs): a
// block for each quarter of a row's dims, first the weights of all parts (one
// a thread), then 16 part lanes of 16 threads with four parts' loads in flight,
// so that 150 parts cost three round trips and not forty.
#include <cuda_bf16.h>

#include "chunk.cuh"
#include "dsa_common.cuh"

namespace dsa {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kBatch = 4;                                 // parts whose loads are issued together
constexpr int kFewThreads = kD / 8;                       // few parts: threads of a row, 8 dims each
constexpr int kFewRows = kMergeThreads / kFewThreads;
constexpr int kVec = 2;                                   // many parts: float4 of a thread
constexpr int kDimThreads = 16;                           // threads of a quarter of a row's dims
constexpr int kLanes = kMergeThreads / kDimThreads;       // part lanes
constexpr int kQuarter = kD / 4 / 4;                      // float4 of a quarter
constexpr int kMaxParts = 1024;                           // CTAs of the attention grid (one per SM)

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

// One quarter of one row of a unit of many parts, by the whole block.
__device__ void merge_many(const ChunkWork& w, const ChunkSplit& sp, int col, int dq) {
  __shared__ float wt[kMaxParts];
  __shared__ float red[kMergeThreads / 32], red2[kMergeThreads / 32];
  __shared__ float4 acc_s[kLanes][kQuarter];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto slot = [&](int p) { return (int64_t)(p == 0 ? sp.slot0 : sp.next + 2 * (p - 1)) * w.nc + col; };
  float m = -INFINITY;
  bool nan = false;
  for (int p = tid; p < sp.parts; p += kMergeThreads) {
    const float v = __ldcg(w.part_lse + slot(p));
    wt[p] = v;
    m = fmaxf(m, v);
    nan |= v != v;
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
  const int pl = tid / kDimThreads, dt = tid % kDimThreads;
  float4 acc[kVec] = {};
  for (int p0 = pl; p0 < sp.parts; p0 += kLanes * kBatch) {
    float4 v[kBatch][kVec];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int p = p0 + q * kLanes;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[q][i] = p < sp.parts ? __ldcg(reinterpret_cast<const float4*>(w.part_o + slot(p) * kD) + dq * kQuarter + dt + i * kDimThreads)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    }
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
  if (tid < kQuarter) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < kLanes; ++i) fold(o, 1.f, acc_s[i][tid]);
    store_row(w.a, sp.row0 + col, dq * kQuarter + tid, o, sum == 0.f ? 0.f : 1.f / sum);
    if (tid == 0 && dq == 0) w.a.lse[sp.row0 + col] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
  __syncthreads();   // acc_s, wt and the sums are free for the next row
}

__global__ void __launch_bounds__(kMergeThreads, 4) chunk_merge_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.wait;" ::: "memory");               // every part is written
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // the units of many parts, a bit for each CTA that one begins in
  __shared__ uint32_t many[kMaxParts / 32];
  for (int c0 = threadIdx.x & ~31; c0 < w.grid; c0 += kMergeThreads) {
    const int c = c0 + (threadIdx.x & 31);
    const uint32_t bits = __ballot_sync(0xffffffffu, c < w.grid && __ldcg(&w.splits[c].parts) > kFewParts);
    if ((threadIdx.x & 31) == 0) many[c0 / 32] = bits;
  }
  const ChunkSplit sp = split_of(w.splits + blockIdx.x);           // blockIdx.y: four rows of the unit
  const int col = blockIdx.y * kFewRows + threadIdx.x / kFewThreads, d8 = threadIdx.x % kFewThreads;
  if (sp.parts > 0 && sp.parts <= kFewParts && col < sp.cols) {
    float m = -INFINITY, sum = 0.f;
    float4 acc[2] = {};
    for (int p0 = 0; p0 < sp.parts; p0 += kBatch) {
      float ls[kBatch];
      float4 v[kBatch][2];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int p = p0 + q;
        const int64_t at = (int64_t)(p == 0 ? sp.slot0 : sp.next + 2 * (p - 1)) * w.nc + col;
        const float4* src = reinterpret_cast<const float4*>(w.part_o + at * kD) + 2 * d8;
        ls[q] = p < sp.parts ? __ldcg(w.part_lse + at) : -INFINITY;
        v[q][0] = p < sp.parts ? __ldcg(src) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[q][1] = p < sp.parts ? __ldcg(src + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (ls[q] == -INFINITY) continue;                          // a part without a visible key
        const float mn = fmaxf(m, ls[q]);
        const float r = m == -INFINITY ? 0.f : expf(m - mn), e = expf(ls[q] - mn);
        sum = fmaf(sum, r, e);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[i] = make_float4(acc[i].x * r, acc[i].y * r, acc[i].z * r, acc[i].w * r);
          fold(acc[i], e, v[q][i]);
        }
        m = mn;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    store_row(w.a, sp.row0 + col, 2 * d8, acc[0], inv);
    store_row(w.a, sp.row0 + col, 2 * d8 + 1, acc[1], inv);
    if (d8 == 0) w.a.lse[sp.row0 + col] = sum == 0.f ? -INFINITY : m + logf(sum);
  }
  __syncthreads();
  // the quarter rows of those units, over all blocks
  const int blocks = gridDim.x * gridDim.y;
  int item = blockIdx.y * gridDim.x + blockIdx.x;                  // from the unit's first on
  for (int i = 0; i < (w.grid + 31) / 32; ++i)
    for (uint32_t bits = many[i]; bits != 0; bits &= bits - 1) {
      const ChunkSplit big = split_of(w.splits + 32 * i + __ffs(bits) - 1);
      for (; item < 4 * big.cols; item += blocks) merge_many(w, big, item / 4, item % 4);
      item -= 4 * big.cols;
    }
}

}  // namespace

bool launch_chunk_merge(const ChunkWork& w, cudaStream_t stream) {
  if (w.grid > kMaxParts) return false;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.grid, w.nc / kFewRows);
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
