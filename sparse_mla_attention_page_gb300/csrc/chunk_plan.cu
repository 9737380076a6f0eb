// The work list of the dense attention of new tokens, and the merge of the
// units that the persistent grid spread over CTAs.
//
// Plan: one block.  Two prefix sums (units of each request, tiles of each
// unit), then every unit's entry is written, and with it where each CTA's
// range starts and the list of split units.  A few hundred to a few
// thousand units: bound by its launch and three dependent passes, which the
// attention kernel's set-up overlaps (programmatic dependent launch).
//
// Merge: a split unit's parts are normalised (O_c, LSE_c) of its query rows
// over disjoint keys: LSE = log sum_c exp(LSE_c), O = sum_c exp(LSE_c - LSE) O_c.
// Units of few parts (nearly all): a thread for each 8 dims of a row folds the
// parts four at a time.  Units of many parts (a long context over most SMs): a
// block for each quarter of a row's dims, first the weights of all parts (one
// a thread), then 16 part lanes of 16 threads with four parts' loads in flight,
// so that 150 parts cost three round trips and not forty.
#include <cuda_bf16.h>

#include "chunk.cuh"
#include "dsa_common.cuh"
#include "scan.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = kScanThreads;
constexpr int kMergeThreads = 256;
constexpr int kBatch = 4;                                 // parts whose loads are issued together
constexpr int kFewThreads = kD / 8;                       // few parts: threads of a row, 8 dims each
constexpr int kFewRows = kMergeThreads / kFewThreads;
constexpr int kVec = 2;                                   // many parts: float4 of a thread
constexpr int kDimThreads = 16;                           // threads of a quarter of a row's dims
constexpr int kLanes = kMergeThreads / kDimThreads;       // part lanes
constexpr int kQuarter = kD / 4 / 4;                      // float4 of a quarter
constexpr int kMaxParts = 1024;                           // CTAs of the attention grid (one per SM)

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

__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int32_t first_unit[];    // [B]
  __shared__ int n_many, cta_unit[kMaxParts];
  const ChunkArgs& a = w.a;
  const int tid = threadIdx.x;
  if (tid == 0) n_many = 0;
  for (int c = tid; c < w.grid; c += kPlanThreads) w.few[c].parts = 0;
  int err = 0;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  int last_units = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    err |= r.err;
    last_units = units_of(a, r, w.nc);
    mine += last_units;
  }
  int64_t total;
  int64_t at = block_scan(mine, &total);
  if (total > w.max_units) {     // only when the requests' ranges overlap: the list has no room
    err = DSA_DEV_ERR_LENGTH;
    total = 0;
  }
  if (err) set_err(a.err, err);
  const int n_units = (int)total;
  for (int b = b0; b < b1; ++b) {
    first_unit[b] = (int)min(at, (int64_t)INT32_MAX);
    at += b + 1 == b1 ? last_units : units_of(a, request_of(a, b), w.nc);
  }
  __syncthreads();

  // thread -> a run of consecutive units
  const int uper = (n_units + kPlanThreads - 1) / kPlanThreads;
  const int u0 = (int)min((int64_t)tid * uper, (int64_t)n_units), u1 = min(u0 + uper, n_units);
  const int first_b = u0 < u1 ? scan_owner(first_unit, a.B, u0) : 0;
  int64_t tiles = 0;
  ChunkUnit only{};              // of a thread that has one unit (up to 1024 units): worked out once
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
  int64_t tile0 = block_scan(tiles, &n_tiles);
  // cost: position v of the list, of length V, is tile v - v0 - kUnitCost of the
  // unit that begins at v0, or its first; CTA c begins at floor(c V / grid)
  const int64_t V = n_tiles + (int64_t)n_units * kUnitCost;
  const int grid = (int)(n_tiles < w.grid ? n_tiles : w.grid);
  int64_t v0 = tile0 + (int64_t)u0 * kUnitCost;
  walk([&](int u, ChunkUnit e) {
    e.tile0 = tile0;
    w.units[u] = e;
    const int64_t body = v0 + kUnitCost, end = body + e.tiles;
    // floor(c V / grid) >= x for c >= ceil(x grid / V)
    const int c_lo = (int)((v0 * grid + V - 1) / V);
    const int c_hi = min((int)((end * grid + V - 1) / V), grid);
    for (int c = c_lo; c < c_hi; ++c) cta_unit[c] = u;
    const int c_in = (int)(((body + 1) * grid + V - 1) / V);       // the first CTA that begins inside the unit's tiles
    if (c_in < c_hi) {
      const int c0 = c_in - 1, parts = c_hi - c0;
      ChunkSplit sp;
      sp.row0 = e.row0;
      sp.cols = e.cols;
      sp.parts = parts;
      // slot 0 of a CTA holds the unit its range starts in, slot 1 its last one
      sp.slot0 = 2 * c0 + (c0 < c_lo ? 1 : 0);
      sp.next = 2 * (c0 + 1);
      sp.pad[0] = sp.pad[1] = 0;
      if (parts > kFewParts) w.many[atomicAdd(&n_many, 1)] = sp;
      else w.few[c0] = sp;
    }
    tile0 += e.tiles;
    v0 = end;
  });
  __syncthreads();
  for (int c = tid; c <= w.grid; c += kPlanThreads) {
    ChunkStart st{};
    st.t0 = n_tiles;
    if (c < grid) {
      const int u = cta_unit[c];
      st.unit = u;
      st.u = w.units[u];
      const int64_t in = (int64_t)c * V / grid - (st.u.tile0 + (int64_t)(u + 1) * kUnitCost);
      st.t0 = st.u.tile0 + (in > 0 ? in : 0);
    }
    w.starts[c] = st;
  }
  if (tid == 0) *w.n_many = n_many;
}

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
  const int n_many = __ldcg(w.n_many);
  const ChunkSplit sp = split_of(w.few + blockIdx.x);              // blockIdx.y: four rows of the unit
  const int col = blockIdx.y * kFewRows + threadIdx.x / kFewThreads, d8 = threadIdx.x % kFewThreads;
  if (sp.parts > 0 && col < sp.cols) {
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
  const int blocks = gridDim.x * gridDim.y;
  for (int item = blockIdx.y * gridDim.x + blockIdx.x; item < n_many * w.nc * 4; item += blocks) {
    const ChunkSplit big = split_of(w.many + item / 4 / w.nc);
    const int c = item / 4 % w.nc;
    if (c < big.cols) merge_many(w, big, c, item % 4);
  }
}

}  // namespace

void launch_chunk_plan(const ChunkWork& w, cudaStream_t stream) {
  const size_t smem = (size_t)w.a.B * sizeof(int32_t);
  if (smem > 40 * 1024)
    cudaFuncSetAttribute(chunk_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  chunk_plan_kernel<<<1, kPlanThreads, smem, stream>>>(w);
}

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
