// The work list of the dense attention of new tokens, and the merge of the
// units that the persistent grid spread over CTAs.
//
// Plan: one block.  Two prefix sums (units of each request, tiles of each
// unit), then every unit's entry is written, and with it the unit that each
// CTA's range starts in and the list of split units.  A few hundred to a few
// thousand units: bound by its launch and three dependent passes, which the
// attention kernel's set-up overlaps (programmatic dependent launch).
//
// Merge: a split unit's parts are normalised (O_c, LSE_c) of its query rows
// over disjoint keys: LSE = log sum_c exp(LSE_c), O = sum_c exp(LSE_c - LSE) O_c.
// One block at a time per (split unit, query row): first the weights of all
// parts (one part per thread), then eight part lanes of 32 threads with 16
// dims each, so that a long context's 150 parts cost a few rounds of loads.
#include <cuda_bf16.h>

#include "chunk.cuh"
#include "dsa_common.cuh"
#include "scan.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = kScanThreads;
constexpr int kMergeThreads = 256;
constexpr int kPartLanes = 8;
constexpr int kDimThreads = kMergeThreads / kPartLanes;   // 32 threads x 4 float4 = 512 dims
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
  u.vis0 = a.causal ? (int)max((int64_t)INT32_MIN / 2, (int64_t)r.kv - r.n + 1) : r.kv;
  u.kv = r.kv;
  const int vis = chunk_visible(a, u, u.cols - 1);
  u.tiles = vis <= kChunkTile ? 1 : (vis + kChunkTile - 1) / kChunkTile;
  u.pad[0] = u.pad[1] = 0;
  return u;
}

__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(const __grid_constant__ ChunkWork w) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int32_t first_unit[];    // [B]
  __shared__ int n_splits;
  const ChunkArgs& a = w.a;
  const int tid = threadIdx.x;
  if (tid == 0) n_splits = 0;
  int err = 0;
  const int per = (a.B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) {
    const Request r = request_of(a, b);
    err |= r.err;
    mine += units_of(a, r, w.nc);
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
    at += units_of(a, request_of(a, b), w.nc);
  }
  __syncthreads();

  // thread -> a run of consecutive units
  const int uper = (n_units + kPlanThreads - 1) / kPlanThreads;
  const int u0 = (int)min((int64_t)tid * uper, (int64_t)n_units), u1 = min(u0 + uper, n_units);
  const int first_b = u0 < u1 ? scan_owner(first_unit, a.B, u0) : 0;
  int64_t tiles = 0;
  auto walk = [&](auto&& visit) {
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
  walk([&](int, const ChunkUnit& e) { tiles += e.tiles; });
  int64_t n_tiles;
  int64_t tile0 = block_scan(tiles, &n_tiles);
  const int grid = (int)(n_tiles < w.grid ? n_tiles : w.grid);
  walk([&](int u, ChunkUnit e) {
    e.tile0 = tile0;
    w.units[u] = e;
    // CTAs whose range starts in this unit: tile_begin(c) >= x for c >= ceil(x grid / n)
    const int64_t end = tile0 + e.tiles;
    const int c_lo = (int)((tile0 * grid + n_tiles - 1) / n_tiles);
    const int c_hi = (int)((end * grid + n_tiles - 1) / n_tiles);
    for (int c = c_lo; c < c_hi && c < grid; ++c) w.cta_unit[c] = u;
    const int c_in = chunk_tile_begin(c_lo, n_tiles, grid) > tile0 ? c_lo : c_lo + 1;   // first that starts inside
    if (c_in < c_hi && c_in < grid) {
      const int c0 = c_in - 1, c1 = (c_hi < grid ? c_hi : grid) - 1;
      w.splits[atomicAdd(&n_splits, 1)] =
          ChunkSplit{u, c0, c1, 2 * c0 + (chunk_tile_begin(c0, n_tiles, grid) < tile0 ? 1 : 0)};
    }
    tile0 = end;
  });
  __syncthreads();
  if (tid == 0) *w.hdr = ChunkHeader{n_tiles, n_units, n_splits};
}

__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkWork w) {
  __shared__ float wt[kMaxParts];
  __shared__ float red[kMergeThreads / 32], red2[kMergeThreads / 32];
  __shared__ float4 acc_s[kPartLanes][kD / 4];
  asm volatile("griddepcontrol.wait;" ::: "memory");               // every part is written
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_items = __ldcg(&w.hdr->n_splits) * w.nc;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int4 s4 = __ldcg(reinterpret_cast<const int4*>(w.splits) + item / w.nc);
    const int c0 = s4.y, n_parts = s4.z - s4.y + 1, slot0 = s4.w;
    const int col = item % w.nc;
    const ChunkUnit& u = w.units[s4.x];
    if (col >= __ldcg(&u.cols)) continue;
    const int64_t row = __ldcg(&u.row0) + col;
    auto slot = [&](int p) { return (int64_t)(p == 0 ? slot0 : 2 * (c0 + p)) * w.nc + col; };
    // weights exp(LSE_c - max) and their sum
    float m = -INFINITY;
    bool nan = false;
    for (int p = tid; p < n_parts; p += kMergeThreads) {
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
    for (int p = tid; p < n_parts; p += kMergeThreads) {
      const float e = nan ? wt[p] : m == -INFINITY ? 0.f : expf(wt[p] - m);
      wt[p] = nan ? __int_as_float(0x7FC00000) : e;
      sum += wt[p];
    }
    sum = warp_sum(sum);
    if (lane == 0) red2[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeThreads / 32; ++i) sum += red2[i];
    const int pl = tid / kDimThreads, dt = tid % kDimThreads;
    float4 acc[4] = {};
    for (int p = pl; p < n_parts; p += kPartLanes) {
      const float e = wt[p];
      if (e == 0.f) continue;                                      // a part without a visible key
      const float4* src = reinterpret_cast<const float4*>(w.part_o + slot(p) * kD) + dt;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = __ldcg(src + i * kDimThreads);
        acc[i].x = fmaf(e, v.x, acc[i].x);
        acc[i].y = fmaf(e, v.y, acc[i].y);
        acc[i].z = fmaf(e, v.z, acc[i].z);
        acc[i].w = fmaf(e, v.w, acc[i].w);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) acc_s[pl][dt + i * kDimThreads] = acc[i];
    __syncthreads();
    if (tid < kD / 4) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kPartLanes; ++i) {
        const float4 v = acc_s[i][tid];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      uint2 packed;
      packed.x = *reinterpret_cast<const uint32_t*>(&lo);
      packed.y = *reinterpret_cast<const uint32_t*>(&hi);
      reinterpret_cast<uint2*>(w.a.o + row * kD)[tid] = packed;
      if (tid == 0) w.a.lse[row] = sum == 0.f ? -INFINITY : m + logf(sum);
    }
    __syncthreads();   // acc_s, wt and the sums are free for the next row
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
  cfg.gridDim = dim3(w.grid * 8);
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
