// Chunks over 4-bit rows: the requests' rows are expanded once, to the 8-bit rows
// of the same values (fp4_rows.cuh), before query rows by the hundred attend to
// them.
//
// A unit of 32 query rows that expands its tiles for itself (fp4_expand_role) takes
// 1.5 times as long as one that reads 8-bit rows by TMA, and a chunk has many units
// for each of its request's rows.  So a call of many query rows (kFlatCall) first
// writes the rows, 128 to a page, to its workspace, and attends to those.
// Lengths are known on the GPU alone: where they do not fit (or a length or a page is
// out of range, which the general form answers), this kernel leaves the rows alone,
// gives the attention over 8-bit rows no requests and the one over 4-bit rows all of
// them; else the other way round.
//
// HBM-bound: 416 bytes read and 656 written a row (288 and 528), a few us against
// the hundreds of such a call.  A warp per row, lane l dims [16 l, 16 l + 16): 512
// contiguous bytes a store.
#include <climits>

#include "chunk_plan.cuh"
#include "dsa_common.cuh"
#include "fp4_rows.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;         // rows of a warp loaded before any is used

template <bool kRope>
__global__ void __launch_bounds__(kThreads) fp4_flat_kernel(const __grid_constant__ FlatWork f) {
  constexpr int kFrom = kRope ? kFp4RopeRow : kFp4Row, kTo = kRope ? kRopeRow : kScaledRow;
  __shared__ int32_t base[kFlatRequests], len[kFlatRequests];
  __shared__ int64_t sums[kThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const ChunkArgs& a = f.a;
  const int tid = threadIdx.x, gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  // first tile and rows of each request
  constexpr int kPer = kFlatRequests / kThreads;
  int64_t tiles = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    if (b >= a.B) break;
    const Request r = request_of(a, b);
    bad |= r.err != 0;
    len[b] = r.n > 0 ? r.kv : 0;
    tiles += (len[b] + kChunkTile - 1) / kChunkTile;
  }
  int64_t total;
  int64_t at = block_scan<kThreads>(tiles, &total, sums);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = tid * kPer + i;
    if (b >= a.B) break;
    base[b] = (int32_t)min(at, (int64_t)INT32_MAX);
    at += (len[b] + kChunkTile - 1) / kChunkTile;
  }
  bad = __syncthreads_or(bad || total > f.tiles) != 0;
  // every page that a key lies in
  if (!bad)
    for (int b = 0; b < a.B; ++b) {
      const int pages = (int)(((int64_t)len[b] + a.page_size - 1) / a.page_size);
      for (int p = tid; p < pages; p += kThreads) {
        const int32_t entry = __ldg(a.page_table + (int64_t)b * a.max_pages + p);
        const int last = min(len[b] - p * a.page_size, a.page_size);
        bad |= entry < 0 || (int64_t)entry * a.page_size + last > a.pool_rows;
      }
    }
  bad = __syncthreads_or(bad) != 0;
  for (int b = gtid; b <= a.B; b += gsize) {
    const int32_t cu = __ldg(a.cu_q + b);
    f.cu8[b] = bad ? 0 : cu;
    f.cu4[b] = bad ? cu : 0;
    if (b == a.B) break;
    const int32_t kv = __ldg(a.kv_lens + b);
    f.kv8[b] = bad ? 0 : kv;
    f.kv4[b] = bad ? kv : 0;
  }
  if (bad) return;
  for (int g = gtid; g < (int)total; g += gsize) {
    const int b = scan_owner(base, a.B, g);
    f.table[(int64_t)b * f.width + (g - base[b])] = g;
  }
  const int lane = tid & 31;
  for (int r0 = (gtid >> 5) * kInFlight; r0 < (int)total * kChunkTile; r0 += (gsize >> 5) * kInFlight) {
    const int b = scan_owner(base, a.B, r0 / kChunkTile);      // (a tile's rows are one request's)
    const int j0 = r0 - base[b] * kChunkTile;
    uint2 c[kInFlight];
    uint32_t e[kInFlight];
    uint4 tail[kInFlight];
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int j = min(j0 + k, len[b] - 1), page = j / a.page_size;
      const uint8_t* row = a.pool + ((int64_t)__ldg(a.page_table + (int64_t)b * a.max_pages + page) * a.page_size + (j - page * a.page_size)) * kFrom;
      c[k] = __ldg(reinterpret_cast<const uint2*>(row) + lane);
      e[k] = __ldg(row + kFp4Exps + (lane >> 1)) >> (lane & 1) * 4 & 15;
      // lanes 0 to 7 the RoPE dims, lane 8 the scales
      if (lane < 9 && (kRope || lane == 8)) tail[k] = __ldg(reinterpret_cast<const uint4*>(row + (lane == 8 ? kFp4Scales : kFp4Row + 16 * lane)));
    }
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      if (j0 + k >= len[b]) break;
      uint8_t* row = f.rows + (int64_t)(r0 + k) * kTo;
      const Fp4Lut lut(e[k]);
      uint4 x;
      fp4_expand8(c[k].x, lut, x.x, x.y);
      fp4_expand8(c[k].y, lut, x.z, x.w);
      reinterpret_cast<uint4*>(row)[lane] = x;
      if (lane < 9 && (kRope || lane == 8)) *reinterpret_cast<uint4*>(row + (lane == 8 ? kD : kScaledRow + 16 * lane)) = tail[k];
    }
  }
}

}  // namespace

bool launch_fp4_flat(const FlatWork& f, int sms, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms * 4);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const bool rope = f.a.layout == DSA_KV_FP4_416;
  return cudaLaunchKernelEx(&cfg, rope ? fp4_flat_kernel<true> : fp4_flat_kernel<false>, f) == cudaSuccess;
}

}  // namespace dsa
