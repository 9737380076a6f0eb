// The reader of requests' rows: rows [start_b, start_b + n_b) of each request,
// through its page table, dequantised to BF16 in token order, for attention
// without absorbed projections, for moving a cache, for checks.
//
//   out[cu_b + i][d] = bf16(fp32(value of the code of dim d) * s_g),
// then the 64 RoPE dims as stored, where the layout has them.
//
// HBM-bound: R bytes read and 1024 (1152) written a row: 113000 rows of 416 bytes
// take 33.6 us, 5.3 TB/s of mixed reads and writes, 79 % of the copy rate.  (With six
// blocks an SM in place of four the registers spilled: 39 us.)  A warp takes a run of
// up to 32 rows: each lane finds one row's request (a search in the offsets,
// which lie in shared memory) and page, then four rows at a time are
// loaded before any is used, lane l converting dims [8 l, 8 l + 8) and 256 + the
// same, so that every load and store instruction covers contiguous bytes.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "fp4_rows.cuh"
#include "kernels.h"
#include "scan.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;
constexpr int kNearCu = 2048;        // offsets kept in shared memory; more are searched where they are
constexpr int kBlocks = 4;           // resident on an SM: more of them spill, and are slower

template <int kLayout>
struct Format {
  static constexpr bool kFp4 = kLayout == DSA_KV_FP4_288 || kLayout == DSA_KV_FP4_416;
  static constexpr bool kRope = kLayout == DSA_KV_ROPE656 || kLayout == DSA_KV_FP4_416;
  static constexpr bool kScaled = kLayout != DSA_KV_RAW512;
  static constexpr int64_t R = kLayout == DSA_KV_RAW512 ? kRawRow : kLayout == DSA_KV_SCALED528 ? kScaledRow
                               : kLayout == DSA_KV_ROPE656 ? kRopeRow : kLayout == DSA_KV_FP4_288 ? kFp4Row : kFp4RopeRow;
  static constexpr int kCodes = kFp4 ? kFp4Scales : kD;        // bytes of codes; the scales follow
  static constexpr int kRopeAt = kFp4 ? kFp4Row : kScaledRow;
};

// What a lane holds of a row.
template <int kLayout>
struct Piece {
  using F = Format<kLayout>;
  uint2 c[2];          // codes of its dims of each half (4-bit rows: one word)
  float s[2];
  uint32_t e[2];       // exponent nibbles
  uint32_t rope;
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (F::kFp4) {
        c[h].x = __ldg(reinterpret_cast<const uint32_t*>(row + 128 * h) + lane);
        e[h] = __ldg(row + kFp4Exps + 8 * h + (lane >> 2)) >> (lane & 2) * 2 & 15;
      } else {
        c[h] = __ldg(reinterpret_cast<const uint2*>(row + 256 * h) + lane);
      }
      s[h] = F::kScaled ? __ldg(reinterpret_cast<const float*>(row + F::kCodes) + 2 * h + (lane >> 4)) : 1.f;
    }
    if (F::kRope) rope = __ldg(reinterpret_cast<const uint32_t*>(row + F::kRopeAt) + lane);
  }
  __device__ __forceinline__ void store(uint16_t* out, int lane) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[2] = {c[h].x, c[h].y};
      if (F::kFp4) fp4_expand8(c[h].x, Fp4Lut(e[h]), w[0], w[1]);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float f[4];
        e4m3x4_to_f32(w[i], f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j] * s[h], f[2 * j + 1] * s[h]);
          o[2 * i + j] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      __stcs(reinterpret_cast<uint4*>(out + 256 * h) + lane, make_uint4(o[0], o[1], o[2], o[3]));
    }
    if (F::kRope) __stcs(reinterpret_cast<uint32_t*>(out + kD) + lane, rope);
  }
};

template <int kLayout>
__global__ void __launch_bounds__(kThreads, kBlocks) kv_read_kernel(const __grid_constant__ KvReadArgs a, int span) {
  using F = Format<kLayout>;
  __shared__ int32_t near[kNearCu];
  asm volatile("griddepcontrol.wait;" ::: "memory");      // (launched behind the writers, whose rows are read)
  const int32_t* cu = a.cu_rows;
  bool bad = false;
  for (int b = threadIdx.x; b <= a.B; b += kThreads) {
    const int32_t x = __ldg(a.cu_rows + b);
    if (b < kNearCu) near[b] = x;
    if (blockIdx.x == 0) bad |= x < 0 || x > a.out_rows || (b < a.B && x > __ldg(a.cu_rows + b + 1));
  }
  if (a.B < kNearCu) cu = near;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t n_warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int64_t end = min((int64_t)cu[a.B], a.out_rows);
  bool bad_page = false;
  for (int64_t r0 = (((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5) * span; r0 < end; r0 += n_warps * span) {
    // lane -> row r0 + lane: its pool row, or -1
    int32_t src = -1;
    const int64_t r = r0 + lane;
    if (lane < span && r < end && r >= cu[0]) {
      const int b = scan_owner(cu, a.B, (int)r);
      const int64_t start = a.starts != nullptr ? __ldg(a.starts + b) : 0;
      const int64_t j = start + (r - cu[b]);
      if (r < cu[b] || r >= cu[b + 1] || start < 0 || j >= (int64_t)a.max_pages * a.page_size) {
        bad = true;
      } else {
        const int page = (int)j / a.page_size;
        const int32_t entry = __ldg(a.page_table + (int64_t)b * a.max_pages + page);
        const int64_t row = (int64_t)entry * a.page_size + ((int)j - page * a.page_size);
        if (entry < 0 || row >= a.pool_rows) bad_page = true;
        else src = (int32_t)row;
      }
    }
#pragma unroll 1
    for (int k0 = 0; k0 < span; k0 += kInFlight) {
      int32_t rows[kInFlight];
      Piece<kLayout> p[kInFlight];
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        rows[k] = __shfl_sync(0xffffffffu, src, k0 + k);
        if (rows[k] >= 0) p[k].load(a.pool + rows[k] * F::R, lane);
      }
#pragma unroll
      for (int k = 0; k < kInFlight; ++k)
        if (rows[k] >= 0) p[k].store(a.out + (r0 + k0 + k) * a.out_stride, lane);
    }
  }
  if (bad) set_err(a.err, DSA_DEV_ERR_LENGTH);
  if (bad_page) set_err(a.err, DSA_DEV_ERR_PAGE_RANGE);
}

}  // namespace

bool launch_kv_read(const KvReadArgs& a, int sms, cudaStream_t stream) {
  // as few rows a warp as keep every warp busy, 4 to 32
  const int64_t warps = (int64_t)sms * kBlocks * (kThreads / 32);
  int64_t span = (a.out_rows + warps - 1) / warps;
  span = (span + kInFlight - 1) / kInFlight * kInFlight;
  span = span > 32 ? 32 : span;
  const int64_t blocks = (a.out_rows + span * (kThreads / 32) - 1) / (span * (kThreads / 32)), cap = (int64_t)sms * kBlocks;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks < cap ? blocks : cap));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto kernel = a.layout == DSA_KV_RAW512      ? kv_read_kernel<DSA_KV_RAW512>
                : a.layout == DSA_KV_SCALED528 ? kv_read_kernel<DSA_KV_SCALED528>
                : a.layout == DSA_KV_ROPE656   ? kv_read_kernel<DSA_KV_ROPE656>
                : a.layout == DSA_KV_FP4_288   ? kv_read_kernel<DSA_KV_FP4_288>
                                               : kv_read_kernel<DSA_KV_FP4_416>;
  return cudaLaunchKernelEx(&cfg, kernel, a, (int)span) == cudaSuccess;
}

}  // namespace dsa
