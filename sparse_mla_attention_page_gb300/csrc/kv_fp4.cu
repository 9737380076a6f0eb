// The writer of 4-bit rows (fp4_rows.cuh): new BF16 latent rows, and their RoPE
// dims, quantised and scattered into the paged pool.
//
// For each group of 128 dims s = amax / 384 (FP32, IEEE), y = x / s; for each
// block of 16 dims e is the smallest of 0 .. 11 with max |y| <= 7 2^(e - 5),
// and code = E2M1(y 2^(5 - e)).  7 and not 6: a value between 6 and 7 is off by
// at most 1 as the code 6 of the smaller exponent and by as much under the
// larger one, which would cost the block's other dims a bit.
//
// 1024 (1152) bytes read and 288 (416) written a row: 131072 rows with RoPE dims
// take 49 us, 4.2 TB/s, against 31 at the copy rate.  Neither the issue slots (62 % busy,
// some 270 instructions a warp and row) nor DRAM is full: a warp loads two rows,
// quantises and stores them, and only then loads the next two, and 32 warps an SM do
// not cover all of the wait.  Dividing each value by
// itself and comparing it with every border took 1.5 times as long.  A warp per row, lane l
// dims [8 l, 8 l + 8) and 256 + the same, so that each load instruction reads 512
// contiguous bytes and each store writes 128 or more.  Two lanes hold a block,
// sixteen a group.
#include "dsa_common.cuh"
#include "fp4_rows.cuh"
#include "kernels.h"

namespace dsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// v / s, rounded as IEEE division does: a quotient within an ulp, then its
// remainder, which an FMA gives exactly, times the rounded reciprocal of s
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990; two steps, as the first product may be off by more).  Exact
// where remainders do not underflow: s at least 2^-80 (a smaller quotient than
// 2^-7 has code 0 however it is rounded), its reciprocal a normal number.  Five
// packed operations for two quotients; dividing each took a third of the kernel.
// The scale itself is such a quotient by a constant.
__device__ __forceinline__ void divide8(float* v, float s) {
  const float r1 = __frcp_rn(s);
  const uint64_t r = pack2(r1, r1), n = pack2(-s, -s);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const uint64_t x = pack2(v[k], v[k + 1]);
    uint64_t q = fma2(x, r, 0ull);
    q = fma2(fma2(n, q, x), r, q);
    q = fma2(fma2(n, q, x), r, q);
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v[k]), "=f"(v[k + 1]) : "l"(q));
  }
}

// Eight dims of this lane (one of a block's two and a group's sixteen): their
// word, the block's exponent nibble and the group's scale.
__device__ __forceinline__ void quantise8(const uint4& x, uint32_t& word, uint32_t& e, float& s) {
  // the group's largest magnitude, as 16-bit integers: a NaN is the largest
  const uint32_t p[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = __vmaxu2(__vmaxu2(p[0] & 0x7FFF7FFFu, p[1] & 0x7FFF7FFFu), __vmaxu2(p[2] & 0x7FFF7FFFu, p[3] & 0x7FFF7FFFu));
  top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const bool odd = top >= 0x7F80u;
  const float amax = bf16_bits_to_f32(top);
  float v[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(p[k] << 16);
    v[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
  }
  if (__all_sync(0xffffffffu, amax >= 0x1p-71f && amax <= 0x1p100f)) {
    constexpr float kR = 1.f / kFp4Top;
    s = amax * kR;
    s = fmaf(fmaf(-kFp4Top, s, amax), kR, s);
    s = fmaf(fmaf(-kFp4Top, s, amax), kR, s);
    divide8(v, s);
  } else {
    s = odd ? __int_as_float(0x7FC00000) : __fdiv_rn(amax, kFp4Top);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = odd || s == 0.f ? 0.f : __fdiv_rn(v[k], s);
  }
  float y = 0.f;                       // the block's largest quotient
#pragma unroll
  for (int k = 0; k < 8; ++k) y = fmaxf(y, fabsf(v[k]));
  y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
  // y <= 1.75 2^(e - 3): its exponent, one more where its mantissa is above 1.75
  e = (uint32_t)min(max((int)((__float_as_uint(y) + 0x1FFFFFu) >> 23) - 124, 0), 11);
  const float up = __uint_as_float((127u + 5u - e) << 23);               // 2^(5 - e)
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= up;
  word = fp4_codes(v) | fp4_signs(x);
}

template <bool kRope>
__global__ void __launch_bounds__(kThreads, 4) kv_write_fp4_kernel(const __grid_constant__ Fp4WriteArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");        // as the other writers
  constexpr int kRow = kRope ? kFp4RopeRow : kFp4Row;
  const int lane = threadIdx.x & 31;
  const int64_t n_warps = ((int64_t)gridDim.x * kThreads) >> 5;
  auto put = [&](int64_t slot, const uint4 (&x)[2], uint32_t rope) {
    if (slot < 0) return;
    if (slot >= a.pool_rows) {
      if (lane == 0) set_err(a.err, DSA_DEV_ERR_SLOT_RANGE);
      return;
    }
    uint32_t w[2], e[2];
    float s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) quantise8(x[h], w[h], e[h], s[h]);
    uint8_t* row = a.pool + slot * kRow;
    reinterpret_cast<uint32_t*>(row)[lane] = w[0];
    reinterpret_cast<uint32_t*>(row + 128)[lane] = w[1];
    if (kRope) reinterpret_cast<uint32_t*>(row + kFp4Row)[lane] = rope;
    // nibble l / 2 of each half, from both lanes of a block
    const int at = (lane >> 1 & 7) * 4;
    uint4 n;
    n.x = __reduce_or_sync(0xffffffffu, lane < 16 ? e[0] << at : 0u);
    n.y = __reduce_or_sync(0xffffffffu, lane < 16 ? 0u : e[0] << at);
    n.z = __reduce_or_sync(0xffffffffu, lane < 16 ? e[1] << at : 0u);
    n.w = __reduce_or_sync(0xffffffffu, lane < 16 ? 0u : e[1] << at);
    const float s1 = __shfl_sync(0xffffffffu, s[0], 16), s3 = __shfl_sync(0xffffffffu, s[1], 16);
    if (lane == 0) {
      *reinterpret_cast<float4*>(row + kFp4Scales) = make_float4(s[0], s1, s[1], s3);
      *reinterpret_cast<uint4*>(row + kFp4Exps) = n;
    }
  };
  auto rope_of = [&](int64_t i) {
    return kRope ? __ldcs(reinterpret_cast<const uint32_t*>(a.k_pe + i * a.k_pe_stride) + lane) : 0u;
  };
  auto load = [&](int64_t i, uint4 (&x)[2]) {
    const uint4* p = reinterpret_cast<const uint4*>(a.kv_c + i * a.kv_stride) + lane;
    x[0] = __ldcs(p);
    x[1] = __ldcs(p + 32);
  };
  // two rows per warp and pass, all loads issued before any is used
  for (int64_t i0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; i0 < a.n_rows; i0 += 2 * n_warps) {
    const int64_t i1 = i0 + n_warps;
    const bool two = i1 < a.n_rows;
    const int64_t s0 = __ldg(a.slots + i0), s1 = two ? __ldg(a.slots + i1) : -1;
    uint4 r0[2], r1[2];
    load(i0, r0);
    if (two) load(i1, r1);
    const uint32_t p0 = rope_of(i0), p1 = two ? rope_of(i1) : 0u;
    put(s0, r0, p0);
    if (two) put(s1, r1, p1);
  }
}

}  // namespace

void launch_kv_write_fp4(const Fp4WriteArgs& a, int sms, cudaStream_t stream) {
  // sixteen rows a block and pass, at most one wave of four blocks per SM
  const int64_t blocks = (a.n_rows + 15) / 16, cap = (int64_t)sms * 4;
  const unsigned grid = (unsigned)(blocks < cap ? blocks : cap);
  if (a.k_pe != nullptr) kv_write_fp4_kernel<true><<<grid, kThreads, 0, stream>>>(a);
  else kv_write_fp4_kernel<false><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace dsa
