// Row conversions shared by the KV writers and the rotary writer: one warp
// holds a 512-dim latent row, lane l dims [8l, 8l+8) and [256+8l, 256+8l+8).
#pragma once
#include "dsa_common.cuh"

namespace dsa {

struct Row16 {
  float v[16];  // v[0..7]: dims 8l..8l+7, v[8..15]: dims 256+8l..256+8l+7
};

__device__ __forceinline__ void load_row16(const uint16_t* __restrict__ row, int lane, Row16& r) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4*>(row) + lane);
  const uint4 b = __ldcs(reinterpret_cast<const uint4*>(row + 256) + lane);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    r.v[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}

// Four floats -> four E4M3 bytes (saturating round-to-nearest-even); a NaN
// input gives the FN NaN code 0x7F with the input's sign bit (the cvt
// instruction alone returns 0x7F for NaN of either sign).
__device__ __forceinline__ uint32_t e4m3x4_keep_nan_sign(float a, float b, float c, float d) {
  uint32_t r = e4m3x4_satrne(a, b, c, d);
  const float v[4] = {a, b, c, d};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (v[i] != v[i]) r = (r & ~(0xFFu << (8 * i))) | ((0x7Fu | ((__float_as_uint(v[i]) >> 31) << 7)) << (8 * i));
  return r;
}

__device__ __forceinline__ void store_row16(uint8_t* __restrict__ row, int lane, const Row16& r) {
  uint2 lo, hi;
  lo.x = e4m3x4_keep_nan_sign(r.v[0], r.v[1], r.v[2], r.v[3]);
  lo.y = e4m3x4_keep_nan_sign(r.v[4], r.v[5], r.v[6], r.v[7]);
  hi.x = e4m3x4_keep_nan_sign(r.v[8], r.v[9], r.v[10], r.v[11]);
  hi.y = e4m3x4_keep_nan_sign(r.v[12], r.v[13], r.v[14], r.v[15]);
  reinterpret_cast<uint2*>(row)[lane] = lo;
  reinterpret_cast<uint2*>(row + 256)[lane] = hi;
}

// Scales of the four 128-dim groups (amax / 448, 0 for a zero group) and the
// row divided by them.  A group is held by 16 lanes: groups 0 and 2 by lanes
// 0-15 (first and second half of their registers), groups 1 and 3 by lanes
// 16-31; s0 and s1 are the scales of the lane's own halves.
__device__ __forceinline__ void quantise_groups(Row16& r, float& s0, float& s1) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a0 = fmaxf(a0, fabsf(r.v[k]));
    a1 = fmaxf(a1, fabsf(r.v[8 + k]));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
    a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
  }
  s0 = a0 == 0.f ? 0.f : __fdiv_rn(a0, 448.0f);
  s1 = a1 == 0.f ? 0.f : __fdiv_rn(a1, 448.0f);
  // copysignf: the same quotient (s > 0), and a NaN keeps its input's sign
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    r.v[k] = s0 == 0.f ? 0.f : copysignf(__fdiv_rn(r.v[k], s0), r.v[k]);
    r.v[8 + k] = s1 == 0.f ? 0.f : copysignf(__fdiv_rn(r.v[8 + k], s1), r.v[8 + k]);
  }
}

// The four scales into bytes [512, 528) of a row.
__device__ __forceinline__ void store_scales(uint8_t* row, int lane, float s0, float s1) {
  const float g1 = __shfl_sync(0xffffffffu, s0, 16);
  const float g3 = __shfl_sync(0xffffffffu, s1, 16);
  if (lane == 0) *reinterpret_cast<float4*>(row + 512) = make_float4(s0, g1, s1, g3);
}

}  // namespace dsa
