// Rotary positions of several axes, joined with the query concatenation and
// the 656-byte row writer: one launch between the projections and the
// attention.
//
//   pair (a, b) of dims (2 i, 2 i + 1) or (i, i + 32):
//     angle = positions[axis[i]][t] * inv_freq[i]
//     (a, b) -> mscale (a cos - b sin, b cos + a sin), rounded to BF16 once
//
// The angle's whole turns have no effect, so it is kept as a fraction of a
// turn: inv_freq / 2 pi as a 64-bit fixed-point fraction times the integer
// position, wrapping modulo 2^64, is the exact fraction for a position of any
// size (an FP32 product is off by a radian's thousandth at position 10^4
// already); its top 32 bits give cos and sin of a float in [-1, 1) half turns.
//
// HBM-bound: per token H x 1152 bytes read and written, one 1152-byte row read
// and 656 bytes written.  One warp takes `heads_per_item` heads of a token, so
// cos and sin (lane l: one pair, or two neighbouring ones) are formed once for
// them, or a token's row.  Items are heads-major within a token.  4096 tokens
// of 32 heads take 51.5 us, 6.0 TB/s (55 us with a grid of the resident blocks
// that strides over the items: theirs start and end together), 64 tokens of 16
// heads 3.1 us, launch and one trip to memory.
#include <cuda_bf16.h>

#include "dense.h"
#include "dsa_common.cuh"
#include "row_codec.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kPe = kRopeDims;          // 64 turned dims
constexpr int kQOut = kD + kRopeDims;   // 576

// cos and sin (times mscale) of the pairs whose elements lane l holds as the
// 4-byte word l of the 64 dims: interleaved, word l is pair l; else word l
// holds elements 2 l and 2 l + 1, which belong to pairs (2 l) % 32 and the next.
struct Turn {
  float c[2], s[2];
};

__device__ __forceinline__ Turn turn_of(const RopeArgs& a, int t, int lane) {
  Turn r;
  if (a.interleaved) {
    const int64_t p = __ldg(a.positions + a.axis[lane] * a.pos_stride + t);
    const uint64_t f = (uint64_t)p * a.turn[lane];
    sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &r.s[0], &r.c[0]);
    r.c[0] *= a.mscale;
    r.s[0] *= a.mscale;
    r.c[1] = r.c[0];
    r.s[1] = r.s[0];
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = (2 * lane + k) & 31;
      const int64_t p = __ldg(a.positions + a.axis[i] * a.pos_stride + t);
      const uint64_t f = (uint64_t)p * a.turn[i];
      sincospif((float)(int32_t)(f >> 32) * 4.656612873077393e-10f, &r.s[k], &r.c[k]);
      r.c[k] *= a.mscale;
      r.s[k] *= a.mscale;
    }
  }
  return r;
}

// Word l (two BF16) of the turned 64 dims.
__device__ __forceinline__ uint32_t turned(uint32_t w, const Turn& r, int interleaved, int lane) {
  const float x0 = bf16_bits_to_f32(w & 0xFFFFu), x1 = bf16_bits_to_f32(w >> 16);
  float y0, y1;
  if (interleaved) {
    y0 = x0 * r.c[0] - x1 * r.s[0];
    y1 = x1 * r.c[0] + x0 * r.s[0];
  } else {
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 16);   // the pairs' other halves
    const float z0 = bf16_bits_to_f32(o & 0xFFFFu), z1 = bf16_bits_to_f32(o >> 16);
    const float sg = lane < 16 ? -1.f : 1.f;                  // a cos - b sin below dim 32, b cos + a sin above
    y0 = x0 * r.c[0] + sg * (z0 * r.s[0]);
    y1 = x1 * r.c[1] + sg * (z1 * r.s[1]);
  }
  const __nv_bfloat162 y = __floats2bfloat162_rn(y0, y1);
  return *reinterpret_cast<const uint32_t*>(&y);
}

__global__ void __launch_bounds__(kThreads) rope_qkv656_kernel(const __grid_constant__ RopeArgs a, int heads_per_item,
                                                               int items_per_token) {
  // as the KV writers: the attention behind it, a programmatic dependent, may
  // set itself up meanwhile
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t n_warps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int64_t q_items = a.q_pe ? (int64_t)a.T * items_per_token : 0;
  const int64_t n_items = q_items + (a.kv_c ? a.T : 0);
  for (int64_t it = warp0; it < n_items; it += n_warps) {
    if (it < q_items) {
      const int t = (int)(it / items_per_token);
      const int h0 = (int)(it - (int64_t)t * items_per_token) * heads_per_item;
      const int h1 = min(h0 + heads_per_item, a.H);
      const Turn r = turn_of(a, t, lane);
#pragma unroll 1
      for (int h = h0; h < h1; ++h) {
        const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(a.q_pe + t * a.qp_t + h * a.qp_h) + lane);
        uint16_t* out = a.q_out + ((int64_t)t * a.H + h) * kQOut;
        if (a.q_nope) {
          const uint4* src = reinterpret_cast<const uint4*>(a.q_nope + t * a.qn_t + h * a.qn_h);
          const uint4 v0 = __ldcs(src + lane), v1 = __ldcs(src + 32 + lane);
          reinterpret_cast<uint4*>(out)[lane] = v0;
          reinterpret_cast<uint4*>(out)[32 + lane] = v1;
        }
        reinterpret_cast<uint32_t*>(out + kD)[lane] = turned(w, r, a.interleaved, lane);
      }
    } else {
      const int t = (int)(it - q_items);
      const int64_t slot = __ldg(a.slots + t);
      Row16 row;
      load_row16(a.kv_c + t * a.kv_stride, lane, row);
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(a.k_pe + t * a.kp_stride) + lane);
      const Turn r = turn_of(a, t, lane);
      const uint32_t pe = turned(w, r, a.interleaved, lane);
      if (slot < 0) continue;
      if (slot >= a.pool_rows) {
        if (lane == 0) set_err(a.err, DSA_DEV_ERR_SLOT_RANGE);
        continue;
      }
      float s0, s1;
      quantise_groups(row, s0, s1);
      uint8_t* dst = a.pool + slot * kRopeRow;
      store_row16(dst, lane, row);
      reinterpret_cast<uint32_t*>(dst + kScaledRow)[lane] = pe;
      store_scales(dst, lane, s0, s1);
    }
  }
}

}  // namespace

void launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  // Heads of an item: as many, up to eight, as leave a quarter of the resident
  // warps an item each.  us for 1024 tokens of 16 heads and for 4096 of 32: one
  // head 12.4 / 78, two 9.2 / 57, four 7.5 / 53, eight 7.5 / 52, sixteen 7.4 /
  // 56; for 256 tokens of 16 heads one 5.0, two 3.9.
  const int64_t warps = (int64_t)sms * 8 * (kThreads / 32);
  int hpi = 1;
  while (hpi < 8 && (int64_t)a.T * a.H / hpi >= warps / 4) hpi *= 2;
  const int ipt = (a.H + hpi - 1) / hpi;
  const int64_t items = (a.q_pe ? (int64_t)a.T * ipt : 0) + (a.kv_c ? a.T : 0);
  const int64_t blocks = (items + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t cap = 1 << 30;       // (of a grid; larger calls stride)
  rope_qkv656_kernel<<<(unsigned)(blocks < cap ? blocks : cap), kThreads, 0, stream>>>(a, hpi, ipt);
}

}  // namespace dsa
