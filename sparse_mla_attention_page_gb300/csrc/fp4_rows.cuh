// The 4-bit rows (DSA_KV_FP4_288, DSA_KV_FP4_416): bytes [0, 256) hold the codes
// of the 512 latent dims, [256, 272) four FP32 scales (one for each 128 dims),
// [272, 288) an exponent nibble for each block of 16 dims (low nibble first),
// [288, 416) the 64 BF16 RoPE dims.
//
//   value of dim d = E2M1(code) 2^(e - 5) s,   e in 0 .. 11
//
// E2M1 has two significant bits and E4M3 four, and 2^(e - 5) keeps every
// non-zero product a normal E4M3 number (2^-6 .. 384).  So a row expands
// without rounding to the E4M3 bytes and four scales of a 528-byte row, and
// everything that works on those rows works on these (a scale a block in any
// other type would need a product of its own for every 16 dims).
//
// A word holds 8 dims: magnitude codes in the low three bits of its nibbles in
// order, signs where one mask and one shift put them into the top bits of the
// bytes that a byte permutation makes of the codes: of dim i < 4 in bit 8 i + 7,
// of dim 4 + i in bit 8 i + 3.
#pragma once
#include "dsa_common.cuh"

namespace dsa {

constexpr int kFp4Row = 288;
constexpr int kFp4RopeRow = 416;
constexpr int kFp4Scales = 256;      // byte offsets within a row
constexpr int kFp4Exps = 272;
constexpr float kFp4Top = 384.f;     // largest value of a code and exponent: 6 2^6

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// E4M3 bytes of the eight magnitude codes times 2^(e - 5): zero stays zero, an
// exponent step adds one to the exponent fields of the others.
struct Fp4Lut {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Fp4Lut(uint32_t e) : lo(0x14100800u + e * 0x08080800u), hi(0x24201C18u + e * 0x08080808u) {}
};

// The E4M3 bytes of a word's dims 0..3 and 4..7.
__device__ __forceinline__ void fp4_expand8(uint32_t w, const Fp4Lut& t, uint32_t& a, uint32_t& b) {
  const uint32_t m = w & 0x77777777u;
  a = prmt(t.lo, t.hi, m) | (w & 0x80808080u);
  b = prmt(t.lo, t.hi, m >> 16) | ((w << 4) & 0x80808080u);
}

// The magnitude codes of eight values (times a power of two), rounded to
// nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t fp4_codes(const float* v) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return w & 0x77777777u;
}

// The sign bits of a word, from its eight dims as BF16 pairs: those of values that
// round to zero are kept.
__device__ __forceinline__ uint32_t fp4_signs(const uint4& x) {
  return (prmt(x.x, x.y, 0x7531) & 0x80808080u) | (prmt(x.z, x.w, 0x7531) >> 4 & 0x08080808u);
}

}  // namespace dsa
