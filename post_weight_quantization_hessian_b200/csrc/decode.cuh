// Packed codes to bf16 pairs, shared by the kernels of the grouped product.
//
// A b-bit code q (b <= 7) placed in the top mantissa bits of bf16 1.0 is
// 1 + q 2^-b exactly, so codes become registers of two adjacent
// codes with a shift and one three-input logic operation a pair: of a word v
// that starts at an even code, v >> b holds the odd codes where v holds the even
// ones, and one byte permutation puts the low halves of both side by side. The
// pairs of a half then differ by a shift alone.
//
// From it the group's own zero is taken, as 1 + z 2^-b rounded to bf16: C, a
// multiple of 2^-7 in [1, 2). v = 1 + q 2^-b - C is then exact in bf16 (a multiple
// of 2^-7, at most 1), so it costs one bf16x2 addition and rounds nothing.
// 8-bit codes do not fit the mantissa; they become q - rint(z), exact in bf16.
//
// What a group of width b, scale s and zero z then adds, with D = sum x v and
// xs = sum x:  s (sum x q - z xs) = s 2^b D + s 2^b (C - 1 - z 2^-b) xs.
// The first term is the group's share but for 2^-8 of its range, the second what is
// left of the zero, so neither is larger than the result's own whatever the mean
// of x, and a group of equal weights w (codes 0, scale 1, zero -w) adds w xs alone.
// (With one centre for all codes of a width, the terms of such groups are
// hundreds of times the result: padded outputs of zero weights came out at up to
// 2e-3 of the others' rms, and fp32 results for x of mean 1 were off by 1e-6 to
// 1e-5 of their norm.)
#pragma once
#include <cstdint>
#include "common.cuh"

namespace slim {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What is added to the codes of a group: -C twice, or (8 bits) the float -rint(z).
// (A zero outside the codes' range is met at its end.)
__device__ __forceinline__ uint32_t code_shift(int b, float z) {
  if (b >= 8) return __float_as_uint(-rintf(fminf(fmaxf(z, 0.f), 255.f)));
  const float C = 1.f + fminf(fmaxf(z * __int_as_float((127 - b) << 23), 0.f), 1.f - 0.0078125f);
  return pack_bf16(-C, -C);
}
__device__ __forceinline__ float coef_d(int b, float s) {
  return b >= 8 ? s : s * __int_as_float((127 + b) << 23);
}
__device__ __forceinline__ float coef_x(int b, float s, float z, uint32_t shift) {
  if (b >= 8) return s * (-__uint_as_float(shift) - z);
  return coef_d(b, s) * ((-__uint_as_float(shift << 16) - 1.f) - z * __int_as_float((127 - b) << 23));
}

// kCodes codes (8, 16 or 32) of B bits from the start of w into kCodes / 2 registers.
template <int B, int kCodes>
__device__ __forceinline__ void decode_codes(const uint32_t (&w)[(B * kCodes + 31) / 32], uint32_t shift,
                                             uint32_t (&out)[kCodes / 2]) {
  constexpr int kAll = kCodes / 2, kWords = (B * kCodes + 31) / 32;
  if constexpr (B == 8) {
#pragma unroll
    for (int p = 0; p < kAll; ++p) {
      const uint32_t v = w[p >> 1] >> ((p & 1) * 16);
      const float c = __uint_as_float(shift), lo = (float)(v & 0xFFu) + c, hi = (float)((v >> 8) & 0xFFu) + c;
      out[p] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);  // |q - rint(z)| <= 255: exact in bf16
    }
  } else {
    constexpr int kPairs = 1 + (16 - B) / (2 * B);  // pairs whose fields fit one 16-bit half
    constexpr uint32_t kField = ((1u << B) - 1) << (7 - B);
#pragma unroll
    for (int p0 = 0; p0 < kAll; p0 += kPairs) {
      const int pos = 2 * B * p0, wi = pos >> 5, off = pos & 31;
      const int need = 2 * B * (p0 + kPairs <= kAll ? kPairs : kAll - p0);
      const uint32_t v =
          off + need <= 32 ? w[wi] >> off : __funnelshift_r(w[wi], w[wi + 1 < kWords ? wi + 1 : wi], off);
      const uint32_t both = __byte_perm(v, v >> B, 0x5410);
#pragma unroll
      for (int i = 0; i < kPairs; ++i)
        if (p0 + i < kAll) {
          const int to = 7 - B - 2 * B * i;
          const uint32_t f = to >= 0 ? both << (to >= 0 ? to : 0) : both >> (to < 0 ? -to : 0);
          uint32_t r = (f & (kField * 0x10001u)) | 0x3F803F80u;
          asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(shift));
          out[p0 + i] = r;
        }
    }
  }
}

}  // namespace slim
