// Packed codes to bf16 pairs, shared by the kernels of the grouped product.
//
// A b-bit code q (b <= 7) placed in the top mantissa bits of bf16 1.0 is
// 1 + q 2^-b exactly, so codes become registers of two adjacent
// codes with a shift and one three-input logic operation a pair: of a word v
// that starts at an even code, v >> b holds the odd codes where v holds the even
// ones, and one byte permutation puts the low halves of both side by side. The
// pairs of a half then differ by a shift alone.
//
// With kCenter the value is moved to q 2^-b - 1/2 (exact, one bf16x2 addition).
// Without it a group's sum carries about 1.5 sum x, several times the group's own
// share of the result, and its fp32 roundings with it: far below half a step of
// a bf16 result, but not of an fp32 one. So fp32 results take the addition (their
// error against 64 bits is 1e-7 to 4e-7 of their norm).
// 8-bit codes do not fit the mantissa; they become q - 128, exact in bf16.
//
// What a group of width b, scale s and zero z then adds, with D = sum x v and
// xs = sum x:  s (sum x q - z xs) = coef_d(b, s) D + coef_x(b, s, z) xs.
#pragma once
#include <cstdint>
#include "common.cuh"

namespace slim {

// kCodes codes (8, 16 or 32) of B bits from the start of w into kCodes / 2 registers.
template <int B, int kCodes, bool kCenter>
__device__ __forceinline__ void decode_codes(const uint32_t (&w)[(B * kCodes + 31) / 32], uint32_t (&out)[kCodes / 2]) {
  constexpr int kAll = kCodes / 2, kWords = (B * kCodes + 31) / 32;
  if constexpr (B == 8) {
#pragma unroll
    for (int p = 0; p < kAll; ++p) {
      const uint32_t v = w[p >> 1] >> ((p & 1) * 16);
      const float lo = (float)(v & 0xFFu) - 128.f, hi = (float)((v >> 8) & 0xFFu) - 128.f;
      out[p] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);  // |q - 128| <= 128: exact in bf16
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
          if constexpr (kCenter) asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0xBFC0BFC0u));
          out[p0 + i] = r;
        }
    }
  }
}

template <bool kCenter>
__device__ __forceinline__ float coef_d(int b, float s) {
  return b >= 8 ? s : s * __int_as_float((127 + b) << 23);
}
template <bool kCenter>
__device__ __forceinline__ float coef_x(int b, float s, float z) {
  const float p2 = __int_as_float((127 + b) << 23);
  return kCenter || b >= 8 ? -s * (z - 0.5f * p2) : -s * (z + p2);
}

}  // namespace slim
