// Packed codes to bf16 pairs, shared by the kernels of the grouped product.
//
// A b-bit code q (b <= 7) placed in the top mantissa bits of bf16 1.0 is
// 1 + q 2^-b exactly, so codes become registers of two adjacent
// codes with a shift and one three-input logic operation a pair: of a word v
// that starts at an even code, v >> b holds the odd codes where v holds the even
// ones, and one byte permutation puts the low halves of both side by side. The
// pairs of a half then differ by a shift alone.
//
// From it the middle of the width's codes is taken, v = (q - mid(b)) 2^-b with
// mid(b) = (2^b - 1) / 2, by one bf16x2 addition that is exact for b <= 6 (v is a
// multiple of 2^-(b+1) below 1/2). 1.5 - 2^-8 is no bf16 value, so 7-bit codes
// are centred at 64. 8-bit codes do not fit the mantissa; they become
// q - 127.5, exact in bf16.
// The centre is not for the codes' sake but for the sums': 1 + q 2^-b would put
// about 1.5 sum x into every group's sum, and min-max quantized weights have
// their zeros near mid(b), so with v both terms below are of the size of the
// result's own, for inputs x of one sign or with a mean as well. (Rounded to bf16,
// uncentred codes put 6 percent of the values of many rows on the wrong side for x
// of mean 1, against 0.1 percent. Centred at 2^(b-1), the zeros' terms have one
// sign, and their sum's roundings left fp32 results off by 5e-6 to 1.7e-5 of the
// norm; at mid(b) 1.1e-6 to 1.8e-6, and 3e-7 to 4e-7 for x without a mean.)
//
// What a group of width b, scale s and zero z then adds, with D = sum x v and
// xs = sum x:  s (sum x q - z xs) = coef_d(b, s) D + coef_x(b, s, z) xs.
#pragma once
#include <cstdint>
#include "common.cuh"

namespace slim {

// kCodes codes (8, 16 or 32) of B bits from the start of w into kCodes / 2 registers.
template <int B, int kCodes>
__device__ __forceinline__ void decode_codes(const uint32_t (&w)[(B * kCodes + 31) / 32], uint32_t (&out)[kCodes / 2]) {
  constexpr int kAll = kCodes / 2, kWords = (B * kCodes + 31) / 32;
  if constexpr (B == 8) {
#pragma unroll
    for (int p = 0; p < kAll; ++p) {
      const uint32_t v = w[p >> 1] >> ((p & 1) * 16);
      const float lo = (float)(v & 0xFFu) - 127.5f, hi = (float)((v >> 8) & 0xFFu) - 127.5f;
      out[p] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);  // at most 8 bits: exact in bf16
    }
  } else {
    constexpr int kPairs = 1 + (16 - B) / (2 * B);  // pairs whose fields fit one 16-bit half
    constexpr uint32_t kField = ((1u << B) - 1) << (7 - B);
    constexpr uint32_t kMid = 0xBFC0u - (B < 7 ? 1u << (6 - B) : 0u);  // -(1.5 - 2^-(B+1)), B = 7: -1.5
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
          asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(kMid * 0x10001u));
          out[p0 + i] = r;
        }
    }
  }
}

__device__ __forceinline__ float coef_d(int b, float s) {
  return b >= 8 ? s : s * __int_as_float((127 + b) << 23);
}
__device__ __forceinline__ float coef_x(int b, float s, float z) {
  const float mid = b == 7 ? 64.f : 0.5f * __int_as_float((127 + b) << 23) - 0.5f;
  return -s * (z - mid);
}

}  // namespace slim
