// Exact decode of packed slot values, shared by the reader (kvc_reader.cu)
// and the attention over slots (kvc_attend.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace kvc {
namespace {

// A stored value is q * 2^e for an int8 code q (any of its 256 byte values)
// and e = b - 127 for a scale byte b (any of its 256 values).  The product
// has at most 8 significant bits, so it is exact in fp32 -- and in bf16 --
// unless |q| 2^e reaches 2^128, where correct rounding gives +-inf; zero
// codes give +0.  It is formed from exact pieces with no conversion
// instruction and no library scaling call:
//   q       = float(2^23 + (q + 128)) - (2^23 + 128): the byte (q + 128) is
//             placed in the mantissa of 2^23 (integer bit operations), and
//             the subtraction of two integers below 2^24 is exact;
//   2^(e-1) = the fp32 with those bits: exponent field b - 1 for b >= 2,
//             the subnormals 2^-127 (b = 1) and 2^-128 (b = 0);
//   q 2^e   = (q * 2^(e-1)) * 2: both products are exact or overflow, and
//             b = 255 (e = 128, whose 2^e is not an fp32 value) needs no
//             special case: a zero code stays +0, any other overflows.
// The fp32 result's low 16 bits are zero (at most 8 significant bits, and
// subnormal results keep their bits at or above 2^-128), so its bf16 form
// is exactly its high half.

// 2^(e - 1) for the scale byte b = e + 127.
__device__ __forceinline__ float half_scale(uint32_t b) {
  return __uint_as_float(b >= 2u ? (b - 1u) << 23 : 0x00200000u << b);
}

// The four codes of `word` (little-endian int8) times 2^e, hs = half_scale.
__device__ __forceinline__ void decode4(uint32_t word, float hs, float v[4]) {
  const uint32_t x = word ^ 0x80808080u;  // q + 128 in every byte
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes (q + 128, 0, 0, 0x4B): 2^23 + q + 128
    const float q = __uint_as_float(__byte_perm(x, 0x4B00u, 0x5440u | i)) - 8388736.0f;
    v[i] = (q * hs) * 2.0f;
  }
}

// Two decoded values (each exactly a bf16) as one word of bf16 bits.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632u);
}

}  // namespace
}  // namespace kvc
