// Exact decode of packed codes with bf16 arithmetic, for the kernels that read slots.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace kvc {

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// 8 codes of a 4-bit slot times its scale as four words of bf16, exactly.  A code
// lies 8 above itself in its 4 bits, u; as the low bits of 128's bf16 it is
// 128 + u, and one fused multiply-add by s less 136 s leaves (u - 8) s: s has 4
// significant bits, 136 s = 17 x 8 s no more than 8, the result 7.
__device__ __forceinline__ uint4 decode8_bf16(uint32_t word, uint32_t s, uint32_t less) {
  uint4 v;
  v.x = fma_bf16x2((word & 0x000F000Fu) | 0x43004300u, s, less);
  v.y = fma_bf16x2((word >> 4 & 0x000F000Fu) | 0x43004300u, s, less);
  v.z = fma_bf16x2((word >> 8 & 0x000F000Fu) | 0x43004300u, s, less);
  v.w = fma_bf16x2((word >> 12 & 0x000F000Fu) | 0x43004300u, s, less);
  return v;
}

}  // namespace kvc
