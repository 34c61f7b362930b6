// Angles of rotary positions with one or several axes, for the kernels that turn
// the rotated dims (kvc_store.cu, kvc_rotate.cu).
//
// Pair i (dims 2 i, 2 i + 1) of a row is turned by the angle whose cosine and sine
// are entries i and 32 + i of row positions[axis(i)] of the table:
//   y0 = x0 cos - x1 sin,  y1 = x1 cos + x0 sin,
// each operation rounded once in fp32, as the compressor does.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kvc_operators.h"

namespace kvc {

__device__ __forceinline__ int pair_axis(const Rotation& r, int pair) {
  return static_cast<int>(r.axes >> (2 * pair)) & 3;
}

// (cos, sin) of a pair at a position that lies in the table.
__device__ __forceinline__ float2 pair_angle(const Rotation& r, int64_t position, int pair) {
  const float* const entry = r.table + position * kRopeDim + pair;
  return make_float2(entry[0], entry[kPairs]);
}

// The angles of pairs first .. first + kCount - 1 (first a multiple of kCount) of a
// row; false if a position lies outside the table.
template <int kCount>
__device__ __forceinline__ bool load_angles(const Rotation& r, int64_t row, int first, float (&cos)[kCount], float (&sin)[kCount]) {
  static_assert(kCount == 2 || kCount == 4, "pairs in 16 bytes of a row");
  using Run = std::conditional_t<kCount == 4, float4, float2>;
  const int64_t* const at = r.positions + row * r.row_stride;
  const uint32_t axes = static_cast<uint32_t>(r.axes >> (2 * first)) & ((1u << (2 * kCount)) - 1);
  bool ok = true;
  if (axes == (axes & 3u) * (((1u << (2 * kCount)) - 1) / 3)) {  // one axis: its number in every place
    const int64_t position = at[(axes & 3u) * r.axis_stride];
    ok = static_cast<uint64_t>(position) < static_cast<uint64_t>(r.num_positions);
    const float* const entry = r.table + (ok ? position : 0) * kRopeDim + first;
    *reinterpret_cast<Run*>(cos) = *reinterpret_cast<const Run*>(entry);
    *reinterpret_cast<Run*>(sin) = *reinterpret_cast<const Run*>(entry + kPairs);
  } else {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const int64_t position = at[(axes >> (2 * i) & 3u) * r.axis_stride];
      const bool in = static_cast<uint64_t>(position) < static_cast<uint64_t>(r.num_positions);
      const float2 angle = pair_angle(r, in ? position : 0, first + i);
      cos[i] = angle.x;
      sin[i] = angle.y;
      ok = ok && in;
    }
  }
  return ok;
}

__device__ __forceinline__ float2 turn_pair(float2 x, float cos, float sin) {
  return make_float2(__fsub_rn(__fmul_rn(x.x, cos), __fmul_rn(x.y, sin)),
                     __fadd_rn(__fmul_rn(x.y, cos), __fmul_rn(x.x, sin)));
}

}  // namespace kvc
