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

#include "kvc_operators.h"

namespace kvc {

// Of pairs first .. first + kCount - 1 (first a multiple of kCount).
template <int kCount>
struct Angles {
  float cos[kCount], sin[kCount];

  // False if a position lies outside the table; the angles are then 0.
  __device__ __forceinline__ bool load(const Rotation& r, int64_t row, int first) {
    const int64_t* const at = r.positions + row * r.row_stride;
    const uint32_t axes = static_cast<uint32_t>(r.axes >> (2 * first)) & ((1u << (2 * kCount)) - 1);
    bool ok = true;
    // one axis for all of them: its number in every place
    if (axes == (axes & 3u) * (((1u << (2 * kCount)) - 1) / 3)) {
      int64_t pos = at[(axes & 3u) * r.axis_stride];
      ok = static_cast<uint64_t>(pos) < static_cast<uint64_t>(r.num_positions);
      const float* const entry = r.table + (ok ? pos : 0) * kRopeDim + first;
      load_run(entry, cos);
      load_run(entry + kPairs, sin);
    } else {
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const int64_t pos = at[(axes >> (2 * i) & 3u) * r.axis_stride];
        const bool in = static_cast<uint64_t>(pos) < static_cast<uint64_t>(r.num_positions);
        const float* const entry = r.table + (in ? pos : 0) * kRopeDim + first + i;
        cos[i] = entry[0];
        sin[i] = entry[kPairs];
        ok = ok && in;
      }
    }
    return ok;
  }

  __device__ __forceinline__ void invert() {
#pragma unroll
    for (int i = 0; i < kCount; ++i) sin[i] = -sin[i];
  }

  __device__ __forceinline__ void turn(float* x) const {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(a, cos[i]), __fmul_rn(b, sin[i]));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(b, cos[i]), __fmul_rn(a, sin[i]));
    }
  }

 private:
  __device__ __forceinline__ static void load_run(const float* src, float* dst) {
    if constexpr (kCount == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      dst[0] = v.x, dst[1] = v.y, dst[2] = v.z, dst[3] = v.w;
    } else {
      static_assert(kCount == 2, "pairs in 16 bytes of a row");
      const float2 v = *reinterpret_cast<const float2*>(src);
      dst[0] = v.x, dst[1] = v.y;
    }
  }
};

}  // namespace kvc
