// Join of attention parts: rows whose softmax ran over disjoint sets of keys.
//   L = log(sum_i exp(lse_i)),  out = sum_i exp(lse_i - L) out_i.
// A part that held no key has lse -inf; its row is not read into the sum, so
// its out may hold anything.  A row whose parts all held none is zeros with
// lse -inf.
//
// One warp per row of 512, 16 dims a lane; sums in fp32, one rounding at the
// store for bf16 rows.  A row's parts are read one after the other, each only
// if its lse says that it holds keys: what is in flight beside them are other
// rows.  Large calls are bound by the bytes of the parts and the result (5 parts
// of 509 x 64 fp32 rows take 58 us, 6.9 TB/s), small ones by the latency of each
// part in turn (2 parts of 8 x 64 rows 4.8 us).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kvc_internal.h"
#include "kvc_operators.h"

namespace kvc {
namespace {

constexpr int kJoinWarps = 4;

__device__ __forceinline__ void unpack(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kJoinWarps * 32) kvc_join_kernel(const __grid_constant__ JoinParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // 16-byte pieces of a row: 64 (bf16) or 128 (fp32); lane, lane + 32, ...
  constexpr int kPieces = kBf16 ? 2 : 4, kDims = kBf16 ? 8 : 4;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (row >= p.num_rows) return;
  float lse[kMaxParts], top = -INFINITY;
  for (int i = 0; i < p.num_parts; ++i) {
    lse[i] = p.lses[i][row];
    top = fmaxf(top, lse[i]);
  }
  if (top == -INFINITY) top = 0.f;
  float total = 0.f, acc[kPieces * kDims];
#pragma unroll
  for (int j = 0; j < kPieces * kDims; ++j) acc[j] = 0.f;
  for (int i = 0; i < p.num_parts; ++i) {
    if (lse[i] == -INFINITY) continue;
    const float w = expf(lse[i] - top);
    total += w;
    const uint4* src = static_cast<const uint4*>(p.outs[i]) + row * (32 * kPieces) + lane;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const uint4 v = src[32 * j];
      if constexpr (kBf16) {
        float f[8];
        unpack(v, f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[8 * j + k] += w * f[k];
      } else {
        acc[4 * j] += w * __uint_as_float(v.x);
        acc[4 * j + 1] += w * __uint_as_float(v.y);
        acc[4 * j + 2] += w * __uint_as_float(v.z);
        acc[4 * j + 3] += w * __uint_as_float(v.w);
      }
    }
  }
  const float f = total == 0.f ? 0.f : 1.f / total;
  __syncwarp();  // lse may be one of the parts' own: every lane has read the row's
  uint4* dst = static_cast<uint4*>(p.out) + row * (32 * kPieces) + lane;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    if constexpr (kBf16) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 b =
            __floats2bfloat162_rn(acc[8 * j + 2 * k] * f, acc[8 * j + 2 * k + 1] * f);
        w[k] = *reinterpret_cast<const uint32_t*>(&b);
      }
      dst[32 * j] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      dst[32 * j] = make_uint4(__float_as_uint(acc[4 * j] * f), __float_as_uint(acc[4 * j + 1] * f),
                               __float_as_uint(acc[4 * j + 2] * f),
                               __float_as_uint(acc[4 * j + 3] * f));
    }
  }
  if (lane == 0 && p.lse != nullptr) p.lse[row] = total == 0.f ? -INFINITY : top + logf(total);
}

}  // namespace

cudaError_t launch_join(const JoinParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.num_rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.bf16 ? cudaLaunchKernelEx(&cfg, kvc_join_kernel<true>, p) : cudaLaunchKernelEx(&cfg, kvc_join_kernel<false>, p);
}

}  // namespace kvc
