// Rotary positions of queries and of attention's rows.
//
//   out[t, h, 2 i]     = x[t, h, 2 i] cos - x[t, h, 2 i + 1] sin
//   out[t, h, 2 i + 1] = x[t, h, 2 i + 1] cos + x[t, h, 2 i] sin
// with the cos and sin of pair i at position positions[t, axis(i)]; the inverse
// has -sin: it turns attention's rows back (a slot's rotated dims are values too),
// and is the gradient's map.  fp32 throughout, one rounding to bf16 at the end.
//
// A row of 64 is 8 lanes' (bf16) or 16 lanes' (fp32) 16 bytes.  A run of lanes keeps
// its token's angles in registers and takes kHeads heads, all loads ahead of the
// first store, so that `out` may be x itself.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kvc_device.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"
#include "kvc_rotation.cuh"

namespace kvc {
namespace {

constexpr int kThreadsTurn = 256, kHeads = 4;

template <bool kF32>
__global__ void __launch_bounds__(kThreadsTurn) kvc_rotate_kernel(const __grid_constant__ RotateParams p, int runs) {
  constexpr int kLanes = kF32 ? 16 : 8, kElems = kF32 ? 4 : 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t run = (static_cast<int64_t>(blockIdx.x) * kThreadsTurn + threadIdx.x) / kLanes;
  const int l = threadIdx.x % kLanes;
  const int64_t token = run / runs;
  const int first = static_cast<int>(run % runs);
  if (token >= p.num_tokens) return;
  using Word = uint4;
  const uint8_t* const src = static_cast<const uint8_t*>(p.x) + 16 * l;
  uint8_t* const dst = static_cast<uint8_t*>(p.out) + 16 * l;
  constexpr int kSize = kF32 ? 4 : 2;
  Word v[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = first + j * runs;
    if (h < p.num_heads)
      v[j] = *reinterpret_cast<const Word*>(src + (token * p.x_token_stride + h * p.x_head_stride) * kSize);
  }
  Angles<kElems / 2> angles;
  const bool ok = angles.load(p.rotation, token, l * (kElems / 2));
  // the row's lanes agree: no head of a token is turned in part
  const uint32_t row = (kF32 ? 0xFFFFu : 0xFFu) << (threadIdx.x & 31 & ~(kLanes - 1));
  if (!__all_sync(row, ok)) {
    if (l == 0) dev::record_error(p.error, dev::kErrBadIndex);
    return;
  }
  if (p.inverse) angles.invert();
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    const int h = first + j * runs;
    if (h >= p.num_heads) break;
    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
    float x[kElems];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kF32)
        x[i] = __uint_as_float(w[i]);
      else
        x[2 * i] = dev::bf16_lo(w[i]), x[2 * i + 1] = dev::bf16_hi(w[i]);
    }
    angles.turn(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kF32) {
        w[i] = __float_as_uint(x[i]);
      } else {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    *reinterpret_cast<Word*>(dst + (token * p.out_token_stride + h * p.out_head_stride) * kSize) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream) {
  const int runs = (p.num_heads + kHeads - 1) / kHeads;
  const int64_t threads = p.num_tokens * runs * (p.f32 ? 16 : 8), ctas = (threads + kThreadsTurn - 1) / kThreadsTurn;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreadsTurn);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.f32 ? cudaLaunchKernelEx(&cfg, kvc_rotate_kernel<true>, p, runs)
               : cudaLaunchKernelEx(&cfg, kvc_rotate_kernel<false>, p, runs);
}

}  // namespace kvc
