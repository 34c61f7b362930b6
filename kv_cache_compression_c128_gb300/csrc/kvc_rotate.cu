// Rotary positions of queries and of attention's rows.
//
//   out[t, h, 2 i]     = x[t, h, 2 i] cos - x[t, h, 2 i + 1] sin
//   out[t, h, 2 i + 1] = x[t, h, 2 i + 1] cos + x[t, h, 2 i] sin
// with the cos and sin of pair i at position positions[t, axis(i)]; the inverse
// has -sin: it turns attention's rows back (a slot's rotated dims are values too),
// and is the gradient's map.  fp32 throughout, one rounding to bf16 at the end.
//
// A row of 64 is 8 lanes' (bf16) or 16 lanes' (fp32) 16 bytes.  A run of lanes keeps
// its token's angles in registers and takes up to four heads, all loads ahead of the
// first store, so that `out` may be x itself.  A block is (lanes of a row, runs of a
// token, tokens): no index is divided (it cost a tenth of the time).
//
// Bound by the bytes in and out: 16384 tokens x 64 heads, bf16 with three axes, take
// 44.3 us (273 MB, 91 % of the copy bandwidth), 8192 x 64 in fp32 41.4 (97 %: pieces of
// 256 bytes instead of 128).  Angles in shared memory, read once a block, took 46 to
// 60 us, runs of eight heads 49: a block's loads all wait for its barrier, or for room.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kvc_device.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"
#include "kvc_rotation.cuh"

namespace kvc {
namespace {

constexpr int kTurnThreads = 256;
// Rows of 64 up to which a run of lanes takes one head, and two: calls that do not
// fill the card, or hardly, are quickest with many short runs, large ones with their
// angles read once for four heads (us, one / two / four heads a run: 16384 tokens
// without heads 1.89 / 2.06 / 2.75; 3000 x 8 2.56 / 2.06 / 2.22; 4099 x 16 fp32 7.4 /
// 6.1 / 6.2; 16384 x 64 with three axes 67 / 46.4 / 44.3).
constexpr int64_t kFewRows = 152 * 64, kManyRows = 16 * kFewRows;

template <bool kF32, int kHeads>
__global__ void __launch_bounds__(kTurnThreads) kvc_rotate_kernel(const __grid_constant__ RotateParams p) {
  constexpr int kLanes = kF32 ? 16 : 8, kElems = kF32 ? 4 : 8, kSize = kF32 ? 4 : 2, kMine = kElems / 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int l = threadIdx.x;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * blockDim.z + threadIdx.z;
  const int run = blockIdx.y * blockDim.y + threadIdx.y, runs = gridDim.y * blockDim.y;
  if (token >= p.num_tokens) return;
  const uint8_t* const src = static_cast<const uint8_t*>(p.x) + (token * p.x_token_stride + run * p.x_head_stride) * kSize + 16 * l;
  const int64_t src_step = runs * p.x_head_stride * kSize;
  uint4 v[kHeads];
#pragma unroll
  for (int j = 0; j < kHeads; ++j)
    if (run + j * runs < p.num_heads) v[j] = *reinterpret_cast<const uint4*>(src + j * src_step);
  alignas(16) float cos[kMine], sin[kMine];
  const bool ok = load_angles<kMine>(p.rotation, token, l * kMine, cos, sin);
  // the row's lanes agree: no head of a token is turned in part
  const int lane = (l + kLanes * (threadIdx.y + blockDim.y * threadIdx.z)) & 31;
  const uint32_t row = (kF32 ? 0xFFFFu : 0xFFu) << (lane & ~(kLanes - 1));
  if (!__all_sync(row, ok)) {
    if (l == 0) dev::record_error(p.error, dev::kErrBadIndex);
    return;
  }
  if (p.inverse) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) sin[i] = -sin[i];
  }
  uint8_t* const dst = static_cast<uint8_t*>(p.out) + (token * p.out_token_stride + run * p.out_head_stride) * kSize + 16 * l;
  const int64_t dst_step = runs * p.out_head_stride * kSize;
#pragma unroll
  for (int j = 0; j < kHeads; ++j) {
    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if constexpr (kF32) {
        const float2 y = turn_pair(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), cos[i], sin[i]);
        w[2 * i] = __float_as_uint(y.x), w[2 * i + 1] = __float_as_uint(y.y);
      } else {
        const float2 y = turn_pair(make_float2(dev::bf16_lo(w[i]), dev::bf16_hi(w[i])), cos[i], sin[i]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    if (run + j * runs < p.num_heads) *reinterpret_cast<uint4*>(dst + j * dst_step) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <bool kF32, int kHeads>
cudaError_t launch_of(const RotateParams& p, cudaStream_t stream) {
  constexpr int kLanes = kF32 ? 16 : 8, kRuns = kTurnThreads / kLanes;
  const int runs = (p.num_heads + kHeads - 1) / kHeads, here = runs < kRuns ? runs : kRuns, tokens = kRuns / here;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.num_tokens + tokens - 1) / tokens), (runs + here - 1) / here);
  cfg.blockDim = dim3(kLanes, here, tokens);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kvc_rotate_kernel<kF32, kHeads>, p);
}

}  // namespace

cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream) {
  const int64_t rows = p.num_tokens * p.num_heads;
  if (rows <= kFewRows || p.num_heads == 1) return p.f32 ? launch_of<true, 1>(p, stream) : launch_of<false, 1>(p, stream);
  if (rows <= kManyRows) return p.f32 ? launch_of<true, 2>(p, stream) : launch_of<false, 2>(p, stream);
  return p.f32 ? launch_of<true, 4>(p, stream) : launch_of<false, 4>(p, stream);
}

}  // namespace kvc
