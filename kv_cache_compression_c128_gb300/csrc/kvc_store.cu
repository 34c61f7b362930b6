// Vectors into packed slots as they come, and 4-bit slots back into vectors.
//
// kvc_store: row n of x (bf16 or fp32, 512 dims) goes to slot slots[n]:
//   dims 0 .. 447: z = bf16(x); per group of dims a = max |z| (a NaN counts as 0),
//     8-bit slots, 64 dims: a >= 1e-4, e = ceil(log2(a / 127)), code trunc(z 2^-e);
//     4-bit slots, 32 dims: s the smallest (1 + m / 8) 2^(e - 16) with 7 s >= a,
//       code z / s to the nearest, halves away from zero;
//   dims 448 .. 511: pairs (2 i, 2 i + 1) turned by the angles of the row's
//     positions, one rounding per operation in fp32, then bf16.
// The 8-bit form is what the compressor stores for the same vector.
//
// A warp has a row: lane l dims 8 l .. + 7 and 256 + 8 l .. + 7, so that every load
// and store covers one run of the row, a scale group is 4 or 8 lanes, and lanes
// 24 .. 31 of the second half hold the rotated dims.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kvc_device.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"
#include "kvc_rotation.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 8;

// 8 values as 4 words of bf16.
__device__ __forceinline__ uint4 round8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The largest magnitude of 8 values, NaN passed over.
__device__ __forceinline__ float most8(const float (&z)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(z[i]));
  return a;
}

// The scale byte of a group whose largest magnitude is a.  Where 7 s = a holds, a / 7
// in fp32 is s; elsewhere it is 2^-9 of s or more away from every s (both are
// multiples of the same power of two), so rounding up to 4 significant bits is exact.
__device__ __forceinline__ uint32_t scale_byte(float a) {
  const uint32_t up = (__float_as_uint(__fdiv_rn(a, 7.f)) + 0xFFFFFu) >> 20;  // 8 exponent + 3 mantissa bits
  constexpr int kLeast = (127 - 16) * 8;
  return static_cast<uint32_t>(max(0, min(255, static_cast<int>(up) - kLeast)));
}

// 8 codes of the group with scale s, 8 above themselves.
__device__ __forceinline__ uint32_t codes4(const float (&z)[8], float s) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // |z| / s is exact at halves, and 2^-9 or more away from them elsewhere
    const float size = fminf(floorf(__fdiv_rn(fabsf(z[i]), s) + 0.5f), 7.f);
    const int q = z[i] == z[i] ? static_cast<int>(copysignf(size, z[i])) : 0;
    word |= static_cast<uint32_t>(q + 8) << (4 * (i >> 1) + 16 * (i & 1));
  }
  return word;
}

template <typename F, bool kF32>
__global__ void __launch_bounds__(kWarps * 32) kvc_store_kernel(const __grid_constant__ StoreParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= p.num_rows) return;
  const int64_t slot = p.slots[row];
  if (slot < 0) return;
  const int64_t page = slot / kSlotsPerPage;
  const int place = static_cast<int>(slot % kSlotsPerPage);
  float x[2][8];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t at = row * p.x_row_stride + 256 * k + 8 * lane;
    if constexpr (kF32) {
      const float4* const src = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + at);
      const float4 a = src[0], b = src[1];
      x[k][0] = a.x, x[k][1] = a.y, x[k][2] = a.z, x[k][3] = a.w;
      x[k][4] = b.x, x[k][5] = b.y, x[k][6] = b.z, x[k][7] = b.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + at);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[k][2 * i] = dev::bf16_lo(w[i]), x[k][2 * i + 1] = dev::bf16_hi(w[i]);
    }
  }
  const bool rope = lane >= 24;  // of the second half
  bool ok = page < p.num_pages;
  if (p.rotation.positions != nullptr && rope) {
    Angles<4> angles;
    ok = angles.load(p.rotation, row, 4 * (lane - 24)) && ok;
    angles.turn(x[1]);
  }
  if (!__all_sync(0xFFFFFFFFu, ok)) {
    if (lane == 0) dev::record_error(p.error, dev::kErrBadIndex);
    return;
  }
  uint8_t* const base = p.kv_cache + page * F::kPage;
  uint8_t* const payload = base + place * F::kStride;
  uint8_t* const scales = base + F::kScaleBase + place * F::kScales;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 w = round8(x[k]);
    if (k == 1 && rope) *reinterpret_cast<uint4*>(payload + F::kCodes + 16 * (lane - 24)) = w;
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    float z[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[2 * i] = dev::bf16_lo(words[i]), z[2 * i + 1] = dev::bf16_hi(words[i]);
    float a = most8(z);
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 1));
    a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 2));
    if constexpr (F::kFour) {
      const uint32_t byte = k == 1 && rope ? 0u : scale_byte(a);  // (two bytes behind the 14 scales are zero)
      if (!(k == 1 && rope))
        *reinterpret_cast<uint32_t*>(payload + 4 * (32 * k + lane)) =
            codes4(z, __uint_as_float((byte + (127 - 16) * 8) << 20));
      if ((lane & 3) == 0) scales[8 * k + lane / 4] = static_cast<uint8_t>(byte);
    } else {
      a = fmaxf(fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, 4)), 1.0e-4f);
      const int e = dev::scale_exponent(a);
      const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
      uint32_t code[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = max(-127, min(127, __float2int_rz(__fmul_rn(z[i], inv))));
        code[i >> 2] |= static_cast<uint32_t>(q & 0xFF) << (8 * (i & 3));
      }
      if (!(k == 1 && rope)) *reinterpret_cast<uint2*>(payload + 8 * (32 * k + lane)) = make_uint2(code[0], code[1]);
      if ((lane & 7) == 0) scales[4 * k + lane / 8] = static_cast<uint8_t>(k == 1 && rope ? 0 : e + 127);
    }
  }
}

// A warp has a slot: lane l dims 4 l + 128 k .. + 3, k < 4, so that every store of
// fp32 values covers one run.
template <bool kBf16>
__global__ void __launch_bounds__(kWarps * 32) kvc_dequantize4_kernel(const uint8_t* kv, int64_t num_pages,
                                                                      const int64_t* slots, int64_t num_slots, void* out,
                                                                      uint32_t* err) {
  using F = Slots4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (m >= num_slots) return;
  const int64_t slot = slots[m], page = slot / kSlotsPerPage;
  const bool there = slot >= 0 && page < num_pages;
  if (slot >= 0 && !there && lane == 0) dev::record_error(err, dev::kErrBadIndex);
  const uint8_t* const base = kv + (there ? page : 0) * F::kPage;
  const int place = there ? static_cast<int>(slot % kSlotsPerPage) : 0;
  const uint8_t* const payload = base + place * F::kStride;
  const uint8_t* const scales = base + F::kScaleBase + place * F::kScales;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (there && k == 3 && lane >= 16) {
      const uint2 w = *reinterpret_cast<const uint2*>(payload + F::kCodes + 8 * (lane - 16));
      v[0] = dev::bf16_lo(w.x), v[1] = dev::bf16_hi(w.x), v[2] = dev::bf16_lo(w.y), v[3] = dev::bf16_hi(w.y);
    } else if (there) {
      const uint32_t word = *reinterpret_cast<const uint32_t*>(payload + 4 * (16 * k + lane / 2)) >> (8 * (lane & 1));
      const float s = __uint_as_float((scales[4 * k + lane / 8] + (127u - 16u) * 8u) << 20);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = (static_cast<int>(word >> (4 * (i >> 1) + 16 * (i & 1)) & 15u) - 8) * s;
    }
    const int64_t at = m * kHeadDim + 128 * k + 4 * lane;
    if constexpr (kBf16) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

cudaLaunchConfig_t warp_per_row(int64_t rows, cudaStream_t stream, cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, bool four_bits, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = warp_per_row(p.num_rows, stream, attr);
  if (four_bits)
    return p.x_f32 ? cudaLaunchKernelEx(&cfg, kvc_store_kernel<Slots4, true>, p)
                   : cudaLaunchKernelEx(&cfg, kvc_store_kernel<Slots4, false>, p);
  return p.x_f32 ? cudaLaunchKernelEx(&cfg, kvc_store_kernel<Slots8, true>, p)
                 : cudaLaunchKernelEx(&cfg, kvc_store_kernel<Slots8, false>, p);
}

cudaError_t launch_dequantize4(const uint8_t* kv, int64_t num_pages, const int64_t* slots, int64_t num_slots, void* out,
                               int out_bf16, uint32_t* err, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = warp_per_row(num_slots, stream, attr);
  return out_bf16 ? cudaLaunchKernelEx(&cfg, kvc_dequantize4_kernel<true>, kv, num_pages, slots, num_slots, out, err)
                  : cudaLaunchKernelEx(&cfg, kvc_dequantize4_kernel<false>, kv, num_pages, slots, num_slots, out, err);
}

}  // namespace kvc
