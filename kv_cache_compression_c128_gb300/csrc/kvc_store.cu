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
// A warp has a row: lane l dims 8 l .. + 7, 256 + 8 l .. + 7 and pair l of the rotated
// ones, so that every load and store covers one run of the row, a scale group is 4 or
// 8 lanes, and each lane asks for one angle.  Large calls are bound by the rows in and
// the slots out: 65537 fp32 rows to 8-bit slots in order take 26.7 us (96 % of the copy
// bandwidth), to 4-bit ones turned to one axis 27.5 (95 %); bf16 rows to 4 bits with
// three axes 18.9 (86 %), which is near what its instructions take to issue, to 8 bits
// as they are 19.0 (82 %); three inputs in turn, replayed.  (Two rows a warp, in a run that
// took 25.8, 26.9 and 19.1 for the first three: 29.8, 30.1, 21.7.  Codes by division,
// angles by the eight lanes of the rotated dims: 340 instructions a row, 26.7 us for the
// third.)

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kvc_codes.cuh"
#include "kvc_device.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"
#include "kvc_rotation.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ---- codes: 8 values of a lane -----------------------------------------------------

// The largest magnitudes of each lane's two runs of 8 as bits of bf16, whose order
// is that of the values, infinities and NaN above all: the first's in the low half.
__device__ __forceinline__ uint32_t most_of(const uint4& v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
}
template <int kLanes>
__device__ __forceinline__ uint32_t most_of_groups(const uint4& v, const uint4& w) {
  const uint32_t a = most_of(v), b = most_of(w);
  uint32_t m = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// Each half of the words in magnitude at most `most` (bits of bf16), NaN as 0.
__device__ __noinline__ uint4 bring_in(uint4 v, uint32_t most) {
  uint32_t* const words = &v.x;
  for (int i = 0; i < 4; ++i) {
    uint32_t out = 0;
    for (int h = 0; h < 32; h += 16) {
      const uint32_t x = words[i] >> h & 0xFFFFu, size = x & 0x7FFFu;
      out |= (size > 0x7F80u ? 0u : (x & 0x8000u) | min(size, most)) << h;
    }
    words[i] = out;
  }
  return v;
}

// 7 times the largest scale of 4-bit slots, as bf16: 105 x 2^12.
constexpr uint32_t kMost4 = 0x48D2;

// The scale byte of a 4-bit group, a <= 7 times the largest scale.  A bf16 a that is
// not 7 s lies 2^-9 of s or more from it (both are multiples of one power of two), so
// a little less than a / 7, rounded up to 4 significant bits, is the scale sought.
__device__ __forceinline__ uint32_t scale_byte(float a) {
  const uint32_t up = (__float_as_uint(__fmul_rn(a, (1.f - 0x1p-16f) / 7.f)) + 0xFFFFFu) >> 20;
  constexpr int kLeast = (127 - 16) * 8;
  return static_cast<uint32_t>(max(0, static_cast<int>(up) - kLeast));
}

// 8 codes of 4 bits, each 8 above itself.  z / s is a half or 2^-10 and more from
// one, by the same argument, so z times a little more than 1 / s, rounded to the
// nearest whole number by the sum with 2^23, has its halves rounded away from zero.
__device__ __forceinline__ uint32_t codes4(const uint4& w, uint32_t byte) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float((byte << 20) + ((127 - 16) << 23))));
  r = __fmul_rn(r, 1.f + 0x1p-16f);
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t word = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const uint32_t even = __float_as_uint(__fmaf_rn(dev::bf16_lo(words[i]), r, 8388616.f));
    const uint32_t odd = __float_as_uint(__fmaf_rn(dev::bf16_hi(words[i]), r, 8388616.f));
    word = word * 16 + __byte_perm(even, odd, 0x5410);  // below 2^23 the sum's bits are the number
  }
  return word;
}

// 8 codes of 8 bits with the scale 2^e: z 2^-e is exact, and at most 127 in size unless
// it is infinite (kInfinite: some may be).
template <bool kInfinite>
__device__ __forceinline__ uint2 codes8(const uint4& w, int e) {
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
  uint32_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int lo = __float2int_rz(__fmul_rn(dev::bf16_lo(words[i]), inv));
    int hi = __float2int_rz(__fmul_rn(dev::bf16_hi(words[i]), inv));
    if constexpr (kInfinite) {
      lo = max(-127, min(127, lo));
      hi = max(-127, min(127, hi));
    }
    two[i] = __byte_perm(lo, hi, 0x0040);
  }
  return make_uint2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[2], two[3], 0x5410));
}

// Lane l has dims 8 l .. + 7, if l < 24 256 + 8 l .. + 7, and pair l of the rotated ones.
template <typename F, bool kF32>
__global__ void __launch_bounds__(kWarps * 32) kvc_store_kernel(const __grid_constant__ StoreParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (row >= p.num_rows) return;
  const int64_t slot = p.slots[row];
  const bool turns = p.rotation.positions != nullptr;
  int64_t at = 0;
  if (turns) at = p.rotation.positions[row * p.rotation.row_stride + pair_axis(p.rotation, lane) * p.rotation.axis_stride];
  uint4 v, w = make_uint4(0, 0, 0, 0);
  float2 pair;
  if constexpr (kF32) {
    const float* const src = static_cast<const float*>(p.x) + row * p.x_row_stride;
    const float4 a = reinterpret_cast<const float4*>(src)[2 * lane], b = reinterpret_cast<const float4*>(src)[2 * lane + 1];
    v = make_uint4(round2(a.x, a.y), round2(a.z, a.w), round2(b.x, b.y), round2(b.z, b.w));
    if (lane < 24) {
      const float4 c = reinterpret_cast<const float4*>(src)[64 + 2 * lane], d = reinterpret_cast<const float4*>(src)[65 + 2 * lane];
      w = make_uint4(round2(c.x, c.y), round2(c.z, c.w), round2(d.x, d.y), round2(d.z, d.w));
    }
    pair = reinterpret_cast<const float2*>(src)[kNopeDim / 2 + lane];
  } else {
    const uint16_t* const src = static_cast<const uint16_t*>(p.x) + row * p.x_row_stride;
    v = reinterpret_cast<const uint4*>(src)[lane];
    if (lane < 24) w = reinterpret_cast<const uint4*>(src)[32 + lane];
    const uint32_t two = reinterpret_cast<const uint32_t*>(src)[kNopeDim / 2 + lane];
    pair = make_float2(dev::bf16_lo(two), dev::bf16_hi(two));
  }
  if (slot < 0) return;
  bool ok = slot < p.num_pages * kSlotsPerPage;
  if (turns) {
    const bool in = static_cast<uint64_t>(at) < static_cast<uint64_t>(p.rotation.num_positions);
    const float2 angle = pair_angle(p.rotation, in ? at : 0, lane);
    pair = turn_pair(pair, angle.x, angle.y);
    ok = ok && in;
  }
  if (!__all_sync(0xFFFFFFFFu, ok)) {
    if (lane == 0) dev::record_error(p.error, dev::kErrBadIndex);
    return;
  }
  const uint32_t place = static_cast<uint32_t>(slot) % kSlotsPerPage;
  uint8_t* const base = p.kv_cache + static_cast<uint64_t>(static_cast<uint32_t>(slot / kSlotsPerPage)) * F::kPage;
  uint8_t* const payload = base + place * F::kStride;
  uint8_t* const scales = base + F::kScaleBase + place * F::kScales;
  reinterpret_cast<uint32_t*>(payload + F::kCodes)[lane] = round2(pair.x, pair.y);
  constexpr int kLanes = F::kFour ? 4 : 8;
  // above what a scale holds, infinite or NaN (infinities have the largest 8-bit code)
  constexpr uint32_t kMost = F::kFour ? kMost4 : 0x7F7Fu;
  uint32_t m = most_of_groups<kLanes>(v, w);
  const bool beyond = __any_sync(0xFFFFFFFFu, (m & 0xFFFFu) > kMost || m >> 16 > kMost);
  if (beyond) {
    v = bring_in(v, F::kFour ? kMost : 0x7F80u);
    w = bring_in(w, F::kFour ? kMost : 0x7F80u);
    m = most_of_groups<kLanes>(v, w);
  }
  const float a = __uint_as_float(m << 16), b = __uint_as_float(m & 0xFFFF0000u);
  if constexpr (F::kFour) {
    // (two bytes behind the 14 scales are zero: lanes 24 .. 31 hold no second run)
    const uint32_t byte0 = scale_byte(a), byte1 = scale_byte(b);
    reinterpret_cast<uint32_t*>(payload)[lane] = codes4(v, byte0);
    if (lane < 24) reinterpret_cast<uint32_t*>(payload)[32 + lane] = codes4(w, byte1);
    if ((lane & 3) == 0) {
      scales[lane / 4] = static_cast<uint8_t>(byte0);
      scales[8 + lane / 4] = static_cast<uint8_t>(byte1);
    }
  } else {
    const int e0 = dev::scale_exponent(fmaxf(a, 1.0e-4f)), e1 = dev::scale_exponent(fmaxf(b, 1.0e-4f));
    const uint2 c0 = beyond ? codes8<true>(v, e0) : codes8<false>(v, e0);
    const uint2 c1 = beyond ? codes8<true>(w, e1) : codes8<false>(w, e1);
    reinterpret_cast<uint2*>(payload)[lane] = c0;
    if (lane < 24) reinterpret_cast<uint2*>(payload)[32 + lane] = c1;
    if ((lane & 7) == 0) {
      scales[lane / 8] = static_cast<uint8_t>(e0 + 127);
      scales[4 + lane / 8] = static_cast<uint8_t>(lane < 24 ? e1 + 127 : 0);
    }
  }
}

// ---- 4-bit slots back ---------------------------------------------------------------

// A warp has kSlots slots, all loads of all of them ahead of the first store.  Where
// bf16 is asked for, lane l has dims 8 l .. + 7 and 256 + 8 l .. + 7 of each; of fp32
// values dims 4 l + 128 k .. + 3, k < 4: every store covers one run.  Bound by the
// bytes: 262144 slots in any order take 60 us in bf16 (6.1 TB/s of what a slot and a
// row have, and a slot's bytes come in pieces of 64) and 96 in fp32 (6.6 TB/s; 98
// without stores that are evicted first; in bf16 they are level).
// Slots of a warp, us, 1 / 2 / 3 / 4: 500 slots, bf16 1.6 / 1.7 / 1.9 / 2.0; 10000
// 2.9 / 3.4 / 2.9 / 3.8; 40000 11.3 / 10.9 / 10.5 / 11.4; 262144 65.1 / 60.2 / 60.2 /
// 62.2; fp32 98.1 / 98.7 / 99.4 / 103.4, and one is best at every size.
constexpr int64_t kFewSlots = 152 * 64;  // as many warps as fit at once
template <bool kBf16, int kSlots>
__global__ void __launch_bounds__(kWarps * 32) kvc_dequantize4_kernel(const uint8_t* kv, int64_t num_pages,
                                                                      const int64_t* slots, int64_t num_slots, void* out,
                                                                      uint32_t* err) {
  using F = Slots4;
  constexpr int kParts = kBf16 ? 2 : 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * kSlots;
  if (first >= num_slots) return;
  const bool rope = lane >= (kBf16 ? 24 : 16);  // of the last part
  int64_t slot[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) slot[u] = first + u < num_slots ? slots[first + u] : -1;
  uint32_t words[kSlots][kParts];
  uint4 tail[kSlots], scale[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
#pragma unroll
    for (int k = 0; k < kParts; ++k) words[u][k] = 0x88888888u;  // zeros
    tail[u] = scale[u] = make_uint4(0, 0, 0, 0);
    if (slot[u] < 0) continue;
    if (slot[u] >= num_pages * kSlotsPerPage) {
      if (lane == 0) dev::record_error(err, dev::kErrBadIndex);
      continue;
    }
    const uint8_t* const base = kv + slot[u] / kSlotsPerPage * F::kPage;
    const int place = static_cast<int>(slot[u] % kSlotsPerPage);
    const uint8_t* const payload = base + place * F::kStride;
    scale[u] = *reinterpret_cast<const uint4*>(base + F::kScaleBase + place * F::kScales);
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      if (k < kParts - 1 || !rope) {
        words[u][k] = *reinterpret_cast<const uint32_t*>(payload + (kBf16 ? 4 * (32 * k + lane) : 4 * (16 * k + lane / 2)));
      } else if constexpr (kBf16) {
        tail[u] = *reinterpret_cast<const uint4*>(payload + F::kCodes + 16 * (lane - 24));
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(payload + F::kCodes + 8 * (lane - 16));
        tail[u].x = v.x, tail[u].y = v.y;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    if (first + u >= num_slots) break;
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
      // the scale byte of group 8 k + l / 4, or 4 k + l / 8
      uint32_t record;
      if constexpr (kBf16)
        record = k == 0 ? (lane < 16 ? scale[u].x : scale[u].y) : (lane < 16 ? scale[u].z : scale[u].w);
      else
        record = k == 0 ? scale[u].x : k == 1 ? scale[u].y : k == 2 ? scale[u].z : scale[u].w;
      const uint32_t byte = record >> (8 * (kBf16 ? lane / 4 & 3 : lane / 8)) & 0xFFu;
      const uint32_t s = byte * 0x00100010u + kScale4Bits * 0x00010001u, less = mul_bf16x2(s, 0xC308C308u);
      const bool tails = k == kParts - 1 && rope;
      if constexpr (kBf16) {
        uint4 v = decode8_bf16(words[u][k], s, less);
        if (tails) v = tail[u];
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + (first + u) * kHeadDim)[32 * k + lane] = v;
      } else {
        const uint32_t half = words[u][k] >> (8 * (lane & 1));  // of a word's 8 dims
        uint32_t a = fma_bf16x2((half & 0x000F000Fu) | 0x43004300u, s, less);
        uint32_t b = fma_bf16x2((half >> 4 & 0x000F000Fu) | 0x43004300u, s, less);
        if (tails) a = tail[u].x, b = tail[u].y;
        __stcs(reinterpret_cast<float4*>(static_cast<float*>(out) + (first + u) * kHeadDim) + 32 * k + lane,
               make_float4(dev::bf16_lo(a), dev::bf16_hi(a), dev::bf16_lo(b), dev::bf16_hi(b)));
      }
    }
  }
}

template <typename... Params, typename... Args>
cudaError_t launch_rows(void (*kernel)(Params...), int64_t rows, int each, cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kWarps * each - 1) / (kWarps * each)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_store(const StoreParams& p, bool four_bits, cudaStream_t stream) {
  if (four_bits)
    return p.x_f32 ? launch_rows(kvc_store_kernel<Slots4, true>, p.num_rows, 1, stream, p)
                   : launch_rows(kvc_store_kernel<Slots4, false>, p.num_rows, 1, stream, p);
  return p.x_f32 ? launch_rows(kvc_store_kernel<Slots8, true>, p.num_rows, 1, stream, p)
                 : launch_rows(kvc_store_kernel<Slots8, false>, p.num_rows, 1, stream, p);
}

cudaError_t launch_dequantize4(const uint8_t* kv, int64_t num_pages, const int64_t* slots, int64_t num_slots, void* out,
                               int out_bf16, uint32_t* err, cudaStream_t stream) {
  if (!out_bf16)
    return launch_rows(kvc_dequantize4_kernel<false, 1>, num_slots, 1, stream, kv, num_pages, slots, num_slots, out, err);
  return num_slots <= kFewSlots
             ? launch_rows(kvc_dequantize4_kernel<true, 1>, num_slots, 1, stream, kv, num_pages, slots, num_slots, out, err)
             : launch_rows(kvc_dequantize4_kernel<true, 3>, num_slots, 3, stream, kv, num_pages, slots, num_slots, out, err);
}

}  // namespace kvc
