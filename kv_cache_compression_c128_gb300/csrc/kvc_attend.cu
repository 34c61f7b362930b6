// Attention of one new token per request over the packed slots of its pages.
//
// Slots n < length_r of request r decode to vectors k_n (exactly; each is the
// key and the value of every head).  For head h:
//   s_n = scale * q_h . k_n,  L = log(sum_n exp(s_n) + exp(sink_h)),
//   out_h = sum_n exp(s_n - L) k_n,  lse_h = L,
// and, where the slots' weights are wanted,
//   weights_out[r, n] = weights_in[r, n] + sum_h exp(s_n - L_h).
// A row that sees no key (no slots, or every score -inf, and no sink) is
// zeros with lse -inf.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kvc_decode.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"

namespace kvc {
namespace {

constexpr uint32_t kErrBadIndexAttend = 4;
constexpr int kRowThreads = kHeadDim / 4;

// Four dims d0 .. d0 + 3 of slot n of a request's pages.
__device__ __forceinline__ void read4(const AttendParams& p, const int32_t* table, int n, int d0,
                                      float v[4]) {
  const uint8_t* page = p.kv_cache + table[n / kSlotsPerPage] * kPageBytes;
  const int off = n % kSlotsPerPage;
  if (d0 < kNopeDim) {
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(page + off * kTokenStride + d0);
    decode4(codes, half_scale(page[kScaleBase + off * kScaleDim + d0 / kGroup]), v);
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(page + off * kTokenStride + kNopeDim +
                                                    2 * (d0 - kNopeDim));
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
  }
}

// Whether the request's length and pages are in range; the whole block calls.
__device__ bool request_ok(const AttendParams& p, const int32_t* table, int64_t length) {
  bool ok = length >= 0 && length <= p.max_slots;
  if (ok)
    for (int64_t i = threadIdx.x; i * kSlotsPerPage < length; i += blockDim.x)
      ok = ok && static_cast<uint32_t>(table[i]) < p.num_pages;
  ok = __syncthreads_and(ok);
  if (!ok && threadIdx.x == 0) atomicCAS(p.error, 0u, kErrBadIndexAttend);
  return ok;
}

__global__ void __launch_bounds__(kRowThreads) kvc_attend_rows_kernel(AttendParams p) {
  __shared__ float part[2][4];
  const int h = blockIdx.x, t = threadIdx.x;
  const int64_t r = blockIdx.y;
  const int32_t* table = p.page_table + r * p.page_table_row_stride;
  const int64_t length = p.lengths[r];
  if (!request_ok(p, table, length)) return;
  const uint16_t* q = p.q + r * p.q_req_stride + h * p.q_head_stride + 4 * t;
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < 4; ++i) qv[i] = __uint_as_float(static_cast<uint32_t>(q[i]) << 16);
  float top = -INFINITY, total = 0.f;
  if (p.sinks != nullptr) {
    top = p.sinks[h];
    total = top == -INFINITY ? 0.f : 1.f;
  }
  for (int n = 0; n < length; ++n) {
    float v[4], dot = 0.f;
    read4(p, table, n, 4 * t, v);
    for (int i = 0; i < 4; ++i) dot += qv[i] * v[i];
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
    if ((t & 31) == 0) part[n & 1][t >> 5] = dot;
    __syncthreads();
    const float* w = part[n & 1];
    const float s = (w[0] + w[1] + w[2] + w[3]) * p.scale;
    const float next = fmaxf(top, s);
    if (next == -INFINITY && !isnan(s)) continue;
    const float keep = expf(top - next), e = expf(s - next);
    total = total * keep + e;
    for (int i = 0; i < 4; ++i) acc[i] = acc[i] * keep + e * v[i];
    top = next;
  }
  const float f = total == 0.f ? 0.f : 1.f / total;
  const int64_t row = r * p.num_heads + h;
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat16 b = __float2bfloat16_rn(acc[i] * f);
    p.out[row * kHeadDim + 4 * t + i] = *reinterpret_cast<const uint16_t*>(&b);
  }
  if (t == 0) p.lse[row] = total == 0.f ? -INFINITY : top + logf(total);
}

__global__ void __launch_bounds__(kRowThreads) kvc_attend_weights_kernel(AttendParams p) {
  __shared__ float part[4];
  const int t = threadIdx.x;
  const int64_t r = blockIdx.y;
  const int32_t* table = p.page_table + r * p.page_table_row_stride;
  const int64_t length = p.lengths[r];
  if (!request_ok(p, table, length)) return;
  for (int n = blockIdx.x; n < length; n += gridDim.x) {
    float v[4], sum = 0.f;
    read4(p, table, n, 4 * t, v);
    for (int h = 0; h < p.num_heads; ++h) {
      const uint16_t* q = p.q + r * p.q_req_stride + h * p.q_head_stride + 4 * t;
      float dot = 0.f;
      for (int i = 0; i < 4; ++i) dot += __uint_as_float(static_cast<uint32_t>(q[i]) << 16) * v[i];
      for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, d);
      __syncthreads();
      if ((t & 31) == 0) part[t >> 5] = dot;
      __syncthreads();
      const float s = (part[0] + part[1] + part[2] + part[3]) * p.scale;
      const float lse = p.lse[r * p.num_heads + h];
      if (lse != -INFINITY) sum += expf(s - lse);
    }
    if (t == 0)
      p.weights_out[r * p.weights_out_row_stride + n] =
          (p.weights_in == nullptr ? 0.f : p.weights_in[r * p.weights_in_row_stride + n]) + sum;
  }
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, cudaStream_t stream) {
  const unsigned reqs = static_cast<unsigned>(p.num_reqs);
  kvc_attend_rows_kernel<<<dim3(p.num_heads, reqs), kRowThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.weights_out == nullptr) return e;
  const unsigned wide = static_cast<unsigned>(p.max_slots < 1024 ? p.max_slots : 1024);
  kvc_attend_weights_kernel<<<dim3(wide, reqs), kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvc
