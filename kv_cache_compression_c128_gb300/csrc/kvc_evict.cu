// Eviction from a packed kv_cache by accumulated attention weight.
//
// Of a request's slots n < L the `keep` of largest weight stay (equal weights:
// the lowest index), the `recent` newest by birth number before all others.
// With new = min(L, keep), a kept slot n < new stays where it is, and the i-th
// hole below `new` takes the i-th kept slot behind it:
//   holes  h_0 < h_1 < ... = { n <  new : not kept }
//   movers m_0 < m_1 < ... = { n >= new : kept },    #holes == #movers.
// That is the fewest slots that can move (an order-preserving compaction would
// move nearly every kept slot behind the first hole), and since every source
// lies at or behind `new` and every destination before it, no copy waits for
// another and a repeated call writes the same bytes again.
//
// Two kernels: one CTA per request selects (radix select over 32-bit keys,
// then two block scans) and writes the small arrays and the list of moves;
// a grid of warps then moves the slots, 584 bytes read and written each.

#include <cuda_runtime.h>

#include <cstdint>

#include "kvc_internal.h"
#include "kvc_operators.h"

namespace kvc {
namespace {

constexpr uint32_t kErrBadIndexEvict = 4;
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigitBits = 11;  // 32-bit keys in digits of 11, 11 and 10 bits
constexpr int kBins = 1 << kDigitBits;
constexpr int kCachedKeys = 40960;  // keys held in shared memory (160 KiB); the rest are formed anew
constexpr int kMoveWarps = 8;

// Weights as whole numbers of the same order: -0 equals +0, NaN lies below
// all values, and protected slots above all.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t b = __float_as_uint(w + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_inclusive(uint32_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Exclusive sum over the block of one value a thread; every thread calls it.
__device__ uint32_t block_exclusive(uint32_t v, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t inc = warp_inclusive(v, lane);
  __syncthreads();
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const uint32_t s = warp_sums[lane];
    warp_sums[lane] = warp_inclusive(s, lane) - s;
  }
  __syncthreads();
  return warp_sums[warp] + inc - v;
}

struct SelectShared {
  uint32_t bins[kBins];
  uint32_t warp_sums[kSelectWarps];
  uint32_t digit, left;
  int newest;
  int bad;
};

__global__ void __launch_bounds__(kSelectThreads) kvc_evict_select_kernel(EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ SelectShared s;
  const int64_t r = blockIdx.x;
  const int t = threadIdx.x, lane = t & 31;
  int32_t* const count = p.counts + r;
  const int64_t length = p.lengths[r];
  const int64_t pages = length > 0 ? (length + kSlotsPerPage - 1) / kSlotsPerPage : 0;
  const int32_t* const table = p.page_table + r * p.page_table_row_stride;
  if (t == 0) {
    s.bad = length < 0 || length > p.max_slots;
    s.newest = INT32_MIN;
  }
  __syncthreads();
  if (!s.bad)
    for (int64_t i = t; i < pages; i += kSelectThreads)
      if (static_cast<uint32_t>(table[i]) >= p.num_pages) s.bad = 1;
  __syncthreads();
  if (s.bad) {  // the request stays as it is
    if (t == 0) {
      atomicCAS(p.error, 0u, kErrBadIndexEvict);
      *count = 0;
    }
    return;
  }
  const int L = static_cast<int>(length);
  const int keep = static_cast<int>(p.keep < length ? p.keep : length);
  const float* const weights = p.weights + r * p.weights_row_stride;
  const int32_t* const births = p.births == nullptr ? nullptr : p.births + r * p.births_row_stride;
  int32_t* const kept = p.kept == nullptr ? nullptr : p.kept + r * p.keep;
  float* const weights_out =
      p.weights_out == nullptr ? nullptr : p.weights_out + r * p.weights_out_row_stride;
  int32_t* const births_out =
      p.births_out == nullptr ? nullptr : p.births_out + r * p.births_out_row_stride;
  int32_t* const holes = p.moves + 2 * r * p.move_stride;
  int32_t* const movers = holes + p.move_stride;

  uint32_t threshold = 0;  // keys above it are kept
  uint32_t equal_left = 0;  // and this many of those equal to it, from the lowest index
  // a thread's share in index order; an odd width keeps the threads of a warp on 32 banks
  const int width = ((L + kSelectThreads - 1) / kSelectThreads) | 1;
  const int lo = min(L, t * width), hi = min(L, lo + width);
  long long protect_above = INT64_MAX;  // births above it are protected
  auto make_key = [&](int n) {
    if (births != nullptr && births[n] > protect_above) return 0xFFFFFFFFu;
    return order_key(weights[n]);
  };
  auto key_at = [&](int n) { return n < kCachedKeys ? keys[n] : make_key(n); };
  if (L > keep && keep > 0) {
    if (births != nullptr && p.recent > 0) {
      int newest = INT32_MIN;
      for (int n = t; n < L; n += kSelectThreads) newest = max(newest, births[n]);
      newest = __reduce_max_sync(0xFFFFFFFFu, newest);
      if (lane == 0) atomicMax(&s.newest, newest);
      __syncthreads();
      protect_above = static_cast<long long>(s.newest) - p.recent;
    }
    for (int n = t; n < min(L, kCachedKeys); n += kSelectThreads) keys[n] = make_key(n);
    // radix select: the keep-th largest key, a digit at a time from the top
    uint32_t left = keep, prefix = 0, mask = 0;
    for (int shift = 32 - kDigitBits; ; shift = max(0, shift - kDigitBits)) {
      for (int b = t; b < kBins; b += kSelectThreads) s.bins[b] = 0;
      __syncthreads();
      const uint32_t digit_mask = (0xFFFFFFFFu & ~mask) >> shift;
      for (int n0 = t - lane; n0 < L; n0 += kSelectThreads) {
        const int n = n0 + lane;
        const uint32_t key = n < L ? key_at(n) : 0u;
        const bool in = n < L && (key & mask) == prefix;
        const uint32_t d = (key >> shift) & digit_mask;
        // a warp of one digit (weights all alike) adds once
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, in);
        if (in) {
          int alike;
          __match_all_sync(who, d, &alike);
          if (!alike) {
            atomicAdd(&s.bins[d], 1u);
          } else if (lane == __ffs(who) - 1) {
            atomicAdd(&s.bins[d], static_cast<uint32_t>(__popc(who)));
          }
        }
      }
      __syncthreads();
      // keys in higher bins, for the two bins of each thread from the top down
      const int b1 = kBins - 1 - 2 * t, b0 = b1 - 1;
      const uint32_t c1 = s.bins[b1], c0 = s.bins[b0];
      const uint32_t above = block_exclusive(c1 + c0, s.warp_sums);
      if (above < left && left <= above + c1) {
        s.digit = b1;
        s.left = left - above;
      } else if (above + c1 < left && left <= above + c1 + c0) {
        s.digit = b0;
        s.left = left - above - c1;
      }
      __syncthreads();
      prefix |= s.digit << shift;
      mask |= digit_mask << shift;
      left = s.left;
      if (shift == 0) break;
    }
    threshold = prefix;
    uint32_t equal = 0;
    for (int n = lo; n < hi; ++n) equal += key_at(n) == threshold;
    const uint32_t before = block_exclusive(equal, s.warp_sums);
    equal_left = left > before ? left - before : 0;
  }
  const bool all = L <= keep, none = keep == 0;
  // holes in the low half and movers in the high half of one sum would pass
  // 16 bits: two sums
  uint32_t n_holes = 0, n_movers = 0, eq = equal_left;
  auto is_kept = [&](int n, uint32_t* eq_left) {
    if (all) return true;
    if (none) return false;
    const uint32_t k = key_at(n);
    if (k != threshold) return k > threshold;
    if (*eq_left == 0) return false;
    --*eq_left;
    return true;
  };
  for (int n = lo; n < hi; ++n) {
    const bool in = is_kept(n, &eq);
    n_holes += !in && n < keep;
    n_movers += in && n >= keep;
  }
  uint32_t h = block_exclusive(n_holes, s.warp_sums);
  uint32_t m = block_exclusive(n_movers, s.warp_sums);
  if (t == kSelectThreads - 1) s.left = m + n_movers;
  eq = equal_left;
  for (int n = lo; n < hi; ++n) {
    const bool in = is_kept(n, &eq);
    if (!in && n < keep) holes[h++] = n;
    if (in && n >= keep) movers[m++] = n;
    if (in && n < keep) {
      if (kept != nullptr) kept[n] = n;
      if (weights_out != nullptr) weights_out[n] = weights[n];
      if (births_out != nullptr) births_out[n] = births[n];
    }
  }
  __syncthreads();
  const int moves = static_cast<int>(s.left);
  for (int i = t; i < moves; i += kSelectThreads) {
    const int to = holes[i], of = movers[i];
    if (kept != nullptr) kept[to] = of;
    if (weights_out != nullptr) weights_out[to] = weights[of];
    if (births_out != nullptr) births_out[to] = births[of];
  }
  if (kept != nullptr)
    for (int64_t j = keep + t; j < p.keep; j += kSelectThreads) kept[j] = -1;
  if (t == 0) {
    *count = moves;
    p.lengths_out[r] = keep;
  }
}

// One warp per moved slot: 36 16-byte pieces and the 8-byte scale record.
__global__ void __launch_bounds__(kMoveWarps * 32) kvc_evict_move_kernel(EvictParams p) {
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 31;
  const int moves = p.counts[r];
  const int32_t* const table = p.page_table + r * p.page_table_row_stride;
  const int32_t* const holes = p.moves + 2 * r * p.move_stride;
  const int32_t* const movers = holes + p.move_stride;
  for (int i = blockIdx.y * kMoveWarps + (threadIdx.x >> 5); i < moves; i += gridDim.y * kMoveWarps) {
    const int to = holes[i], of = movers[i];
    uint8_t* const dst = p.kv_cache + table[to / kSlotsPerPage] * kPageBytes;
    const uint8_t* const src = p.kv_cache + table[of / kSlotsPerPage] * kPageBytes;
    const int64_t dp = (to % kSlotsPerPage) * kTokenStride, sp = (of % kSlotsPerPage) * kTokenStride;
    const int ds = kScaleBase + (to % kSlotsPerPage) * kScaleDim;
    const int ss = kScaleBase + (of % kSlotsPerPage) * kScaleDim;
    const uint4 a = *reinterpret_cast<const uint4*>(src + sp + 16 * lane);
    uint4 b = make_uint4(0, 0, 0, 0);
    uint2 c = make_uint2(0, 0);
    if (lane < 4) b = *reinterpret_cast<const uint4*>(src + sp + 512 + 16 * lane);
    if (lane == 4) c = *reinterpret_cast<const uint2*>(src + ss);
    *reinterpret_cast<uint4*>(dst + dp + 16 * lane) = a;
    if (lane < 4) *reinterpret_cast<uint4*>(dst + dp + 512 + 16 * lane) = b;
    if (lane == 4) *reinterpret_cast<uint2*>(dst + ds) = c;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const size_t smem = sizeof(uint32_t) * (p.max_slots < kCachedKeys ? p.max_slots : kCachedKeys);
  cudaError_t e = cudaFuncSetAttribute(kvc_evict_select_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(sizeof(uint32_t) * kCachedKeys));
  if (e != cudaSuccess) return e;
  kvc_evict_select_kernel<<<static_cast<unsigned>(p.num_reqs), kSelectThreads, smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.move_stride == 0) return e;
  const int64_t wide = (p.move_stride + 4 * kMoveWarps - 1) / (4 * kMoveWarps);
  const dim3 grid(static_cast<unsigned>(p.num_reqs), static_cast<unsigned>(wide < 64 ? wide : 64));
  kvc_evict_move_kernel<<<grid, kMoveWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace kvc
