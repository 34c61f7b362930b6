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
// One CTA per request selects and writes the small arrays and the list of
// moves; a grid of warps then moves the slots, 584 bytes read and written each.
// Up to 8192 slots a request the CTA keeps 32-bit keys in registers, a run of
// neighbours a thread, and finds the keep-th largest two bits at a time by
// counting: 16 rounds of one barrier each, whatever the weights are (a histogram
// of digits took 24.7 us with its scans and its second pass over the keys on
// 64 x 8192, this TIME_SELECT).  Longer requests go by digits, with the keys in
// shared memory.  Where a request can move 64 slots at most (it has outgrown
// its share by less than a page), the selecting CTA moves them itself and the
// second kernel is not launched.

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
constexpr int kPerThread = 8;
constexpr int kShortSlots = kSelectThreads * kPerThread;  // 8192
constexpr int kFewMoves = 64;

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

__global__ void __launch_bounds__(kSelectThreads) kvc_evict_long_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t keys[];
  __shared__ SelectShared s;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  int2* const list = p.moves + r * p.move_stride;  // to, of

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
    if (!in && n < keep) list[h++].x = n;
    if (in && n >= keep) list[m++].y = n;
    if (in && n < keep) {
      if (kept != nullptr) kept[n] = n;
      if (weights_out != nullptr) weights_out[n] = weights[n];
      if (births_out != nullptr) births_out[n] = births[n];
    }
  }
  __syncthreads();
  const int moves = static_cast<int>(s.left);
  for (int i = t; i < moves; i += kSelectThreads) {
    const int to = list[i].x, of = list[i].y;
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

// Eight moves by one warp: 8 x 36 pieces of 16 bytes are 9 a lane, and lanes
// 0..7 have a scale record each.  Lane l < 8 holds move l's addresses.
__device__ __forceinline__ void move_eight(uint8_t* kv, const int32_t* table, const int2* moves, int count) {
  const int lane = threadIdx.x & 31;
  uint8_t *dst = nullptr, *src = nullptr;
  uint2 scale = make_uint2(0, 0);
  uint8_t* scale_to = nullptr;
  if (lane < count) {
    const int2 m = moves[lane];  // to, of
    uint8_t* const to = kv + table[m.x / kSlotsPerPage] * kPageBytes;
    uint8_t* const of = kv + table[m.y / kSlotsPerPage] * kPageBytes;
    dst = to + (m.x % kSlotsPerPage) * kTokenStride;
    src = of + (m.y % kSlotsPerPage) * kTokenStride;
    scale_to = to + kScaleBase + (m.x % kSlotsPerPage) * kScaleDim;
    scale = *reinterpret_cast<const uint2*>(of + kScaleBase + (m.y % kSlotsPerPage) * kScaleDim);
  }
  uint4 v[9];
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int slot = (32 * k + lane) / 36, piece = (32 * k + lane) % 36;
    const uint64_t from = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(src), slot);
    if (slot < count) v[k] = *reinterpret_cast<const uint4*>(from + 16 * piece);
  }
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int slot = (32 * k + lane) / 36, piece = (32 * k + lane) % 36;
    const uint64_t to = __shfl_sync(0xFFFFFFFFu, reinterpret_cast<uint64_t>(dst), slot);
    if (slot < count) *reinterpret_cast<uint4*>(to + 16 * piece) = v[k];
  }
  if (lane < count) *reinterpret_cast<uint2*>(scale_to) = scale;
}

// The moves of a request by the warps of grid.y CTAs.
__global__ void __launch_bounds__(kMoveWarps * 32) kvc_evict_move_kernel(const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x;
  const int moves = p.counts[r];
  const int32_t* const table = p.page_table + r * p.page_table_row_stride;
  const int2* const list = p.moves + r * p.move_stride;
  for (int i = 8 * (blockIdx.y * kMoveWarps + (threadIdx.x >> 5)); i < moves; i += 8 * gridDim.y * kMoveWarps)
    move_eight(p.kv_cache, table, list + i, min(8, moves - i));
}

// ---- up to kShortSlots slots a request --------------------------------------------

struct ShortShared {
  int holes[kShortSlots / 2], movers[kShortSlots / 2];  // as many as can be: of L slots, min(keep, L - keep)
  uint32_t counts[2][kSelectWarps];
  uint32_t warp_sums[kSelectWarps];
  int newest[kSelectWarps];
};

template <bool kMoves>
__global__ void __launch_bounds__(kSelectThreads) kvc_evict_short_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint8_t raw_shared[];
  ShortShared& s = *reinterpret_cast<ShortShared*>(raw_shared);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int64_t length = p.lengths[r];
  const int32_t* const table = p.page_table + r * p.page_table_row_stride;
  const float* const weights = p.weights + r * p.weights_row_stride;
  const int32_t* const births = p.births == nullptr ? nullptr : p.births + r * p.births_row_stride;
  const bool fits = length >= 0 && length <= p.max_slots;
  const int L = fits ? static_cast<int>(length) : 0, keep = static_cast<int>(p.keep < L ? p.keep : L);
  const int width = (L + kSelectThreads - 1) / kSelectThreads, lo = t * width;  // slots lo .. lo + width - 1
  // every load that the selection needs, at once
  float w[kPerThread];
  int born[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const bool in = j < width && lo + j < L;
    w[j] = in ? weights[lo + j] : 0.f;
    born[j] = in && births != nullptr ? births[lo + j] : INT32_MIN;
  }
  bool ok = fits;
  if (t * kSlotsPerPage < L) ok = static_cast<uint32_t>(table[t]) < p.num_pages;  // 128 pages at most
  int newest = INT32_MIN;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) newest = max(newest, born[j]);
  newest = __reduce_max_sync(0xFFFFFFFFu, newest);
  if (lane == 0) s.newest[warp] = newest;
  if (!__syncthreads_and(ok)) {  // the request stays as it is
    if (t == 0) {
      atomicCAS(p.error, 0u, kErrBadIndexEvict);
      p.counts[r] = 0;
    }
    return;
  }
  int32_t* const kept = p.kept == nullptr ? nullptr : p.kept + r * p.keep;
  float* const weights_out = p.weights_out == nullptr ? nullptr : p.weights_out + r * p.weights_out_row_stride;
  int32_t* const births_out = p.births_out == nullptr ? nullptr : p.births_out + r * p.births_out_row_stride;
  uint32_t key[kPerThread];  // 0 behind the length: below every slot's but a NaN's, and behind it in order
  const long long protect_above =
      p.recent > 0 ? static_cast<long long>(__reduce_max_sync(0xFFFFFFFFu, s.newest[lane])) - p.recent : INT64_MAX;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const bool in = j < width && lo + j < L;
    key[j] = !in ? 0u : born[j] > protect_above ? 0xFFFFFFFFu : order_key(w[j]);
  }
  // the keep-th largest key: the largest x with at least `keep` keys >= x
  uint32_t threshold = 0;
  if (keep > 0 && keep < L) {
#pragma unroll 1
    for (int shift = 30, turn = 0; shift >= 0; shift -= 2, turn ^= 1) {
      const uint32_t x1 = threshold | 1u << shift, x2 = threshold | 2u << shift, x3 = threshold | 3u << shift;
      uint32_t mine = 0;  // how many reach x1, x2, x3, in 10 bits each: 256 of a warp at most
#pragma unroll
      for (int j = 0; j < kPerThread; ++j)
        mine += (key[j] >= x1 ? 1u : 0u) + (key[j] >= x2 ? 1u << 10 : 0u) + (key[j] >= x3 ? 1u << 20 : 0u);
      mine = __reduce_add_sync(0xFFFFFFFFu, mine);
      if (lane == 0) s.counts[turn][warp] = mine;
      __syncthreads();
      const uint32_t all = s.counts[turn][lane];
      const uint32_t n1 = __reduce_add_sync(0xFFFFFFFFu, all & 1023u);
      const uint32_t n2 = __reduce_add_sync(0xFFFFFFFFu, all >> 10 & 1023u);
      const uint32_t n3 = __reduce_add_sync(0xFFFFFFFFu, all >> 20);
      threshold = n3 >= keep ? x3 : n2 >= keep ? x2 : n1 >= keep ? x1 : threshold;
    }
  }
  // of the keys equal to it, as many as are left to keep, from the lowest index
  uint32_t above = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const bool in = j < width && lo + j < L;
    above += in && key[j] > threshold;
    equal += in && key[j] == threshold;
  }
  uint32_t stays = 0;  // by bit, of this thread's slots
  if (keep == L) {
    stays = 0xFFu;
  } else if (keep > 0) {
    // 8192 slots at most: two sums of 16 bits in one scan
    const uint32_t before = block_exclusive(above << 16 | equal, s.warp_sums);
    if (t == kSelectThreads - 1) s.counts[0][0] = (before >> 16) + above;
    __syncthreads();
    const uint32_t spare = keep - s.counts[0][0];
    uint32_t rank = before & 0xFFFFu;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (key[j] > threshold || (key[j] == threshold && rank < spare)) stays |= 1u << j;
      rank += key[j] == threshold;
    }
  }
  uint32_t n_holes = 0, n_movers = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int n = lo + j;
    const bool in = j < width && n < L, stay = in && (stays >> j & 1u);
    n_holes += in && !stay && n < keep;
    n_movers += stay && n >= keep;
  }
  const uint32_t before = block_exclusive(n_holes << 16 | n_movers, s.warp_sums);
  int h = before >> 16, m = before & 0xFFFFu;
  if (t == kSelectThreads - 1) s.counts[1][0] = m + n_movers;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int n = lo + j;
    const bool in = j < width && n < L, stay = in && (stays >> j & 1u);
    if (in && !stay && n < keep) s.holes[h++] = n;
    if (stay && n >= keep) s.movers[m++] = n;
    if (stay && n < keep) {
      if (kept != nullptr) kept[n] = n;
      if (weights_out != nullptr) weights_out[n] = w[j];
      if (births_out != nullptr) births_out[n] = born[j];
    }
  }
  __syncthreads();
  const int moves = static_cast<int>(s.counts[1][0]);
  int2* const list = p.moves + r * p.move_stride;
  for (int i = t; i < moves; i += kSelectThreads) {
    const int to = s.holes[i], of = s.movers[i];
    list[i] = make_int2(to, of);
    if (kept != nullptr) kept[to] = of;
    // (an array written in place: sources lie at and behind the new length)
    if (weights_out != nullptr) weights_out[to] = weights[of];
    if (births_out != nullptr) births_out[to] = births[of];
  }
  if (kept != nullptr)
    for (int64_t j = keep + t; j < p.keep; j += kSelectThreads) kept[j] = -1;
  if (t == 0) {
    p.counts[r] = moves;
    p.lengths_out[r] = keep;
  }
  if constexpr (kMoves) {
    __syncthreads();
    for (int i = 8 * warp; i < moves; i += 8 * kSelectWarps) move_eight(p.kv_cache, table, list + i, min(8, moves - i));
  }
}

}  // namespace

namespace {

// Sets a kernel's shared memory once per context and launches it.
template <typename Kernel>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, size_t smem, const EvictParams& p, cudaStream_t stream) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  const dim3 reqs(static_cast<unsigned>(p.num_reqs));
  cudaError_t e;
  if (p.max_slots > kShortSlots) {
    const size_t smem = sizeof(uint32_t) * (p.max_slots < kCachedKeys ? p.max_slots : kCachedKeys);
    e = launch(kvc_evict_long_kernel, reqs, kSelectThreads, smem, p, stream);
  } else if (p.move_stride <= kFewMoves) {
    return launch(kvc_evict_short_kernel<true>, reqs, kSelectThreads, sizeof(ShortShared), p, stream);
  } else {
    e = launch(kvc_evict_short_kernel<false>, reqs, kSelectThreads, sizeof(ShortShared), p, stream);
  }
  if (e != cudaSuccess || p.move_stride == 0) return e;
  // a round of 8 moves for each warp if all the moves there can be are made,
  // unless that is more than fits the card several times
  const int64_t wide = (p.move_stride + 8 * kMoveWarps - 1) / (8 * kMoveWarps);
  const int64_t most = 2432 / p.num_reqs > 0 ? 2432 / p.num_reqs : 1;
  return launch(kvc_evict_move_kernel, dim3(reqs.x, static_cast<unsigned>(wide < most ? wide : most)),
                kMoveWarps * 32, 0, p, stream);
}

}  // namespace kvc
