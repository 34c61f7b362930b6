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
// Up to 8192 slots a request the CTA keeps 32-bit keys in registers, 8 a
// thread, and finds the keep-th largest two bits at a time by
// counting: at most 16 rounds of one barrier each, fewer where a threshold is
// met that exactly `keep` keys reach (a histogram of digits took 24.7 us with its
// scans and its second pass over the keys on 64 x 8192, this 23 us).  Longer
// requests go by digits, with the keys in shared memory (32 x 16384 to 8192:
// 76.6 us).  Where a request can move 64 slots at most (it has outgrown
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
constexpr int kMoveWarps = 8, kMoveCtasPerSm = 3;
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

// A move as the list holds it: the slots' numbers in the cache, page * 64 + place.
__device__ __forceinline__ longlong2 move_of(const int32_t* table, int to, int of) {
  return make_longlong2(static_cast<long long>(table[to / kSlotsPerPage]) * kSlotsPerPage + to % kSlotsPerPage,
                        static_cast<long long>(table[of / kSlotsPerPage]) * kSlotsPerPage + of % kSlotsPerPage);
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
  longlong2* const list = p.moves + r * p.move_stride;  // places first, then the slots' numbers

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
    const int to = static_cast<int>(list[i].x), of = static_cast<int>(list[i].y);
    list[i] = move_of(table, to, of);
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
// 0..7 have a move and its scale record each.
__device__ __forceinline__ void move_eight(uint8_t* kv, longlong2 m, int count) {
  const int lane = threadIdx.x & 31;
  uint64_t dst = 0, src = 0;
  uint2 scale = make_uint2(0, 0);
  uint8_t* scale_to = nullptr;
  if (lane < count) {
    uint8_t* const to = kv + m.x / kSlotsPerPage * kPageBytes;
    const uint8_t* const of = kv + m.y / kSlotsPerPage * kPageBytes;
    const int p = static_cast<int>(m.x % kSlotsPerPage), q = static_cast<int>(m.y % kSlotsPerPage);
    dst = reinterpret_cast<uint64_t>(to + p * kTokenStride);
    src = reinterpret_cast<uint64_t>(of + q * kTokenStride);
    scale_to = to + kScaleBase + p * kScaleDim;
    scale = *reinterpret_cast<const uint2*>(of + kScaleBase + q * kScaleDim);
  }
  uint4 v[9];
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int slot = (32 * k + lane) / 36, piece = (32 * k + lane) - 36 * slot;
    const uint64_t from = __shfl_sync(0xFFFFFFFFu, src, slot);
    if (slot < count) v[k] = *reinterpret_cast<const uint4*>(from + 16 * piece);
  }
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    const int slot = (32 * k + lane) / 36, piece = (32 * k + lane) - 36 * slot;
    const uint64_t to = __shfl_sync(0xFFFFFFFFu, dst, slot);
    if (slot < count) *reinterpret_cast<uint4*>(to + 16 * piece) = v[k];
  }
  if (lane < count) *reinterpret_cast<uint2*>(scale_to) = scale;
}

// The moves of a request by the warps of grid.y CTAs, which are all resident:
// a warp asks for its next moves before it makes the present ones.
__global__ void __launch_bounds__(kMoveWarps * 32, kMoveCtasPerSm) kvc_evict_move_kernel(
    const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int64_t r = blockIdx.x;
  const int lane = threadIdx.x & 31, step = 8 * gridDim.y * kMoveWarps;
  const longlong2* const list = p.moves + r * p.move_stride;
  const int moves = p.counts[r];
  int i = 8 * (blockIdx.y * kMoveWarps + (threadIdx.x >> 5));
  longlong2 m = make_longlong2(0, 0);
  if (lane < 8 && i + lane < moves) m = list[i + lane];
#pragma unroll 1
  for (; i < moves; i += step) {
    longlong2 next = make_longlong2(0, 0);
    if (lane < 8 && i + step + lane < moves) next = list[i + step + lane];
    move_eight(p.kv_cache, m, min(8, moves - i));
    m = next;
  }
}

// ---- up to kShortSlots slots a request --------------------------------------------

struct ShortShared {
  int holes[kShortSlots / 2], movers[kShortSlots / 2];  // as many as can be: of L slots, min(keep, L - keep)
  uint32_t counts[2][kSelectWarps];
  uint32_t ranks[kPerThread][kSelectWarps], rows[kPerThread];
  int newest[kSelectWarps];
};

// Thread t has slots 1024 j + t, j < 8.  From two truth values of each, the
// ranks in slot order of those that are true: `first` in the high halves,
// `second` in the low ones (8192 at most).  Returns both totals; all call.
__device__ uint32_t rank_slots(const bool* first, const bool* second, uint32_t* rank, ShortShared& s) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t below = (1u << lane) - 1;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const uint32_t a = __ballot_sync(0xFFFFFFFFu, first[j]), b = __ballot_sync(0xFFFFFFFFu, second[j]);
    rank[j] = static_cast<uint32_t>(__popc(a & below)) << 16 | __popc(b & below);
    if (lane == 0) s.ranks[j][warp] = static_cast<uint32_t>(__popc(a)) << 16 | __popc(b);
  }
  __syncthreads();
  if (warp < kPerThread) {
    const uint32_t v = s.ranks[warp][lane], inc = warp_inclusive(v, lane);
    s.ranks[warp][lane] = inc - v;
    if (lane == 31) s.rows[warp] = inc;
  }
  __syncthreads();
  uint32_t total = 0;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    rank[j] += total + s.ranks[j][warp];
    total += s.rows[j];
  }
  return total;
}

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
  const int width = (L + kSelectThreads - 1) / kSelectThreads;  // slots of a thread: 1024 j + t
  // every load that the selection needs, at once
  float w[kPerThread];
  int born[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int n = kSelectThreads * j + t;
    w[j] = n < L ? weights[n] : 0.f;
    born[j] = n < L && births != nullptr ? births[n] : INT32_MIN;
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
  for (int j = 0; j < kPerThread; ++j)
    key[j] = kSelectThreads * j + t >= L ? 0u : born[j] > protect_above ? 0xFFFFFFFFu : order_key(w[j]);
  // the keep-th largest key: the largest x with at least `keep` keys >= x, or
  // any x that exactly `keep` keys reach
  uint32_t threshold = 0;
  if (keep > 0 && keep < L) {
#pragma unroll 1
    for (int shift = 30, turn = 0, found = 0; shift >= 0 && !found; shift -= 2, turn ^= 1) {
      const uint32_t x1 = threshold | 1u << shift, x2 = threshold | 2u << shift, x3 = threshold | 3u << shift;
      uint32_t mine = 0;  // how many reach x1, x2, x3, in 10 bits each: 256 of a warp at most
#pragma unroll
      for (int j = 0; j < kPerThread; ++j)
        if (j < width)
          mine += (key[j] >= x1 ? 1u : 0u) + (key[j] >= x2 ? 1u << 10 : 0u) + (key[j] >= x3 ? 1u << 20 : 0u);
      mine = __reduce_add_sync(0xFFFFFFFFu, mine);
      if (lane == 0) s.counts[turn][warp] = mine;
      __syncthreads();
      const uint32_t all = s.counts[turn][lane];
      const uint32_t n1 = __reduce_add_sync(0xFFFFFFFFu, all & 1023u);
      const uint32_t n2 = __reduce_add_sync(0xFFFFFFFFu, all >> 10 & 1023u);
      const uint32_t n3 = __reduce_add_sync(0xFFFFFFFFu, all >> 20);
      threshold = n3 >= keep ? x3 : n2 >= keep ? x2 : n1 >= keep ? x1 : threshold;
      found = n1 == keep || n2 == keep || n3 == keep;
    }
  }
  // of the keys equal to it, as many as are left to keep, from the lowest index
  bool stay[kPerThread], other[kPerThread];
  uint32_t rank[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const bool in = kSelectThreads * j + t < L;
    stay[j] = in && (keep == L || (keep > 0 && key[j] > threshold));
    other[j] = in && keep > 0 && keep < L && key[j] == threshold;
  }
  if (keep < L) {
    const uint32_t spare = keep - (rank_slots(stay, other, rank, s) >> 16);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) stay[j] = stay[j] || (other[j] && (rank[j] & 0xFFFFu) < spare);
  }
  bool hole[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int n = kSelectThreads * j + t;
    hole[j] = n < keep && !stay[j];
    other[j] = n >= keep && stay[j];  // moves
  }
  const int moves = keep == L ? 0 : rank_slots(hole, other, rank, s) & 0xFFFFu;
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int n = kSelectThreads * j + t;
    if (hole[j]) s.holes[rank[j] >> 16] = n;
    if (other[j]) s.movers[rank[j] & 0xFFFFu] = n;
    if (n < keep && stay[j]) {
      if (kept != nullptr) kept[n] = n;
      if (weights_out != nullptr) weights_out[n] = w[j];
      if (births_out != nullptr) births_out[n] = born[j];
    }
  }
  __syncthreads();
  longlong2* const list = p.moves + r * p.move_stride;
  for (int i = t; i < moves; i += kSelectThreads) {
    const int to = s.holes[i], of = s.movers[i];
    const longlong2 move = move_of(table, to, of);
    list[i] = move;
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
    if (moves == 0) return;
    for (int i = 8 * warp; i < moves; i += 8 * kSelectWarps) {
      const int of_list = min(i + (lane & 7), moves - 1);
      move_eight(p.kv_cache, move_of(table, s.holes[of_list], s.movers[of_list]), min(8, moves - i));
    }
  }
}

// Launches a kernel that waits for the one ahead of it on the stream by itself.
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
  // as many CTAs as fit at once, shared out evenly over the requests, and no
  // more than all the moves there can be need
  const int64_t wide = (p.move_stride + 8 * kMoveWarps - 1) / (8 * kMoveWarps);
  const int64_t share = kMoveCtasPerSm * 152 / p.num_reqs, most = share > 0 ? share : 1;
  return launch(kvc_evict_move_kernel, dim3(reqs.x, static_cast<unsigned>(wide < most ? wide : most)),
                kMoveWarps * 32, 0, p, stream);
}

}  // namespace kvc
