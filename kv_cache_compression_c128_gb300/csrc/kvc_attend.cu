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
//
// One page (64 slots) at a time, with the slots and dims on the rows of the
// tensor core's tiles and the heads on their columns, so that the time of a
// page falls with the number of heads (padded to N = 16, 32 or 64; more heads
// make several groups):
//   S[slot, head]  = K[64 x 512] Q^T              (M 64,  N heads, K 512)
//   O[dim, head]  += K^T[128 dims x 64] P, 4 times (M 128, N heads, K 64)
// K is decoded to bf16 (exact) once, into shared memory with the 128-byte
// swizzle; the same bytes serve the first product with the dims innermost and
// the second one transposed.  S (2 buffers) and O are fp32 in tensor memory.
// P = 2^(s - m) goes to shared memory in bf16: its rounding is of the size of
// the output's own, and the sum l that divides is taken before it.  m is a
// column's reference, not its running maximum: any m serves as long as 2^(s - m)
// and its products stay in range, so O is rescaled only where a score exceeds m
// by 32, or at all on a page that holds values beyond 2^64.
//
// Warps of a CTA: 0..3 softmax and epilogue, one issues the products, one copies
// the codes, one the queries, seven decode, one brings the RoPE words.  The codes
// of a page come by TMA, a piece of 64 slots x 64 bytes for each scale group,
// through a ring: 24 KB (N 64) or 56 KB stay on their way whatever the decode
// does.  (Plain loads kept some 14 KB on the way, for the cache that they pass
// through is what shared memory leaves of it: 193 us on 64 requests x 8192 slots
// x 64 heads where the ring takes 125.)
//
// The (request, head group) units are cut into shares of pages, one per CTA: a
// unit to each where the longest takes hardly more than an equal share; else
// shares that begin anew with every unit; else all units' pages laid end to end
// and cut into equal shares.  The rule sees the lengths, on the device.  A unit
// that is divided leaves its parts (m, l, O) in the workspace, and a second kernel
// joins them in the order of the shares, so the same lengths give the same bits.
// That kernel also forms the slots' weights, from the scores that the first one
// left behind.
//
// What bounds it: a page's products take 1792 cycles at N = 64 and 1380 at 16,
// all of them operand reads from shared memory at 128 bytes a cycle (measured
// alone: 32 and 48 cycles for the M 64 and M 128 instruction at N 64, 23.5 and 39
// at N 16).  The decode's stores and loads of the same memory add some 1000, and a
// page takes about 4000 in all (2.1 us; 64 requests x 8192 slots x 64 heads: 125
// us, 2.5 TB/s and 0.55 PFLOP/s): beside the products every other access of
// shared memory is slow, a barrier's question 250 to 450 cycles.  Hence few
// questions, one short issuing loop, rolled loops throughout (180 us with straight
// code in every role, which does not stay in the instruction cache), and no more
// places than one for each decoding warp.  Small calls are bound by latency: 64
// slots of one request take 9 us, lengths, page ids, codes, two products and the
// rows one after the other.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <cstdint>

#include "kvc_device.cuh"
#include "kvc_internal.h"
#include "kvc_operators.h"

namespace kvc {
namespace {

using dev::kErrBadIndex;
using dev::kErrTimeout;
using dev::kLog2e;
using dev::smem_addr;

constexpr int kSoftmaxWarps = 4;
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
// Every fourth warp shares a scheduler: the products' issuer sits with the two
// copying warps, which mostly wait, apart from the decode and its long loop.
constexpr int kIssueWarp = 7, kCopyWarp = 11, kQueryWarp = 15;
constexpr int kAttendThreads = 16 * 32;
// Registers of a thread by group of four warps: 512 x 128 at launch, shared
// out anew so that no role spills (the cache that a spill would sit in is
// shared memory here).  128 x 168 + 384 x 112 <= 512 x 128.
constexpr int kSoftmaxRegs = 168, kOtherRegs = 112;
constexpr int kKeyBlock = kSlotsPerPage * 128;          // 64 slots x 64 dims, bf16
constexpr int kKeyStage = 8 * kKeyBlock;                // a decoded page
constexpr int kGroups = 7;                              // of 64 codes with one scale
constexpr int kPieceBytes = kSlotsPerPage * kGroup;     // a page's codes of one group
constexpr int kScaleBytes = kSlotsPerPage * kScaleDim;
// Pages described at a time.  While the RoPE words of page j are not there, its
// products are not issued, the decode is at page j + 2 at most, and the copies
// at page j + 3 + depth(): a page's place here is taken again eight pages later.
constexpr int kInfos = 8;
// Pages by which the longest unit may exceed an equal share before units are
// divided: joining the parts costs about as much as this many pages.
constexpr int kUndivided = 3;
// Requests at most for which shares begin anew with every unit (152 CTAs take no
// more units; a run of five requests a lane).
constexpr int kFewReqs = 160;
constexpr float kRescaleAbove = 32.f;                   // log2
// A page is large if a scale byte of it is above this, or a RoPE word not below
// 2^65: all others' values are below 2^65, and 2^30 slots (more than a request
// can have) of them times 2^32 stay in range.  On a large page the reference
// follows the maximum, so that no value is multiplied by more than 1.
constexpr uint32_t kLargeScale = 184;                   // 128 x 2^(184 - 127) = 2^64
constexpr int kJoinThreads = kAttendThreads, kJoinCtasPerSm = 2;
constexpr int kStatsPerLane = (kAttendCtas + 31) / 32;  // of a unit's parts

// Groups of a page whose codes come through the ring, one warp and depth()
// places each.  At N = 64 the 227 KB leave six places: the seventh group's warp
// loads its codes itself.  (Seven groups in turn on six places held the seventh
// piece up behind the first one's store; half places asked for twice a page, or
// loads a page ahead into registers, took longer.)
template <int N>
__host__ __device__ constexpr int ring_groups() { return N == 64 ? 6 : 7; }
// Pages that the ring holds, and pages whose scales are kept for its groups:
// page i's are asked for when all pieces of page i - 1 - depth() are read, and
// their scales before them.
template <int N>
__host__ __device__ constexpr int depth() { return N == 64 ? 1 : 2; }
template <int N>
__host__ __device__ constexpr int scale_slots() { return N == 64 ? 2 : 4; }

// A page on its way: its id (clamped), slots that count, whether it ends its segment.
struct PageInfo {
  int id;
  int16_t valid, last;
};

template <int N>
struct Barriers {
  // Of a stage's halves of 256 dims, and of its chunks of 128.  A wait of the
  // issuer costs some 250 cycles even if nothing is to be waited for, since
  // the products' operands keep shared memory busy: two a page, not eight.
  unsigned long long half_full[2][2], chunk_empty[2][4];
  unsigned long long s_full[2];
  unsigned long long p_full, q_full, q_empty, o_full, drain;
  unsigned long long piece_full[depth<N>()][ring_groups<N>()], piece_empty[depth<N>()][ring_groups<N>()], info_full[kInfos];
};

// What is left of a segment once its products are done: the rows of O, dims on
// the lanes and heads on the columns, times `factor` to `out` if the segment is
// the whole unit, as they are to its part otherwise.
struct Rows {
  int64_t row0;     // of out
  int part, heads;  // heads 0: nothing
  int whole;
};

template <int N>
struct AttendShared {
  alignas(1024) uint8_t keys[2][kKeyStage];
  alignas(1024) uint8_t q[N * 1024];
  alignas(1024) uint8_t p[kSlotsPerPage * 2 * N];
  alignas(1024) uint8_t codes[depth<N>()][ring_groups<N>()][kPieceBytes];
  alignas(16) uint8_t scales[scale_slots<N>()][kScaleBytes];
  union {
    float red[kSoftmaxWarps][N];
    int4 scan[kAttendThreads / 32];
  };
  float ref[N];
  alignas(8) float factor[N];
  Barriers<N> bar;
  PageInfo info[kInfos];
  uint8_t bad[8];  // of the last segments: a page was outside the cache
  uint8_t large[kInfos];  // of the pages in info
  int count, ctas, total, each;  // pages in all, and of a share that begins anew with every unit (0: equal shares)
  int start[4];  // request, length, unit and page of the share's first page
  Rows rows;     // of the last segment
  uint32_t tmem;
  volatile int abort;
};

// ---- tensor core and tensor memory ---------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Arrives on `bar` once every product issued so far by this thread is done.
__device__ __forceinline__ void tc_commit(unsigned long long* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_addr(bar))
               : "memory");
}

// Shared-memory operands are described by 64 bits: the start in the low word,
// the strides and the swizzle (2: 128 bytes, 4: 64, 6: 32).  Rows innermost
// (the first product): `sbo` bytes between groups of 8 rows.  Columns
// innermost (the second product): `lbo` between swizzle rows' widths along the
// columns, `sbo` between groups of 8 along the summed axis.
__host__ __device__ constexpr uint32_t operand_lo(uint32_t addr, uint32_t lbo) {
  return (addr >> 4) | (lbo >> 4) << 16;  // shared addresses lie below 2^18
}
__host__ __device__ constexpr uint32_t operand_hi(uint32_t sbo, uint32_t swizzle) {
  return (sbo >> 4) | (1u << 14) | (swizzle << 29);
}

template <uint32_t kHiA, uint32_t kHiB, uint32_t kInstruction>
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint32_t b, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %6, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(static_cast<uint32_t>(accumulate)), "n"(kHiA), "n"(kHiB), "r"(kInstruction)
      : "memory");
}

// One thread of a converged warp, the same one at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// fp32 accumulator, bf16 operands; `transposed`: both with their columns innermost.
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool transposed) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (transposed ? (1u << 15) | (1u << 16) : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

#define KVC_R4(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3])
#define KVC_R16(v, i) KVC_R4(v, i), KVC_R4(v, i + 4), KVC_R4(v, i + 8), KVC_R4(v, i + 12)

// 16 lanes x 16 columns: thread t gets columns 2 (t % 4) + {0, 1} of each 8,
// of lane t / 4 (values 0, 1) and t / 4 + 8 (values 2, 3).
__device__ __forceinline__ void tmem_ld_16x16(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : KVC_R4(v, 0), KVC_R4(v, 4)
               : "r"(addr));
}

// 32 lanes x 16 columns: thread t gets all columns of lane t.
__device__ __forceinline__ void tmem_ld_32x16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : KVC_R16(v, 0)
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st_32x16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// dev::mbar_wait_bounded in line (a call would have its registers counted
// against every role), and with the clock read only if the phase is not
// complete at once: read at every wait it took 270 cycles of the issuing
// thread each, 9 times a page.
__device__ __forceinline__ bool wait_for(unsigned long long* bar, uint32_t parity, long long limit) {
  const bool poll = limit < dev::kPollBelowCycles;
  if (!poll && dev::mbar_try_wait(bar, parity)) return true;
  const long long start = clock64();
  do {
    if (poll ? dev::mbar_test_wait(bar, parity) : dev::mbar_try_wait(bar, parity)) return true;
  } while (clock64() - start <= limit);
  return false;
}

// Barrier over the softmax warps; `or` of a predicate.
__device__ __forceinline__ void softmax_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kSoftmaxThreads) : "memory");
}
__device__ __forceinline__ bool softmax_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 3, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "n"(kSoftmaxThreads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// ---- the walk over a CTA's share -------------------------------------------------

// Pages of a request; none if its length is out of range.
__device__ __forceinline__ int pages_of(const AttendParams& p, int64_t length) {
  if (length <= 0 || length > p.max_slots) return 0;
  return static_cast<int>((length + kSlotsPerPage - 1) / kSlotsPerPage);
}

// Where a CTA is in its share: page `page` of `pages` of unit (req, group).
struct Walk {
  int req, group, page, pages, length;
  int left;  // pages of the share from here on

  __device__ int segment() const {
    return min(pages - page, left);
  }
  // On by `n` pages, at most to the unit's end.
  __device__ void advance(const AttendParams& p, int n) {
    left -= n;
    page += n;
    if (left <= 0 || page < pages) return;
    page = 0;
    if (++group < p.groups) return;
    group = 0;
    do {
      length = p.lengths[++req];
      pages = pages_of(p, length);
    } while (pages == 0);
  }
};

// Start of CTA c's share of `total` pages among `ctas`.
__device__ __forceinline__ int share_start(int total, int c, int ctas) {
  return static_cast<int>(static_cast<long long>(total) * c / ctas);
}

// The CTA whose share holds page `at`.
__device__ __forceinline__ int share_of(int total, int at, int ctas) {
  int c = static_cast<int>((static_cast<long long>(at + 1) * ctas - 1) / total);
  while (c > 0 && share_start(total, c, ctas) > at) --c;
  while (c + 1 < ctas && share_start(total, c + 1, ctas) <= at) ++c;
  return c;
}

// ---- decode -------------------------------------------------------------------------

// One tensor copy global -> shared of the box at (x, y, z), completing on `bar`.
__device__ __forceinline__ void copy_box(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

__device__ __forceinline__ void copy_bytes(void* dst, const void* src, uint32_t bytes, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Slots and tables are read with ordinary loads, not the read-only path's
// (.nc): this kernel may be resident while the one ahead of it on the stream
// still writes them (an eviction moves slots in place, and releases its
// dependents at its start), so they are not read-only for its lifetime.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// The larger magnitudes (with some sign).
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// 4 codes times 2^(b - 127) as two words of bf16, exactly.  u = code + 128 in
// the low bits of a bf16 is u 2^-133 (subnormal below 128, the first binade
// above: one linear scale); times 2^127 it is u 2^-6, and one fused
// multiply-add by 2^(b - 121) less 128 2^(b - 127) leaves code 2^(b - 127),
// 8 bits that are exact down to bf16's last subnormal.  b <= 247, so that
// both constants are bf16 values: `up` = (b + 6) << 7, `less` = -((b + 7) << 7)
// as bits, in both halves.  For a larger b the values of 247 are doubled
// b - 247 times: exact, or infinite where the value is.
__device__ __forceinline__ void decode4_bf16(uint32_t word, uint32_t up, uint32_t less, uint32_t* lo,
                                             uint32_t* hi) {
  const uint32_t u = word ^ 0x80808080u;
  *lo = fma_bf16x2(mul_bf16x2(__byte_perm(u, 0, 0x4140), 0x7F007F00u), up, less);
  *hi = fma_bf16x2(mul_bf16x2(__byte_perm(u, 0, 0x4342), 0x7F007F00u), up, less);
}

// ---- the roles ------------------------------------------------------------------------

template <int N>
__host__ __device__ constexpr uint32_t tmem_columns() { return N == 64 ? 512 : N == 32 ? 256 : 128; }

template <int N>
__device__ __forceinline__ int heads_of(const AttendParams& p, int group) {
  return min(p.group_heads, p.num_heads - group * p.group_heads);
}

// Copies the codes and scales of every page of the share: lane g the codes of
// group g, lane 31 the scales.  (One lane after the other's wait, announcement
// and copy took some 500 cycles a piece, 3500 a page, and held up all the rest.)
template <int N>
__device__ void copy_role(const AttendParams& p, AttendShared<N>& s, Walk w) {
  constexpr int kDepth = depth<N>(), kScales = scale_slots<N>(), kRing = ring_groups<N>();
  const int lane = threadIdx.x & 31;
  int i = 0;       // pages begun
  int asked = 0;   // of this lane's pieces, or pages' scales
  bool ok = true;
#pragma unroll 1
  for (int segment = 0; ok && w.left > 0; ++segment) {
    const int count = w.segment();
    const int32_t* table = p.page_table + w.req * p.page_table_row_stride + w.page;
    int ids = 0;  // of 32 pages, one a lane
#pragma unroll 1
    for (int pg = 0; ok && pg < count; ++pg, ++i) {
      if ((pg & 31) == 0) ids = pg + lane < count ? table[pg + lane] : 0;
      int id = __shfl_sync(0xFFFFFFFFu, ids, pg & 31);
      const bool there = static_cast<uint32_t>(id) < p.num_pages;
      if (!there) id = 0;
      if (lane == 31) {
        if (!there) {
          s.bad[segment & 7] = 1;
          atomicCAS(p.error, 0u, kErrBadIndex);
        }
        const int valid = there ? min(kSlotsPerPage, w.length - (w.page + pg) * kSlotsPerPage) : 0;
        s.info[i % kInfos] = PageInfo{id, static_cast<int16_t>(valid), static_cast<int16_t>(pg + 1 == count)};
        s.large[i % kInfos] = 0;
        dev::mbar_arrive_expect_tx(&s.bar.info_full[i % kInfos], kScaleBytes);
        copy_bytes(s.scales[i % kScales], p.kv_cache + id * kPageBytes + kScaleBase, kScaleBytes,
                   &s.bar.info_full[i % kInfos]);
        ++asked;
      }
      const int place = i % kDepth, turn = i / kDepth;
      if (lane < kRing) {
        ok = turn == 0 || wait_for(&s.bar.piece_empty[place][lane], (turn - 1) & 1, p.wait_limit);
        if (ok) {
          dev::mbar_arrive_expect_tx(&s.bar.piece_full[place][lane], kPieceBytes);
          copy_box(s.codes[place][lane], &p.code_map, lane * kGroup, 0, id, &s.bar.piece_full[place][lane]);
          ++asked;
        }
      }
      ok = __all_sync(0xFFFFFFFFu, ok && !s.abort);
    }
    w.advance(p, count);
  }
  if (!ok) s.abort = 1;
  // no copy may land in memory that the CTA has given back
  if (lane < kRing) {
#pragma unroll 1
    for (int j = max(0, asked - kDepth); j < asked; ++j)
      wait_for(&s.bar.piece_full[j % kDepth][lane], (j / kDepth) & 1, kDefaultWaitLimitCycles);
  } else if (lane == 31) {
#pragma unroll 1
    for (int j = max(0, asked - kInfos); j < asked; ++j)
      wait_for(&s.bar.info_full[j % kInfos], (j / kInfos) & 1, kDefaultWaitLimitCycles);
  }
  __syncwarp();
}

// Copies each segment's queries, in the layout of the products' operand.
template <int N>
__device__ void query_role(const AttendParams& p, AttendShared<N>& s, Walk w) {
#pragma unroll 1
  for (int segment = 0; w.left > 0; ++segment) {
    bool ok = segment == 0 || wait_for(&s.bar.q_empty, (segment - 1) & 1, p.wait_limit);
    if (!__all_sync(0xFFFFFFFFu, ok && !s.abort)) {
      s.abort = 1;
      return;
    }
    if (elect_one()) {
      dev::mbar_arrive_expect_tx(&s.bar.q_full, N * 1024);
#pragma unroll 1
      for (int b = 0; b < 8; ++b)
        copy_box(s.q + b * (N * 128), &p.q_map, 64 * b, w.group * p.group_heads, p.q_shared ? 0 : w.req, &s.bar.q_full);
    }
    __syncwarp();
    wait_for(&s.bar.q_full, segment & 1, kDefaultWaitLimitCycles);
    w.advance(p, w.segment());
  }
}

// Eight times 16 codes and their scale bytes as 16 bf16; sets *large if a scale
// byte is.
__device__ __forceinline__ void decode_rows(const uint4 (&raw)[8], const uint32_t (&scale)[8], uint4 (&lo)[8],
                                            uint4 (&hi)[8], uint8_t* large) {
  uint32_t most = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    most = max(most, scale[j]);
    const uint32_t b = min(scale[j], 247u), up = b * 0x00800080u + 0x03000300u, less = b * 0x00800080u + 0x83808380u;
    decode4_bf16(raw[j].x, up, less, &lo[j].x, &lo[j].y);
    decode4_bf16(raw[j].y, up, less, &lo[j].z, &lo[j].w);
    decode4_bf16(raw[j].z, up, less, &hi[j].x, &hi[j].y);
    decode4_bf16(raw[j].w, up, less, &hi[j].z, &hi[j].w);
  }
  if (__builtin_expect(__any_sync(0xFFFFFFFFu, most > kLargeScale), 0)) {
    *large = 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t more = (127u + max(scale[j], 247u) - 247u) * 0x00800080u;  // 2^(b - 247)
      lo[j] = make_uint4(mul_bf16x2(lo[j].x, more), mul_bf16x2(lo[j].y, more), mul_bf16x2(lo[j].z, more),
                         mul_bf16x2(lo[j].w, more));
      hi[j] = make_uint4(mul_bf16x2(hi[j].x, more), mul_bf16x2(hi[j].y, more), mul_bf16x2(hi[j].z, more),
                         mul_bf16x2(hi[j].w, more));
    }
  }
}

// Decodes group g of every page: 64 slots x 64 codes, 8 times 8 slots, lane l
// slot l / 4 of the 8 and codes 16 (l % 4) .. + 15.
template <int N>
__device__ void decode_role(const AttendParams& p, AttendShared<N>& s, int g, int count) {
  constexpr int kDepth = depth<N>(), kScales = scale_slots<N>();
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  uint32_t scale[8];
  uint4 raw[8];
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int stage = i & 1, place = i % kDepth;
    ok = ok && wait_for(&s.bar.info_full[i % kInfos], (i / kInfos) & 1, p.wait_limit);
    // (what is not described, after a wait that ran out, is not an address)
    const PageInfo info = ok ? s.info[i % kInfos] : PageInfo{0, 0, 0};
    if (g < ring_groups<N>()) {
#pragma unroll
      for (int j = 0; j < 8; ++j) scale[j] = s.scales[i % kScales][(r + 8 * j) * kScaleDim + g];
      ok = ok && wait_for(&s.bar.piece_full[place][g], (i / kDepth) & 1, p.wait_limit);
#pragma unroll
      for (int j = 0; j < 8; ++j) raw[j] = *reinterpret_cast<const uint4*>(s.codes[place][g] + (lane + 32 * j) * 16);
      // The place is given back once the values are there, not once they have
      // been asked for: an arrival does not wait for the loads before it, and
      // beside the products a load can take longer than the copy that then
      // overwrites what it reads.  So who arrives hangs on the values (it does
      // not matter who).
      uint32_t all = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) all ^= raw[j].x ^ scale[j];
      const int arrives = __all_sync(0xFFFFFFFFu, all == 1u) ? 1 : 0;
      if (lane == arrives) dev::mbar_arrive(&s.bar.piece_empty[place][g]);
    } else {
      const uint8_t* page = p.kv_cache + info.id * kPageBytes;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        raw[j] = load16(page + (r + 8 * j) * kTokenStride + g * kGroup + 16 * c);
        scale[j] = page[kScaleBase + (r + 8 * j) * kScaleDim + g];
      }
    }
    if (__builtin_expect(info.valid < kSlotsPerPage, 0)) {  // code 0 in every place of the slots that do not count
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (r + 8 * j >= info.valid) raw[j] = make_uint4(0, 0, 0, 0), scale[j] = 0;
    }
    // decoded before its place is free, so that only the stores are left then
    uint4 lo[8], hi[8];
    decode_rows(raw, scale, lo, hi, &s.large[i % kInfos]);
    if (i >= 2) ok = ok && wait_for(&s.bar.chunk_empty[stage][g >> 1], ((i >> 1) - 1) & 1, p.wait_limit);
    if (!__all_sync(0xFFFFFFFFu, ok && !s.abort)) {
      s.abort = 1;
      return;
    }
    uint8_t* const block = s.keys[stage] + g * kKeyBlock + r * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      *reinterpret_cast<uint4*>(block + 1024 * j + (((2 * c) ^ r) << 4)) = lo[j];
      *reinterpret_cast<uint4*>(block + 1024 * j + (((2 * c + 1) ^ r) << 4)) = hi[j];
    }
    fence_async_shared();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(&s.bar.half_full[stage][g >> 2]);
  }
}

// The RoPE words of every page, read into registers ahead (8 KB, which plain
// loads can keep on their way) and stored once their place is free: lane l has
// piece l % 8 of rows l / 8 + 4 j.
template <int N>
__device__ void rope_role(const AttendParams& p, AttendShared<N>& s, int count) {
  const int lane = threadIdx.x & 31, r = lane >> 3, c = lane & 7;
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    const int stage = i & 1;
    bool ok = wait_for(&s.bar.info_full[i % kInfos], (i / kInfos) & 1, p.wait_limit);
    const PageInfo info = ok ? s.info[i % kInfos] : PageInfo{0, 0, 0};
    const uint8_t* src = p.kv_cache + info.id * kPageBytes + r * kTokenStride + kNopeDim + 16 * c;
    uint4 v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)  // slots that do not count may hold anything, NaN too
      v[j] = r + 4 * j < info.valid ? load16(src + 4 * j * kTokenStride) : make_uint4(0, 0, 0, 0);
    if (i >= 2) ok = ok && wait_for(&s.bar.chunk_empty[stage][3], ((i >> 1) - 1) & 1, p.wait_limit);
    if (!__all_sync(0xFFFFFFFFu, ok && !s.abort)) {
      s.abort = 1;
      return;
    }
    uint8_t* const block = s.keys[stage] + kGroups * kKeyBlock + r * 128;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      *reinterpret_cast<uint4*>(block + 512 * j + ((c ^ (r + 4 * (j & 1))) << 4)) = v[j];
    // While the stores are on their way (before them: 128 requests x 1000 slots
    // x 8 heads 38.3 us instead of 37.9), the largest word: an exponent's two
    // highest bits are set from 2^65 on.  (A NaN is passed over; its slot's
    // scores are NaN.)
    uint32_t most[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      most[0] = max_abs_bf16x2(most[0], v[j].x);
      most[1] = max_abs_bf16x2(most[1], v[j].y);
      most[2] = max_abs_bf16x2(most[2], v[j].z);
      most[3] = max_abs_bf16x2(most[3], v[j].w);
    }
    const uint32_t top = max_abs_bf16x2(max_abs_bf16x2(most[0], most[1]), max_abs_bf16x2(most[2], most[3]));
    if (top & top << 1 & 0x40004000u) s.large[i % kInfos] = 1;
    fence_async_shared();
    __syncwarp();
    if (lane == 0) dev::mbar_arrive(&s.bar.half_full[stage][1]);
  }
}

// The products of every page: whatever can be issued next, a page's second
// product, which frees the place of the page after next, before a half of the
// next page's first.  The whole warp walks, one elected thread issues.  One
// short loop: the questions travel together and behind products already queued,
// and every role's code has to stay in the instruction cache beside the others'.
// (Questions by one lane instead of all: 137 us where this takes 125.)
template <int N>
__device__ void issue_role(const AttendParams& p, AttendShared<N>& s, int count) {
  constexpr uint32_t kFirst = instruction(64, N, false), kSecond = instruction(128, N, true);
  constexpr uint32_t kRows = operand_hi(1024, 2);
  constexpr uint32_t kProbs = operand_hi(16 * N, N == 64 ? 2 : N == 32 ? 4 : 6);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s.tmem, 0);
  const uint32_t q = operand_lo(smem_addr(s.q), 16), all_keys = smem_addr(s.keys);
  const uint32_t probs = operand_lo(smem_addr(s.p), 16);
  int halves = 0, done = 0;      // halves of first products and whole second products issued
  int segment = 0;               // segments begun
  bool begins = true;            // the next half begins a segment
  bool ends[2] = {true, false};  // the page of each stage ends its segment
  bool fresh = true;             // the next second product is its segment's first
  bool ok = true, idle = false;
  long long since = 0;  // idle
#pragma unroll 1
  while (done < count) {
    const int i = halves >> 1, half = halves & 1, stage = i & 1;
    const uint32_t parity = (i >> 1) & 1;
    // asked all at once: an answer takes long while products keep shared memory busy
    bool first = dev::mbar_test_wait(&s.bar.half_full[stage][half], parity);
    const bool other = dev::mbar_test_wait(&s.bar.half_full[stage][1], parity);
    const bool second = dev::mbar_test_wait(&s.bar.p_full, done & 1);
    if (begins) first = first && dev::mbar_test_wait(&s.bar.q_full, segment & 1);
    if (done < i && __all_sync(0xFFFFFFFFu, second)) {
      tc_fence_after();
      const int of = done & 1;
      const bool last = of == 0 ? ends[0] : ends[1];
      const uint32_t keys = operand_lo(all_keys + of * kKeyStage, kKeyBlock);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma<kRows, kProbs, kSecond>(tmem + c * N, keys + (2 * c * kKeyBlock + 2048 * k) / 16,
                                           probs + k * 32 * N / 16, !fresh || k > 0);
          tc_commit(&s.bar.chunk_empty[of][c]);  // the decode of page i + 2 follows chunk by chunk
        }
        if (last) tc_commit(&s.bar.o_full);
      }
      __syncwarp();
      fresh = last;
      ++done;
    } else if (i < count && __all_sync(0xFFFFFFFFu, first)) {
      tc_fence_after();
      const uint32_t into = tmem + 4 * N + stage * N;
      const int to = half == 1 || __all_sync(0xFFFFFFFFu, other) ? 2 : 1;
#pragma unroll 1
      for (int h = half; h < to; ++h) {
        const uint32_t keys = operand_lo(all_keys + stage * kKeyStage + h * (4 * kKeyBlock), 16);
        const uint32_t queries = q + h * (4 * N * 128 / 16);
        if (elect_one()) {
#pragma unroll
          for (int b = 0; b < 4; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma<kRows, kRows, kFirst>(into, keys + (b * kKeyBlock + 32 * k) / 16,
                                           queries + (b * (N * 128) + 32 * k) / 16, h + b + k > 0);
        }
        __syncwarp();
      }
      segment += begins;
      begins = false;
      if (to == 2) {
        begins = __any_sync(0xFFFFFFFFu, s.info[i % kInfos].last);
        ends[0] = stage == 0 ? begins : ends[0];
        ends[1] = stage == 1 ? begins : ends[1];
        if (elect_one()) {
          tc_commit(&s.bar.s_full[stage]);
          if (begins) tc_commit(&s.bar.q_empty);
        }
        __syncwarp();
      }
      halves += to - half;
    } else {
      const long long now = clock64();
      if (!idle) since = now;
      idle = true;
      if (__any_sync(0xFFFFFFFFu, now - since > p.wait_limit || s.abort)) {
        ok = false;
        break;
      }
      continue;
    }
    idle = false;
  }
  if (!ok) s.abort = 1;
  // no product may run on when the CTA's memory is given back
  if (elect_one()) tc_commit(&s.bar.drain);
  __syncwarp();
  wait_for(&s.bar.drain, 0, kDefaultWaitLimitCycles);
}

// Columns `from` .. `to` - 1 of the four chunks' 4 N, the lanes of a warp.
template <int N>
__device__ __forceinline__ void write_rows(const AttendParams& p, const AttendShared<N>& s, const Rows& rows, int from,
                                           int to) {
  constexpr int kWide = N == 16 ? 16 : 32;  // columns at a time
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t tmem = s.tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
  for (int at = from; at < to; at += kWide) {
    const int b = at % N, d = at / N * 128 + warp * 32 + lane;
    if (b >= rows.heads) continue;
    uint32_t o[kWide];
#pragma unroll
    for (int j = 0; j < kWide; j += 16) tmem_ld_32x16(tmem + at + j, o + j);
    tmem_wait_ld();
    if (rows.whole) {
      const bool odd = lane & 1;
      uint16_t* const out = p.out + (rows.row0 + b + odd) * kHeadDim + (d & ~1);
#pragma unroll
      for (int j = 0; j < kWide; j += 2) {
        // lanes 2 i and 2 i + 1 trade: one stores both dims of head j, the other of j + 1
        const float2 f = *reinterpret_cast<const float2*>(&s.factor[b + j]);
        const float a = __uint_as_float(o[j]) * f.x, e = __uint_as_float(o[j + 1]) * f.y;
        const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : e, 1);
        const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(got, e) : __floats2bfloat162_rn(a, got);
        if (b + j + odd < rows.heads) *reinterpret_cast<__nv_bfloat162*>(out + j * kHeadDim) = v;
      }
    } else {
      float* const dst = p.parts + (static_cast<int64_t>(rows.part) * N + b) * kHeadDim + d;
#pragma unroll
      for (int j = 0; j < kWide; ++j)
        if (b + j < rows.heads) dst[j * kHeadDim] = __uint_as_float(o[j]);
    }
  }
}

// Combines, over the eight lanes of equal lane % 4, kCount values a lane each:
// halves of the values are traded instead of all of them, so that
// kCount - 1 + ... shuffles do what 3 kCount would.  Lane l ends up with values
// kCount / 8 * (l / 4 with its bits reversed) and on.
template <int kCount, typename Op>
__device__ __forceinline__ void combine_rows(float (&v)[kCount], int lane, Op op) {
  int n = kCount;
#pragma unroll
  for (int d = 16; d >= 4; d >>= 1) {
    if (n > 1) {
      n >>= 1;
      const bool up = lane & d;
#pragma unroll
      for (int j = 0; j < kCount / 2; ++j) {
        if (j < n) {
          const float send = up ? v[j] : v[j + n], keep = up ? v[j + n] : v[j];
          v[j] = op(keep, __shfl_xor_sync(0xFFFFFFFFu, send, d));
        }
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], d));
    }
  }
}

// Stores what combine_rows left: value j of a thread belongs to column
// 8 (j / 2) + 2 (lane % 4) + j % 2.
template <int kCount>
__device__ __forceinline__ void store_combined(const float (&v)[kCount], int lane, float* columns) {
  constexpr int kLeft = kCount >= 8 ? kCount / 8 : 1;
  int j0 = 0;
  if (kCount >= 2) j0 += (lane & 16) ? kCount / 2 : 0;
  if (kCount >= 4) j0 += (lane & 8) ? kCount / 4 : 0;
  if (kCount >= 8) j0 += (lane & 4) ? kCount / 8 : 0;
#pragma unroll
  for (int k = 0; k < kLeft; ++k) columns[8 * ((j0 + k) >> 1) + 2 * (lane & 3) + ((j0 + k) & 1)] = v[k];
}

// Softmax warps.  Warp w has slots 16 w .. 16 w + 15 of a page: thread t the
// slots t / 4 and t / 4 + 8 of them, and columns 2 (t % 4) + {0, 1} of each 8.
template <int N>
__device__ void softmax_role(const AttendParams& p, AttendShared<N>& s, Walk w) {
  constexpr int kCols = N / 4;  // columns of a thread
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const uint32_t tmem = s.tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const float c = p.scale == 0.f ? 1.f : p.scale * kLog2e;  // scores of scale 0 are zeros
  const int row = warp * 16 + (lane >> 2);
  const int cta = blockIdx.x;
  int i = 0, at = share_start(s.total, cta, s.ctas);  // (used with equal shares)
  bool ok = true;  // once false, the next vote ends the role
#pragma unroll 1
  for (int segment = 0; w.left > 0; ++segment) {
    const int n = w.segment();
    float ref[kCols], sum[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) ref[j] = -FLT_MAX, sum[j] = 0.f;
#pragma unroll 1
    for (int pg = 0; pg < n; ++pg, ++i) {
      const int stage = i & 1;
      ok = __all_sync(0xFFFFFFFFu, ok && wait_for(&s.bar.s_full[stage], (i >> 1) & 1, p.wait_limit));
      tc_fence_after();
      const float above = s.large[i % kInfos] ? 0.f : kRescaleAbove;
      uint32_t v[2 * kCols];
      float x[2 * kCols];  // scores in powers of two
#pragma unroll
      for (int j = 0; j < N / 16; ++j) tmem_ld_16x16(tmem + 4 * N + stage * N + 16 * j, v + 8 * j);
      tmem_wait_ld();
      const int valid = w.length - (w.page + pg) * kSlotsPerPage;
      const bool in0 = row < valid, in1 = row + 8 < valid;
      if (__builtin_expect(p.scale == 0.f, 0)) {
#pragma unroll
        for (int j = 0; j < 2 * kCols; ++j) v[j] = 0;
      }
      // Rounded once, before anything is subtracted: the reference is one of
      // these numbers, and the largest score's distance from it has to be 0
      // (v c - ref in one step keeps what rounding took from the reference:
      // from |v c| of 2^31 on more than the 126 after which exp2 is 0 or
      // infinite, and the row was zeros or NaN).
#pragma unroll
      for (int j = 0; j < 2 * kCols; ++j) x[j] = __fmul_rn(__uint_as_float(v[j]), c);
      if (__builtin_expect(valid < kSlotsPerPage, 0)) {  // slots behind the request's last one
#pragma unroll
        for (int j = 0; j < 2 * kCols; ++j)
          if (!((j & 2) ? in1 : in0)) x[j] = -INFINITY;
      }
      if (__builtin_expect(p.scores != nullptr, 0)) {
        float* dst = p.scores + ((w.req * p.max_pages + w.page + pg) * kSlotsPerPage + row) * p.score_cols +
                     w.group * N + 2 * (lane & 3);
#pragma unroll
        for (int j = 0; j < N / 8; ++j) {
          if (in0) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(x[4 * j], x[4 * j + 1]);
          if (in1) *reinterpret_cast<float2*>(dst + 8 * p.score_cols + 8 * j) = make_float2(x[4 * j + 2], x[4 * j + 3]);
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 2 * kCols; ++j)
        top = fmaxf(top, __fsub_rn(x[j], ref[(j >> 2) * 2 + (j & 1)]));
      if (__builtin_expect(softmax_any(top > above || !ok), 0)) {
        if (softmax_any(!ok)) {
          s.abort = 1;
          return;
        }
        // the columns' maxima over the page
        float m[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) m[j] = fmaxf(x[4 * (j >> 1) + (j & 1)], x[4 * (j >> 1) + 2 + (j & 1)]);
        combine_rows(m, lane, [](float a, float b) { return fmaxf(a, b); });
        store_combined(m, lane, s.red[warp]);
        softmax_sync();
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const int col = 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
          const float next = fmaxf(fmaxf(fmaxf(s.red[0][col], s.red[1][col]),
                                         fmaxf(s.red[2][col], s.red[3][col])), ref[j]);
          const float f = exp2_fast(ref[j] - next);
          sum[j] *= f;
          ref[j] = next;
          if (warp == 0 && lane < 4) s.factor[col] = f;
        }
        softmax_sync();
        if (pg > 0) {  // bring what is summed up so far to the new reference
          ok = __all_sync(0xFFFFFFFFu, wait_for(&s.bar.chunk_empty[stage ^ 1][3], ((i - 1) >> 1) & 1, p.wait_limit));
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < 4 * N; b += 16) {
            uint32_t o[16];
            tmem_ld_32x16(tmem + b, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = __float_as_uint(__uint_as_float(o[j]) * s.factor[(b + j) & (N - 1)]);
            tmem_st_32x16(tmem + b, o);
          }
          tmem_wait_st();
        }
      }
      __nv_bfloat162 pair[kCols];
#pragma unroll
      for (int j = 0; j < kCols; ++j) {  // columns of j / 2, rows of j % 2
        const int col = j & ~1;
        const float a = exp2_fast(__fsub_rn(x[2 * j], ref[col]));
        const float b = exp2_fast(__fsub_rn(x[2 * j + 1], ref[col + 1]));
        sum[col] += a;
        sum[col + 1] += b;
        pair[j] = __floats2bfloat162_rn(a, b);
      }
      if (i > 0)  // the products of the page before have read its P
        ok = __all_sync(0xFFFFFFFFu,
                        ok && wait_for(&s.bar.chunk_empty[stage ^ 1][3], ((i - 1) >> 1) & 1, p.wait_limit));
#pragma unroll
      for (int j = 0; j < kCols; ++j) {
        const uint32_t off = (row + 8 * (j & 1)) * (2 * N) + 16 * (j >> 1) + 4 * (lane & 3);
        constexpr uint32_t kMask = N / 8 - 1;  // 16-byte pieces of a row
        *reinterpret_cast<__nv_bfloat162*>(s.p + (off ^ (((off >> 7) & kMask) << 4))) = pair[j];
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&s.bar.p_full);
    }
    // the segment's end: columns' sums, then the rows of O
    combine_rows(sum, lane, [](float a, float b) { return a + b; });
    store_combined(sum, lane, s.red[warp]);
    if (warp == 0 && lane < 4) {
#pragma unroll
      for (int j = 0; j < kCols; ++j) s.ref[8 * (j >> 1) + 2 * lane + (j & 1)] = ref[j];
    }
    softmax_sync();
    const bool whole = n == w.pages, bad = s.bad[segment & 7] != 0;
    const int part = 2 * cta + (segment > 0);
    const int heads = heads_of<N>(p, w.group);
    const int64_t row0 = static_cast<int64_t>(w.req) * p.num_heads + w.group * p.group_heads;
    if (t < heads) {
      const float l = s.red[0][t] + s.red[1][t] + s.red[2][t] + s.red[3][t], m = s.ref[t];
      float f = 1.f;
      if (whole) {
        float top = m, total = l;
        f = 1.f;
        if (p.sinks != nullptr) {
          const float sink = p.sinks[w.group * p.group_heads + t] * kLog2e;
          top = fmaxf(m, sink);
          f = exp2_fast(m - top);
          total = l * f + exp2_fast(sink - top);
        }
        if (!bad) p.lse[row0 + t] = total == 0.f ? -INFINITY : (top + log2f(total)) / kLog2e;
        if (p.row_stats != nullptr) p.row_stats[row0 + t] = make_float2(top, total == 0.f ? 0.f : 1.f / total);
        f = total == 0.f ? 0.f : f / total;
      } else {
        p.part_stats[part * N + t] = make_float2(m, l);
      }
      s.factor[t] = f;
    }
    if (t == 0) {
      if (w.page == 0) {  // the unit's first part: where its parts lie
        p.unit_parts[static_cast<int64_t>(w.req) * p.groups + w.group] =
            whole ? make_int2(-1, bad)
                  : make_int2(part, s.each > 0 ? cta + (w.pages - 1) / s.each : share_of(s.total, at + w.pages - 1, s.ctas));
      }
      if (!whole) {
        p.part_bad[part] = bad;
        if (w.page + n == w.pages) {  // the unit's last part: this share's joins it
          const int first = s.each > 0 ? cta - w.page / s.each : share_of(s.total, at - w.page, s.ctas);
          const bool at_start = s.each > 0 || share_start(s.total, first, s.ctas) == at - w.page;
          p.joins[cta] = make_int4(w.req, w.group, 2 * first + !at_start, cta);
        }
      }
    }
    ok = ok && wait_for(&s.bar.o_full, segment & 1, p.wait_limit);
    if (softmax_any(!ok)) {  // also makes s.factor visible
      s.abort = 1;
      return;
    }
    if (t == 0) s.bad[segment & 7] = 0;
    tc_fence_after();
    const Rows rows{row0, part, whole && bad ? 0 : heads, whole};
    if (w.left == n) {  // of the last segment the whole CTA writes the rows
      if (t == 0) s.rows = rows;
      return;
    }
    write_rows<N>(p, s, rows, 0, 4 * N);
    tc_fence_before();
    softmax_sync();  // s.red, s.factor and O are free again
    at += n;
    w.advance(p, n);
  }
}

// Shares of `each` pages that begin anew with every unit: the fewest pages for
// which the CTAs suffice, if not too many over an equal share (each 0: none).
// An equal share of several units ends several times, some 4 us each at N = 64:
// 32 requests of up to 4000 slots take 33.7 us with equal shares and 25.8 with
// these, 96 of up to 1500 35.6 and 28.2 (64 heads); 32 of up to 4000 at 16 heads
// 24.3 and 21.0.  Every warp tries a number; `own` and `before` are the finder's
// lanes'.  The search takes 1 us.
struct Shares {
  int each, count, finder, own, before;
};
template <int N>
__device__ __forceinline__ Shares aligned_shares(const AttendParams& p, int4* scan, int lo, int hi, int total, int units,
                                              int shortest, int grid) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, least = (total + grid - 1) / grid;
  Shares of = {0, 0, 0, 0, 0};
  // pages that it is worth: more for N = 64's longer end, and where a share could hold several short units
  const int several = min(least / __reduce_min_sync(0xFFFFFFFFu, shortest), 2);
  const int most = total / grid + (N == 64 ? 4 + 4 * several : 2);
  // a unit's last share is half empty on average: not tried where that is too much
  if (total / most + units / 2 > grid) return of;
#pragma unroll 1
  for (int r = lo; r < hi; ++r) of.own += (pages_of(p, p.lengths[r]) + least + warp - 1) / (least + warp);
  const int all = __reduce_add_sync(0xFFFFFFFFu, of.own) * p.groups;
  if (lane == 0) scan[warp].x = all;
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < kAttendThreads / 32 && least + i <= most; ++i) {
    of.count = scan[i].x;
    if (of.count > grid) continue;
    of.each = least + i;
    of.finder = i;
    of.before = warp_inclusive(of.own, lane) - of.own;
    break;
  }
  return of;
}

// A request without slots: zeros and the sinks; all kAttendThreads threads.
__device__ __forceinline__ void write_empty(const AttendParams& p, int64_t r) {
  const int64_t row0 = r * p.num_heads;
  uint4* const out = reinterpret_cast<uint4*>(p.out + row0 * kHeadDim);
#pragma unroll 1
  for (int i = threadIdx.x; i < p.num_heads * (kHeadDim / 8); i += kAttendThreads) out[i] = make_uint4(0, 0, 0, 0);
  if (threadIdx.x < p.num_heads) p.lse[row0 + threadIdx.x] = p.sinks == nullptr ? -INFINITY : p.sinks[threadIdx.x];
}

template <int N>
__global__ void __launch_bounds__(kAttendThreads, 1) kvc_attend_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(1024) uint8_t raw_shared[];
  AttendShared<N>& s = *reinterpret_cast<AttendShared<N>*>(raw_shared);
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int cta = blockIdx.x;
  if (warp == kIssueWarp) tmem_alloc(&s.tmem, tmem_columns<N>());
  if (t == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int j = 0; j < 2; ++j) dev::mbar_init(&s.bar.half_full[i][j], 4);
      for (int j = 0; j < 4; ++j) dev::mbar_init(&s.bar.chunk_empty[i][j], 1);
      dev::mbar_init(&s.bar.s_full[i], 1);
    }
    dev::mbar_init(&s.bar.p_full, kSoftmaxWarps);
    dev::mbar_init(&s.bar.q_full, 1);
    dev::mbar_init(&s.bar.q_empty, 1);
    dev::mbar_init(&s.bar.o_full, 1);
    dev::mbar_init(&s.bar.drain, 1);
    for (int i = 0; i < depth<N>() * ring_groups<N>(); ++i) {
      dev::mbar_init(&s.bar.piece_full[0][0] + i, 1);
      dev::mbar_init(&s.bar.piece_empty[0][0] + i, 1);
    }
    for (int i = 0; i < kInfos; ++i) dev::mbar_init(&s.bar.info_full[i], 1);
    dev::fence_mbar_init();
    s.abort = 0;
    for (int i = 0; i < 8; ++i) s.bad[i] = 0;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // Where the share lies: the pages (the host has checked that all fit 31 bits)
  // and the units before each thread's run of requests.  Up to kFewReqs requests
  // every warp finds it for itself, a run of requests a lane.
  const int reqs = static_cast<int>(p.num_reqs), grid = static_cast<int>(gridDim.x);
  const bool few = reqs <= kFewReqs;
  const int run = few ? (reqs + 31) / 32 : (reqs + kAttendThreads - 1) / kAttendThreads;
  const int lo = min(reqs, (few ? lane : t) * run), hi = min(reqs, lo + run);
  int mine = 0, mine_units = 0, longest = 0, shortest = INT_MAX;
  bool bad_length = false;
  auto take = [&](int r) {
    const int64_t length = p.lengths[r];
    const int pages = pages_of(p, length);
    mine += pages;
    mine_units += pages > 0;
    longest = max(longest, pages);
    if (pages > 0) shortest = min(shortest, pages);
    bad_length = bad_length || length < 0 || length > p.max_slots;
  };
  if (few) {
#pragma unroll
    for (int k = 0; k < kFewReqs / 32; ++k)  // all on their way at once
      if (lo + k < hi) take(lo + k);
  } else {
#pragma unroll 1
    for (int r = lo; r < hi; ++r) take(r);
  }
  if (bad_length && cta == 0) atomicCAS(p.error, 0u, kErrBadIndex);
  int before = warp_inclusive(mine, lane), before_units = warp_inclusive(mine_units, lane);
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  int total = __shfl_sync(0xFFFFFFFFu, before, 31), units = __shfl_sync(0xFFFFFFFFu, before_units, 31);
  before -= mine;
  before_units -= mine_units;
  if (!few) {
    if (lane == 0) s.scan[warp] = make_int4(total, units, longest, 0);
    __syncthreads();
    total = units = 0;
#pragma unroll 1
    for (int i = 0; i < kAttendThreads / 32; ++i) {
      const int4 of = s.scan[i];
      if (i < warp) before += of.x, before_units += of.y;
      total += of.x;
      units += of.y;
      longest = max(longest, of.z);
    }
  }
  total *= p.groups;
  units *= p.groups;
  // A unit to each CTA, if the longest takes no more than kUndivided pages over
  // an equal share: no parts, nothing to join.
  int each = longest, own = mine_units, shares = units, finder = 0;
  bool aligned = units <= grid && longest <= total / grid + kUndivided;
  if (!aligned && few && units <= grid) {
    const Shares found = aligned_shares<N>(p, s.scan, lo, hi, total, units, shortest, grid);
    aligned = found.each > 0;
    if (aligned) {
      each = found.each;
      own = found.own;
      shares = found.count;
      finder = found.finder;
      before_units = found.before;
    }
  }
  const int ctas = aligned ? shares : min(grid, max(total, 1));
  int start = 0, count = 0;
  if (cta < ctas) {
    start = aligned ? cta : share_start(total, cta, ctas);
    count = aligned ? 1 : share_start(total, cta + 1, ctas) - start;
  }
  const int first = aligned ? before_units : before, here = aligned ? own : mine;
  if (count > 0 && start >= first * p.groups && start < (first + here) * p.groups && (!few || warp == finder)) {
    int off = start - first * p.groups, r = lo;
#pragma unroll 1
    for (;; ++r) {
      const int length = p.lengths[r], pages = pages_of(p, length);
      const int of_unit = aligned ? (pages + each - 1) / each : pages, size = of_unit * p.groups;
      if (off < size) {
        s.start[0] = r;
        s.start[1] = length;
        s.start[2] = off / of_unit;
        s.start[3] = off % of_unit * (aligned ? each : 1);
        break;
      }
      off -= size;
    }
  }
  if (t == 0) {
    s.total = total;
    s.ctas = ctas;
    s.count = count;
    s.each = aligned ? each : 0;
    s.rows.heads = 0;
    p.joins[cta] = make_int4(-1, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s.count > 0) {
    Walk w;
    w.req = s.start[0];
    w.length = s.start[1];
    w.group = s.start[2];
    w.page = s.start[3];
    w.pages = pages_of(p, w.length);
    const int count = s.each > 0 ? min(s.each, w.pages - w.page) : s.count;
    w.left = count;
    if (warp < kSoftmaxWarps) {
      more_registers<kSoftmaxRegs>();
      softmax_role<N>(p, s, w);
    } else {
      fewer_registers<kOtherRegs>();
      const int worker = 3 * (warp / 4 - 1) + warp % 4;  // of those not on the issuer's scheduler
      if (warp == kIssueWarp) {
        issue_role<N>(p, s, count);
      } else if (warp == kCopyWarp) {
        copy_role<N>(p, s, w);
      } else if (warp == kQueryWarp) {
        query_role<N>(p, s, w);
      } else if (worker < kGroups) {
        decode_role<N>(p, s, worker, count);
      } else if (worker == kGroups) {
        rope_role<N>(p, s, count);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s.rows.heads > 0) write_rows<N>(p, s, s.rows, (warp >> 2) * N, (warp >> 2) * N + N);
  if (p.alone) {
#pragma unroll 1
    for (int r = cta; r < reqs; r += grid)
      if (p.lengths[r] == 0) write_empty(p, r);
  }
  if (t == 0 && s.abort) {
    atomicCAS(p.error, 0u, kErrTimeout);
    p.joins[cta] = make_int4(-2, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssueWarp) tmem_free(s.tmem, tmem_columns<N>());
}

// ---- joining kernel -----------------------------------------------------------------

// A divided unit: its parts lie in the first one's place and then in the first
// places of the shares up to the last.
struct Division {
  int first, last;  // first part, last CTA
  __device__ int count() const { return last - (first >> 1) + 1; }
  __device__ int part(int j) const { return j == 0 ? first : 2 * ((first >> 1) + j); }
};

// One head of a divided unit: 4 dims a thread of those at `t`, the sum of parts
// `from`, `from` + `step`, ...  Every warp forms the parts' weights for itself,
// in `w`.  Returns the sum; `scale` and `lse` are what finishes it.
__device__ __forceinline__ float4 join_parts(const AttendParams& p, int n, const Division& d, int col, int head, int t,
                                             int from, int step, float* w, float* scale, float* lse, bool* bad) {
  const int lane = threadIdx.x & 31, count = d.count();
  const float4* const parts = reinterpret_cast<const float4*>(p.parts) + col * (kHeadDim / 4) + t;
  const int64_t apart = static_cast<int64_t>(n) * (kHeadDim / 4);
  const float sink = p.sinks == nullptr ? -INFINITY : p.sinks[head] * kLog2e;
  float2 ml[kStatsPerLane];  // all at once: one latency, not one for each
  int any = 0;
#pragma unroll
  for (int k = 0; k < kStatsPerLane; ++k) {
    const int j = lane + 32 * k;
    ml[k] = make_float2(-FLT_MAX, 0.f);
    if (j < count) {
      ml[k] = p.part_stats[d.part(j) * n + col];
      any |= p.part_bad[d.part(j)];
    }
  }
  float top = sink, total = 0.f;
#pragma unroll
  for (int k = 0; k < kStatsPerLane; ++k) top = fmaxf(top, ml[k].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
#pragma unroll
  for (int k = 0; k < kStatsPerLane; ++k) {
    if (32 * k >= count) break;
    const float f = exp2_fast(ml[k].x - top);
    total += ml[k].y * f;
    w[lane + 32 * k] = f;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (p.sinks != nullptr) total += exp2_fast(sink - top);
  *bad = __any_sync(0xFFFFFFFFu, any != 0);
  *scale = total == 0.f ? 0.f : 1.f / total;
  *lse = total == 0.f ? -INFINITY : (top + log2f(total)) / kLog2e;
  __syncwarp();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = from; j < count; j += step) {
    const float f = w[j];
    const float4 o = parts[d.part(j) * apart];
    acc.x += f * o.x;
    acc.y += f * o.y;
    acc.z += f * o.z;
    acc.w += f * o.w;
  }
  __syncwarp();  // w is free again
  return acc;
}

// What the weights of one head of a divided unit are formed with, by `with`
// threads of a warp: the reference (log2) and 1 / sum, 0 where there is no key.
__device__ __forceinline__ float2 unit_stats(const AttendParams& p, int n, const Division& d, int col, int head,
                                             int first, int with, int* skip) {
  const uint32_t who = 0xFFFFFFFFu >> (32 - with) << (threadIdx.x & 31 & ~(with - 1));
  float top = p.sinks == nullptr ? -FLT_MAX : fmaxf(p.sinks[head] * kLog2e, -FLT_MAX);
  float total = p.sinks == nullptr || first != 0 ? 0.f : exp2_fast(p.sinks[head] * kLog2e - top);
  const int count = d.count();
  int any = 0;
#pragma unroll 8
  for (int j = first; j < count; j += with) {
    const float2 ml = p.part_stats[d.part(j) * n + col];
    any |= p.part_bad[d.part(j)];
    const float next = fmaxf(top, ml.x);
    total = total * exp2_fast(top - next) + ml.y * exp2_fast(ml.x - next);
    top = next;
  }
  for (int o = with / 2; o > 0; o >>= 1) {
    const float other = __shfl_xor_sync(who, top, o), sum = __shfl_xor_sync(who, total, o), next = fmaxf(top, other);
    total = total * exp2_fast(top - next) + sum * exp2_fast(other - next);
    top = next;
  }
  if (any) *skip = 1;
  return make_float2(top, total == 0.f ? 0.f : 1.f / total);
}

__device__ __forceinline__ void store_joined(const AttendParams& p, int64_t row, int t, float4 v, float f, float lse) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * f, v.w * f);
  reinterpret_cast<uint2*>(p.out + row * kHeadDim)[t] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (t == 0) p.lse[row] = lse;
}

// Joins the divided units, zeroes the rows without slots, forms the weights.
// An item is a head of a divided unit, 128 threads' work if that fills the grid.
// Else it is a CTA's, whose four groups of 128 take a quarter of the parts each,
// or, where that leaves CTAs without work, 2 or 4 CTAs', each for a part of the
// dims and with as many more groups.
__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm) kvc_attend_join_kernel(const __grid_constant__ AttendParams p,
                                                                        int n, int ctas, int weight_ctas) {
  __shared__ int4 joins[kAttendCtas];
  __shared__ int warp_joins[kJoinThreads / 32];
  __shared__ float4 sums[kJoinThreads];
  __shared__ float part_weights[kJoinThreads / 32][32 * kStatsPerLane];
  __shared__ __align__(16) float tops[2 * 64], shares[2 * 64];
  __shared__ int skip;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  // the divided units, in order
  const int4 mine = t < ctas ? p.joins[t] : make_int4(-1, 0, 0, 0);
  // what a CTA that gave up has not written is not read
  if (__syncthreads_or(mine.x == -2)) return;
  const uint32_t there = __ballot_sync(0xFFFFFFFFu, mine.x >= 0);
  if (lane == 0) warp_joins[warp] = __popc(there);
  __syncthreads();
  int before = __popc(there & ((1u << lane) - 1)), divided = 0;
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < warp) before += warp_joins[i];
    divided += warp_joins[i];
  }
  if (mine.x >= 0) joins[before] = mine;
  __syncthreads();
  const int heads = divided * p.group_heads, grid = static_cast<int>(gridDim.x);
  const bool apart = heads >= 2 * grid;  // a head to each 128 threads
  const int cuts = 4 * heads <= grid ? 4 : 2 * heads <= grid ? 2 : 1, size = 128 / cuts;
  const int group = t / size, groups = kJoinThreads / size, items = heads * cuts;
  for (int item = apart ? 4 * static_cast<int>(blockIdx.x) + group : static_cast<int>(blockIdx.x); item < items;
       item += apart ? 4 * grid : grid) {
    const int unit = item / cuts, at = item % cuts * size + t % size;
    const int4 join = joins[unit / p.group_heads];
    const int col = unit % p.group_heads, head = join.y * p.group_heads + col;
    if (head >= p.num_heads) continue;
    float f, lse;
    bool bad;
    float4 v = join_parts(p, n, Division{join.z, join.w}, col, head, at, apart ? 0 : group, apart ? 1 : groups,
                          part_weights[warp], &f, &lse, &bad);
    if (!apart) {
      sums[t] = v;
      __syncthreads();
      if (group == 0) {
        for (int g = 1; g < groups; ++g) {
          const float4 o = sums[g * size + t];
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
      }
      __syncthreads();
    }
    if (!bad && (apart || group == 0))
      store_joined(p, static_cast<int64_t>(join.x) * p.num_heads + head, at, v, f, lse);
  }
  // requests: `weight_ctas` CTAs for each
  for (int item = blockIdx.x; item < p.num_reqs * weight_ctas; item += grid) {
    const int r = item / weight_ctas, sub = item % weight_ctas;
    const int64_t length = p.lengths[r];
    if (length < 0 || length > p.max_slots) continue;
    if (length == 0) {
      if (sub != 0) continue;
      write_empty(p, r);
      continue;
    }
    if (p.weights_out == nullptr || length * sub / weight_ctas == length * (sub + 1) / weight_ctas) continue;
    // The heads' references and 1 / sums, by column of the scores: 0 where there is
    // no head or no key.  (Not the log of the sum in their place: it is a number
    // of the scores' size, and what its rounding loses would be a factor of every
    // weight, 2 % at scores of 1e5.)
    if (t == 0) skip = 0;
    __syncthreads();
    {
      // a column to each kJoinThreads / score_cols threads (4 .. 32), which share its parts
      const int with = kJoinThreads / static_cast<int>(p.score_cols), col = t / with, first = t % with;
      const int unit = col / n, c = col % n, head = unit * p.group_heads + c;
      float2 v = make_float2(0.f, 0.f);
      if (c < p.group_heads && head < p.num_heads) {
        const int2 parts = p.unit_parts[static_cast<int64_t>(r) * p.groups + unit];
        if (parts.x < 0) {
          if (parts.y) skip = 1;
          v = p.row_stats[static_cast<int64_t>(r) * p.num_heads + head];
        } else {
          v = unit_stats(p, n, Division{parts.x, parts.y}, c, head, first, with, &skip);
        }
      }
      if (first == 0) {
        tops[col] = v.x;
        shares[col] = v.y;
      }
    }
    __syncthreads();
    if (!skip) {
      // 4 columns a thread, `lanes` threads a slot
      const int lanes = static_cast<int>(p.score_cols) / 4, step = kJoinThreads / lanes;
      const float4 m = *reinterpret_cast<const float4*>(tops + 4 * (t % lanes));
      const float4 f = *reinterpret_cast<const float4*>(shares + 4 * (t % lanes));
      const float* const weights_in = p.weights_in == nullptr ? nullptr : p.weights_in + r * p.weights_in_row_stride;
      float* const weights_out = p.weights_out + r * p.weights_out_row_stride;
      const float4* const scores =
          reinterpret_cast<const float4*>(p.scores + r * p.max_pages * kSlotsPerPage * p.score_cols) + t % lanes;
      const int begin = static_cast<int>(length * sub / weight_ctas), end = static_cast<int>(length * (sub + 1) / weight_ctas);
#pragma unroll 4
      for (int slot = begin + t / lanes; slot < end + t / lanes; slot += step) {  // a warp stays together
        float sum = 0.f, old = 0.f;
        if (slot < end) {
          const float4 x = scores[static_cast<int64_t>(slot) * lanes];
          if (weights_in != nullptr) old = weights_in[slot];
          sum = (f.x == 0.f ? 0.f : exp2_fast(x.x - m.x) * f.x) + (f.y == 0.f ? 0.f : exp2_fast(x.y - m.y) * f.y) +
                (f.z == 0.f ? 0.f : exp2_fast(x.z - m.z) * f.z) + (f.w == 0.f ? 0.f : exp2_fast(x.w - m.w) * f.w);
        }
        for (int d = lanes / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (slot < end && t % lanes == 0) weights_out[slot] = old + sum;
      }
    }
    __syncthreads();  // tops, shares and skip are free again
  }
}

template <int N>
cudaError_t launch_n(const AttendParams& p, int ctas, cudaStream_t stream) {
  constexpr size_t smem = sizeof(AttendShared<N>);
  static_assert(smem <= 232448, "227 KB a CTA");
  cudaError_t e = cudaFuncSetAttribute(kvc_attend_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kAttendThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kvc_attend_kernel<N>, p);
  if (e != cudaSuccess || p.alone) return e;
  // as many as fit at once: they share the divided units' heads, then the requests,
  // one turn each (24 requests of up to 2050 slots, 32 heads: 22.6 us, in two turns 3 more)
  constexpr int kMost = kJoinCtasPerSm * kAttendCtas;
  const int64_t chunks = p.weights_out == nullptr ? 1 : (p.max_slots + kSlotsPerPage - 1) / kSlotsPerPage;
  int64_t weight_ctas = kMost / p.num_reqs;
  weight_ctas = weight_ctas > chunks ? chunks : weight_ctas;
  weight_ctas = weight_ctas < 1 ? 1 : weight_ctas;
  const int64_t joins = 4 * static_cast<int64_t>(ctas) * p.group_heads, items = p.num_reqs * weight_ctas;
  const int64_t work = joins > items ? joins : items;
  cfg.gridDim = dim3(static_cast<unsigned>(work < kMost ? work : kMost));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kvc_attend_join_kernel, p, N, ctas, static_cast<int>(weight_ctas));
}

}  // namespace

AttendShape attend_shape(int num_heads) {
  AttendShape s;
  s.groups = (num_heads + 63) / 64;
  s.group_heads = (num_heads + s.groups - 1) / s.groups;
  s.columns = s.group_heads <= 16 ? 16 : s.group_heads <= 32 ? 32 : 64;
  return s;
}

bool attend_alone(const AttendParams& p, int ctas) {
  return p.weights_out == nullptr && p.max_pages <= kUndivided && p.num_reqs * p.groups <= ctas;
}

cudaError_t launch_attend(const AttendParams& p, int columns, int ctas, cudaStream_t stream) {
  switch (columns) {
    case 16: return launch_n<16>(p, ctas, stream);
    case 32: return launch_n<32>(p, ctas, stream);
    default: return launch_n<64>(p, ctas, stream);
  }
}

}  // namespace kvc
