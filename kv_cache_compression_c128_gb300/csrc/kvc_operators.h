// Internal interface between the C entry points of the operators on packed
// slots (kvc_operators.cu: store, dequantize, attend, join, evict, rotate) and
// their kernels.  Not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "kvc_internal.h"

namespace kvc {

constexpr int kMaxHeads = 128;
constexpr int kMaxParts = 8;

// The two forms of a packed slot (include/kvc.h, KVC_FORMAT_*): 448 codes and 64
// bf16 words, kStride bytes, and a record of kScales scale bytes behind the
// page's slots.  kCodes: bytes of the codes, behind which the RoPE words lie.
struct Slots8 {
  static constexpr bool kFour = false;
  static constexpr int kStride = kTokenStride, kScales = kScaleDim, kCodes = kNopeDim;
  static constexpr int kScaleBase = kvc::kScaleBase;
  static constexpr int64_t kPage = kPageBytes;
};
struct Slots4 {
  static constexpr bool kFour = true;
  static constexpr int kGroup = 32;  // codes with one scale
  static constexpr int kStride = kNopeDim / 2 + 2 * kRopeDim, kScales = 16, kCodes = kNopeDim / 2;
  static constexpr int kScaleBase = kSlotsPerPage * kStride;
  static constexpr int64_t kPage = kSlotsPerPage * (kStride + kScales);
};

// The 4-bit slot's scale (1 + m / 8) 2^(e - 16), its byte 8 e + m: as bits of
// bf16 the byte lies 4 places up, and the exponent's bias 127 - 16 is added.
constexpr uint32_t kScale4Bits = (127 - 16) << 7;

// Angles of the rotated dims: pair i of row t goes by the row positions[t, axis(i)]
// of the cos / sin table.
constexpr int kPairs = kRopeDim / 2, kMaxAxes = 4;
struct Rotation {
  const int64_t* positions;  // null: no rotation
  int64_t row_stride, axis_stride;
  uint64_t axes;             // 2 bits for each pair
  const float* table;        // [num_positions, 64]: cos, then sin
  int64_t num_positions;
};

struct StoreParams {
  const void* x;  // [num_rows, 512] at its row stride
  int64_t x_row_stride;
  int x_f32;
  int64_t num_rows;
  uint8_t* kv_cache;
  int64_t num_pages;
  const int64_t* slots;
  Rotation rotation;
  uint32_t* error;
};

struct RotateParams {
  const void* x;  // [num_tokens, num_heads, 64] at its strides (elements)
  int64_t x_token_stride, x_head_stride;
  int f32;
  int64_t num_tokens;
  int num_heads;
  Rotation rotation;
  int inverse;
  void* out;
  int64_t out_token_stride, out_head_stride;
  uint32_t* error;
};

struct AttendParams {
  CUtensorMap q_map;     // bf16 [num_reqs][num_heads][512], boxes of `columns` heads x 64 dims
  CUtensorMap code_map;  // bytes [num_pages][64][kStride], boxes of 64 slots x 64 codes
  int q_shared;          // every request has the queries of request 0
  int64_t num_reqs;
  int num_heads;
  const uint8_t* kv_cache;
  int four_bits;  // the pages hold Slots4
  int64_t num_pages;
  const int32_t* page_table;
  int64_t max_pages, page_table_row_stride;
  const int32_t* lengths;
  int64_t max_slots;  // a longer request is a bad index
  float scale;
  const float* sinks;  // [num_heads] or null
  uint16_t* out;       // bf16 [num_reqs, num_heads, 512]
  float* lse;          // [num_reqs, num_heads]
  const float* weights_in;  // null: zeros
  float* weights_out;       // null: not wanted
  int64_t weights_in_row_stride, weights_out_row_stride;
  int alone;                // no second kernel follows (attend_alone)
  int groups, group_heads;  // head groups of a request (AttendShape)
  // workspace
  float* scores;         // [num_reqs, max_pages * 64, score_cols] log2 scores, or null
  int64_t score_cols;    // groups * columns
  float* parts;          // [2 * ctas][columns][512]: what divided units summed up
  float2* part_stats;    // [2 * ctas][columns]: their reference (log2) and sum
  int32_t* part_bad;     // [2 * ctas]: a page was outside the cache
  int2* unit_parts;      // [num_reqs * groups]: first part and last CTA; (-1, bad) if whole
  float2* row_stats;     // [num_reqs, num_heads] of undivided units, for the weights: reference (log2) and
                         // 1 / sum (0: no key), or null
  int4* joins;           // [ctas]: (request, group, first part, pages of all units) of a unit whose last
                         // CTA this is, or (-1, ...); (-2, ...) if it gave up
  long long wait_limit;
  uint32_t* error;
};

// How the heads of a request are laid out: `groups` runs of `group_heads`
// (the last may be shorter), each padded to `columns` of a product.
struct AttendShape {
  int groups, group_heads, columns;
};
AttendShape attend_shape(int num_heads);

// CTAs at most (GB300 has 152 SMs); the workspace holds two parts for each.
constexpr int kAttendCtas = 152;

struct JoinParams {
  const void* outs[kMaxParts];
  const float* lses[kMaxParts];
  int num_parts;
  int64_t num_rows;
  int bf16;
  void* out;
  float* lse;  // null: not wanted
};

struct EvictParams {
  uint8_t* kv_cache;
  int four_bits;  // the pages hold Slots4
  int64_t num_pages;
  const int32_t* page_table;
  int64_t num_reqs, page_table_row_stride;
  const int32_t* lengths;
  int64_t max_slots;  // a longer request is a bad index
  const float* weights;
  int64_t weights_row_stride;
  const int32_t* births;  // null: none
  int64_t births_row_stride;
  int64_t keep, recent;
  int32_t* lengths_out;
  int32_t* kept;  // [num_reqs, keep] or null
  float* weights_out;
  int64_t weights_out_row_stride;
  int32_t* births_out;
  int64_t births_out_row_stride;
  int32_t* counts;  // workspace: moves of each request
  longlong2* moves; // workspace: per request, move_stride slots of the cache (to, of)
  int64_t move_stride;
  uint32_t* error;
};

// Whether no lengths at all can leave anything to the joining kernel: there are
// CTAs for all units, none long enough to be divided, and no weights to form.
// (One request of 64 slots, 64 heads: 8.0 us, 8 of 128: 8.9.  With both kernels, before other
// steps that shortened either way, 10.7 instead of 9.1, and 11.3 instead of 9.9.)
bool attend_alone(const AttendParams& p, int ctas);
cudaError_t launch_attend(const AttendParams& p, int columns, int ctas, cudaStream_t stream);
cudaError_t launch_join(const JoinParams& p, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);
cudaError_t launch_store(const StoreParams& p, bool four_bits, cudaStream_t stream);
cudaError_t launch_dequantize4(const uint8_t* kv, int64_t num_pages, const int64_t* slots, int64_t num_slots, void* out,
                               int out_bf16, uint32_t* err, cudaStream_t stream);
cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream);

// The current device's set-up (kvc_api.cu): its SM count, the address of its
// error word, and the limit on a kernel's pipeline waits.
kvc_status operator_device(int* sms, uint32_t** error_word, long long* wait_limit);

}  // namespace kvc
