// Internal interface between the C entry points of the operators on packed
// slots (kvc_operators.cu: attend, join, evict) and their kernels.  Not part
// of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "kvc_internal.h"

namespace kvc {

constexpr int kMaxHeads = 128;
constexpr int kMaxParts = 8;

struct AttendParams {
  CUtensorMap q_map;     // bf16 [num_reqs][num_heads][512], boxes of `columns` heads x 64 dims
  CUtensorMap code_map;  // bytes [num_pages][64][576], boxes of 64 slots x 64 bytes
  int q_shared;          // every request has the queries of request 0
  int64_t num_reqs;
  int num_heads;
  const uint8_t* kv_cache;
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
  int4* joins;           // [ctas]: (request, group, first part, last CTA) to join, or (-1, ...)
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
// (One request of 64 slots, 64 heads: 9.1 us, with both kernels 10.7; 8 of 128: 9.9, 11.3.)
bool attend_alone(const AttendParams& p, int ctas);
cudaError_t launch_attend(const AttendParams& p, int columns, int ctas, cudaStream_t stream);
cudaError_t launch_join(const JoinParams& p, cudaStream_t stream);
cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

// The current device's set-up (kvc_api.cu): its SM count, the address of its
// error word, and the limit on a kernel's pipeline waits.
kvc_status operator_device(int* sms, uint32_t** error_word, long long* wait_limit);

}  // namespace kvc
