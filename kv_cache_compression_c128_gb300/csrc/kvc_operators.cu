// C entry points of the operators on packed slots (declared in
// include/kvc.h): argument validation and workspace sizing for kvc_store
// (kvc_store.cu), kvc_dequantize_format (kvc_reader.cu, kvc_store.cu), kvc_attend
// (kvc_attend.cu), kvc_join (kvc_join.cu), kvc_evict (kvc_evict.cu) and
// kvc_rotate (kvc_rotate.cu).

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kvc.h"
#include "kvc_internal.h"
#include "kvc_operators.h"
#include "kvc_overlap.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxRequests = 65535;
constexpr int64_t kMaxSlots = int64_t{1} << 30;  // slot indices of a request fit int32
constexpr int64_t kMaxRows = int64_t{1} << 32;   // of store, dequantize and rotate
constexpr int32_t kMaxTurnedHeads = 65535;

// Sizes every operator on pages checks alike.
bool pages_ok(const void* kv_cache, int64_t num_kv_pages, const int32_t* page_table,
              int64_t num_reqs, int64_t max_pages, int64_t row_stride, const int32_t* lengths) {
  return kv_cache != nullptr && page_table != nullptr && lengths != nullptr && num_kv_pages > 0 &&
         num_kv_pages <= INT32_MAX && num_reqs > 0 && num_reqs <= kMaxRequests && max_pages > 0 &&
         max_pages <= kMaxSlots / kvc::kSlotsPerPage && row_stride >= 0 && aligned(kv_cache, 16) &&
         aligned(page_table, 4) && aligned(lengths, 4);
}

// Rows that are written do not overlap.
bool rows_apart(int64_t num_reqs, int64_t row_stride, int64_t columns) {
  return num_reqs <= 1 || row_stride >= columns;
}

bool format_ok(int32_t format) { return format == KVC_FORMAT_8BIT || format == KVC_FORMAT_4BIT; }

// Positions, axes and table of a rotation, as every operator that turns takes them
// (no positions for no rows).
bool rotation_ok(int64_t rows, const int64_t* positions, int64_t row_stride, int64_t axis_stride, int32_t num_axes,
                 const uint8_t* pair_axes, const float* table, int64_t num_positions, kvc::Rotation* r) {
  if (num_axes < 1 || num_axes > kvc::kMaxAxes || (rows != 0 && positions == nullptr) || table == nullptr || num_positions < 1 ||
      row_stride < 0 || axis_stride < 0 || !aligned(positions, 8) || !aligned(table, 16) ||
      (pair_axes == nullptr && num_axes > 1))
    return false;
  r->axes = 0;
  for (int i = 0; pair_axes != nullptr && i < kvc::kPairs; ++i) {
    if (pair_axes[i] >= num_axes) return false;
    r->axes |= static_cast<uint64_t>(pair_axes[i]) << (2 * i);
  }
  r->positions = positions;
  r->row_stride = row_stride;
  r->axis_stride = axis_stride;
  r->table = table;
  r->num_positions = num_positions;
  return true;
}

// Rows of 64 elements at two strides that are written do not overlap.
bool heads_apart(int64_t tokens, int64_t token_stride, int64_t heads, int64_t head_stride) {
  if (tokens <= 1) return heads <= 1 || head_stride >= kvc::kRopeDim;
  if (heads <= 1) return token_stride >= kvc::kRopeDim;
  return head_stride < token_stride
             ? head_stride >= kvc::kRopeDim && token_stride / head_stride >= heads - 1 &&
                   token_stride - head_stride * (heads - 1) >= kvc::kRopeDim
             : token_stride >= kvc::kRopeDim && head_stride / token_stride >= tokens - 1 &&
                   head_stride - token_stride * (tokens - 1) >= kvc::kRopeDim;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

// Byte offsets in an attention's workspace.
struct AttendWorkspace {
  size_t parts, stats, bad, units, joins, lse, rows, scores, total;
};

AttendWorkspace attend_workspace(int64_t num_reqs, int num_heads, int64_t max_pages, bool scores) {
  const kvc::AttendShape shape = kvc::attend_shape(num_heads);
  const size_t columns = 2 * static_cast<size_t>(kvc::kAttendCtas) * shape.columns;
  AttendWorkspace w;
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t here = at;
    at += round16(bytes);
    return here;
  };
  w.parts = take(columns * kvc::kHeadDim * sizeof(float));
  w.stats = take(columns * sizeof(float2));
  w.bad = take(2 * kvc::kAttendCtas * sizeof(int32_t));
  w.units = take(num_reqs * shape.groups * sizeof(int2));
  w.joins = take(kvc::kAttendCtas * sizeof(int4));
  w.lse = take(num_reqs * num_heads * sizeof(float));
  w.rows = take(scores ? num_reqs * num_heads * sizeof(float2) : 0);
  w.scores = take(scores ? static_cast<size_t>(num_reqs) * max_pages * kvc::kSlotsPerPage * shape.groups *
                               shape.columns * sizeof(float)
                         : 0);
  w.total = at;
  return w;
}

}  // namespace

extern "C" {

size_t kvc_attend_workspace_bytes(int64_t num_reqs, int32_t num_heads, int64_t max_pages_per_req,
                                  int32_t with_slot_weights) {
  if (num_reqs < 0 || num_reqs > kMaxRequests || num_heads < 1 || num_heads > kvc::kMaxHeads ||
      max_pages_per_req < 0 || max_pages_per_req > kMaxSlots / kvc::kSlotsPerPage)
    return 0;
  return attend_workspace(num_reqs, num_heads, max_pages_per_req, with_slot_weights != 0).total;
}

kvc_status kvc_attend(const void* q, int64_t q_req_stride, int64_t q_head_stride, int64_t num_reqs,
                      int32_t num_heads, const uint8_t* kv_cache, int64_t num_kv_pages,
                      const int32_t* page_table, int64_t max_pages_per_req,
                      int64_t page_table_row_stride, const int32_t* lengths, float scale,
                      const float* sinks, void* out, float* lse, const float* slot_weights_in,
                      int64_t slot_weights_in_row_stride, float* slot_weights,
                      int64_t slot_weights_row_stride, int64_t max_slots, void* workspace,
                      size_t workspace_bytes, uint32_t flags, void* stream) {
  return kvc_attend_format(q, q_req_stride, q_head_stride, num_reqs, num_heads, kv_cache, KVC_FORMAT_8BIT,
                           num_kv_pages, page_table, max_pages_per_req, page_table_row_stride, lengths, scale,
                           sinks, out, lse, slot_weights_in, slot_weights_in_row_stride, slot_weights,
                           slot_weights_row_stride, max_slots, workspace, workspace_bytes, flags, stream);
}

kvc_status kvc_attend_format(const void* q, int64_t q_req_stride, int64_t q_head_stride, int64_t num_reqs,
                             int32_t num_heads, const uint8_t* kv_cache, int32_t kv_format,
                             int64_t num_kv_pages, const int32_t* page_table, int64_t max_pages_per_req,
                             int64_t page_table_row_stride, const int32_t* lengths, float scale,
                             const float* sinks, void* out, float* lse, const float* slot_weights_in,
                             int64_t slot_weights_in_row_stride, float* slot_weights,
                             int64_t slot_weights_row_stride, int64_t max_slots, void* workspace,
                             size_t workspace_bytes, uint32_t flags, void* stream) {
  // (the kernel works in powers of two: scale times log2(e) is finite too)
  if (num_reqs < 0 || num_heads < 1 || num_heads > kvc::kMaxHeads || !format_ok(kv_format) ||
      !std::isfinite(scale * 1.44269504f) || (flags & ~KVC_FLAG_GRID_MASK) != 0)
    return KVC_ERR_INVALID_ARG;
  if (num_reqs == 0) return KVC_OK;
  if (!pages_ok(kv_cache, num_kv_pages, page_table, num_reqs, max_pages_per_req,
                page_table_row_stride, lengths))
    return KVC_ERR_INVALID_ARG;
  if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16) ||
      q_req_stride % 8 != 0 || q_head_stride % 8 != 0 || q_req_stride < 0 || q_head_stride < 0 ||
      (q_head_stride == 0 && num_heads > 1) ||
      !aligned(sinks, 4) || !aligned(lse, 4))
    return KVC_ERR_INVALID_ARG;
  if (slot_weights == nullptr && slot_weights_in != nullptr) return KVC_ERR_INVALID_ARG;
  if (slot_weights != nullptr &&
      (max_slots < 0 || slot_weights_row_stride < 0 || slot_weights_in_row_stride < 0 ||
       !aligned(slot_weights, 4) || !aligned(slot_weights_in, 4) ||
       !rows_apart(num_reqs, slot_weights_row_stride, max_slots)))
    return KVC_ERR_INVALID_ARG;
  const size_t need = kvc_attend_workspace_bytes(num_reqs, num_heads, max_pages_per_req,
                                                 slot_weights != nullptr);
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)
    return KVC_ERR_INVALID_ARG;
  // pages are counted in 31 bits, over all requests and head groups
  if (num_reqs * max_pages_per_req * kvc::attend_shape(num_heads).groups > INT32_MAX) return KVC_ERR_UNSUPPORTED;
  int sms = 0;
  kvc::AttendParams p = {};
  const kvc_status st = kvc::operator_device(&sms, &p.error, &p.wait_limit);
  if (st != KVC_OK) return st;
  const kvc::AttendShape shape = kvc::attend_shape(num_heads);
  {
    // a dimension of one entry has no stride, and one of stride 0 has one entry
    p.q_shared = q_req_stride == 0;
    const cuuint64_t head_bytes = num_heads == 1 ? 1024 : 2 * static_cast<cuuint64_t>(q_head_stride);
    const cuuint64_t reqs = p.q_shared ? 1 : num_reqs;
    const cuuint64_t req_bytes = reqs == 1 ? head_bytes * num_heads : 2 * static_cast<cuuint64_t>(q_req_stride);
    const cuuint64_t q_dims[3] = {kvc::kHeadDim, static_cast<cuuint64_t>(num_heads), reqs};
    const cuuint64_t q_strides[2] = {head_bytes, req_bytes};
    const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(shape.columns), 1};
    const bool four = kv_format == KVC_FORMAT_4BIT;
    const cuuint64_t stride = four ? kvc::Slots4::kStride : kvc::Slots8::kStride;
    const cuuint64_t page_dims[3] = {stride, kvc::kSlotsPerPage, static_cast<cuuint64_t>(num_kv_pages)};
    const cuuint64_t page_strides[2] = {stride, static_cast<cuuint64_t>(four ? kvc::Slots4::kPage : kvc::Slots8::kPage)};
    const cuuint32_t code_box[3] = {static_cast<cuuint32_t>(four ? kvc::kGroup / 2 : kvc::kGroup), kvc::kSlotsPerPage, 1};
    if (!kvc::encode_tensor_map(&p.q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, q_dims, q_strides, q_box,
                                CU_TENSOR_MAP_SWIZZLE_128B))
      return KVC_ERR_UNSUPPORTED;
    if (!kvc::encode_tensor_map(&p.code_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, kv_cache, page_dims, page_strides,
                                code_box, CU_TENSOR_MAP_SWIZZLE_NONE))
      return KVC_ERR_CUDA;
  }
  p.num_reqs = num_reqs;
  p.num_heads = num_heads;
  p.kv_cache = kv_cache;
  p.four_bits = kv_format == KVC_FORMAT_4BIT;
  p.num_pages = num_kv_pages;
  p.page_table = page_table;
  p.max_pages = max_pages_per_req;
  p.page_table_row_stride = page_table_row_stride;
  p.lengths = lengths;
  p.max_slots = max_pages_per_req * kvc::kSlotsPerPage;
  if (slot_weights != nullptr && max_slots < p.max_slots) p.max_slots = max_slots;
  p.scale = scale;
  p.sinks = sinks;
  p.out = static_cast<uint16_t*>(out);
  const AttendWorkspace at = attend_workspace(num_reqs, num_heads, max_pages_per_req, slot_weights != nullptr);
  uint8_t* const base = static_cast<uint8_t*>(workspace);
  p.lse = lse != nullptr ? lse : reinterpret_cast<float*>(base + at.lse);
  p.parts = reinterpret_cast<float*>(base + at.parts);
  p.part_stats = reinterpret_cast<float2*>(base + at.stats);
  p.part_bad = reinterpret_cast<int32_t*>(base + at.bad);
  p.unit_parts = reinterpret_cast<int2*>(base + at.units);
  p.joins = reinterpret_cast<int4*>(base + at.joins);
  p.weights_in = slot_weights_in;
  p.weights_out = slot_weights;
  p.weights_in_row_stride = slot_weights_in_row_stride;
  p.weights_out_row_stride = slot_weights_row_stride;
  p.groups = shape.groups;
  p.group_heads = shape.group_heads;
  p.score_cols = static_cast<int64_t>(shape.groups) * shape.columns;
  if (slot_weights != nullptr) {
    p.scores = reinterpret_cast<float*>(base + at.scores);
    p.row_stats = reinterpret_cast<float2*>(base + at.rows);
  }
  // one CTA per SM, fewer where the table cannot name a page for each
  int64_t ctas = sms < kvc::kAttendCtas ? sms : kvc::kAttendCtas;
  if (num_reqs * max_pages_per_req * shape.groups < ctas) ctas = num_reqs * max_pages_per_req * shape.groups;
  if ((flags & KVC_FLAG_GRID_MASK) != 0 && (flags & KVC_FLAG_GRID_MASK) < ctas) ctas = flags & KVC_FLAG_GRID_MASK;
  p.alone = kvc::attend_alone(p, static_cast<int>(ctas));
  const cudaError_t e =
      kvc::launch_attend(p, shape.columns, static_cast<int>(ctas), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc_status kvc_join(const void* const* outs, const float* const* lses, int32_t num_parts,
                    int64_t num_rows, int32_t dtype, void* out, float* lse, void* stream) {
  if (num_parts < 1 || num_parts > kvc::kMaxParts || num_rows < 0 ||
      num_rows > (int64_t{1} << 32) || (dtype != KVC_DTYPE_F32 && dtype != KVC_DTYPE_BF16))
    return KVC_ERR_INVALID_ARG;
  if (num_rows == 0) return KVC_OK;
  if (outs == nullptr || lses == nullptr || out == nullptr || !aligned(out, 16) || !aligned(lse, 4))
    return KVC_ERR_INVALID_ARG;
  kvc::JoinParams p = {};
  for (int i = 0; i < num_parts; ++i) {
    if (outs[i] == nullptr || lses[i] == nullptr || !aligned(outs[i], 16) || !aligned(lses[i], 4))
      return KVC_ERR_INVALID_ARG;
    p.outs[i] = outs[i];
    p.lses[i] = lses[i];
  }
  p.num_parts = num_parts;
  p.num_rows = num_rows;
  p.bf16 = dtype == KVC_DTYPE_BF16;
  p.out = out;
  p.lse = lse;
  const cudaError_t e = kvc::launch_join(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

size_t kvc_evict_workspace_bytes(int64_t num_reqs, int64_t max_pages_per_req, int64_t keep) {
  if (num_reqs < 0 || num_reqs > kMaxRequests || max_pages_per_req < 0 ||
      max_pages_per_req > kMaxSlots / kvc::kSlotsPerPage || keep < 0 || keep > kMaxSlots)
    return 0;
  // as many moves as slots can lie behind `keep`, or before it
  const int64_t slots = max_pages_per_req * kvc::kSlotsPerPage;
  const int64_t behind = slots > keep ? slots - keep : 0;
  const int64_t stride = behind < keep ? behind : keep;
  return round16(sizeof(int32_t) * num_reqs) + sizeof(longlong2) * num_reqs * stride + 16;
}

kvc_status kvc_evict(uint8_t* kv_cache, int64_t num_kv_pages, const int32_t* page_table,
                     int64_t num_reqs, int64_t max_pages_per_req, int64_t page_table_row_stride,
                     const int32_t* lengths, const float* slot_weights,
                     int64_t slot_weights_row_stride, int64_t max_slots, const int32_t* births,
                     int64_t births_row_stride, int64_t keep, int64_t recent, int32_t* lengths_out,
                     int32_t* kept, float* slot_weights_out, int64_t slot_weights_out_row_stride,
                     int32_t* births_out, int64_t births_out_row_stride, void* workspace,
                     size_t workspace_bytes, void* stream) {
  return kvc_evict_format(kv_cache, KVC_FORMAT_8BIT, num_kv_pages, page_table, num_reqs, max_pages_per_req,
                          page_table_row_stride, lengths, slot_weights, slot_weights_row_stride, max_slots,
                          births, births_row_stride, keep, recent, lengths_out, kept, slot_weights_out,
                          slot_weights_out_row_stride, births_out, births_out_row_stride, workspace,
                          workspace_bytes, stream);
}

kvc_status kvc_evict_format(uint8_t* kv_cache, int32_t kv_format, int64_t num_kv_pages,
                            const int32_t* page_table, int64_t num_reqs, int64_t max_pages_per_req,
                            int64_t page_table_row_stride, const int32_t* lengths,
                            const float* slot_weights, int64_t slot_weights_row_stride,
                            int64_t max_slots, const int32_t* births, int64_t births_row_stride,
                            int64_t keep, int64_t recent, int32_t* lengths_out, int32_t* kept,
                            float* slot_weights_out, int64_t slot_weights_out_row_stride,
                            int32_t* births_out, int64_t births_out_row_stride, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!format_ok(kv_format) || num_reqs < 0 || keep < 0 || keep > kMaxSlots || recent < 0 || recent > keep ||
      (recent > 0 && births == nullptr) || (births_out != nullptr && births == nullptr))
    return KVC_ERR_INVALID_ARG;
  if (num_reqs == 0) return KVC_OK;
  if (!pages_ok(kv_cache, num_kv_pages, page_table, num_reqs, max_pages_per_req,
                page_table_row_stride, lengths))
    return KVC_ERR_INVALID_ARG;
  if (slot_weights == nullptr || lengths_out == nullptr || max_slots < 0 ||
      slot_weights_row_stride < 0 || births_row_stride < 0 || slot_weights_out_row_stride < 0 ||
      births_out_row_stride < 0 || !aligned(slot_weights, 4) || !aligned(births, 4) ||
      !aligned(lengths_out, 4) || !aligned(kept, 4) || !aligned(slot_weights_out, 4) ||
      !aligned(births_out, 4))
    return KVC_ERR_INVALID_ARG;
  const int64_t stay = keep < max_slots ? keep : max_slots;
  if ((slot_weights_out != nullptr && !rows_apart(num_reqs, slot_weights_out_row_stride, stay)) ||
      (births_out != nullptr && !rows_apart(num_reqs, births_out_row_stride, stay)))
    return KVC_ERR_INVALID_ARG;
  const size_t need = kvc_evict_workspace_bytes(num_reqs, max_pages_per_req, keep);
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)
    return KVC_ERR_INVALID_ARG;
  int sms = 0;
  long long wait_limit = 0;
  kvc::EvictParams p = {};
  const kvc_status st = kvc::operator_device(&sms, &p.error, &wait_limit);
  if (st != KVC_OK) return st;
  const int64_t slots = max_pages_per_req * kvc::kSlotsPerPage;
  const int64_t behind = slots > keep ? slots - keep : 0;
  p.kv_cache = kv_cache;
  p.four_bits = kv_format == KVC_FORMAT_4BIT;
  p.num_pages = num_kv_pages;
  p.page_table = page_table;
  p.num_reqs = num_reqs;
  p.page_table_row_stride = page_table_row_stride;
  p.lengths = lengths;
  p.max_slots = max_slots < slots ? max_slots : slots;
  p.weights = slot_weights;
  p.weights_row_stride = slot_weights_row_stride;
  p.births = births;
  p.births_row_stride = births_row_stride;
  p.keep = keep;
  p.recent = recent;
  p.lengths_out = lengths_out;
  p.kept = kept;
  p.weights_out = slot_weights_out;
  p.weights_out_row_stride = slot_weights_out_row_stride;
  p.births_out = births_out;
  p.births_out_row_stride = births_out_row_stride;
  p.counts = static_cast<int32_t*>(workspace);
  p.moves = reinterpret_cast<longlong2*>(static_cast<uint8_t*>(workspace) +
                                       round16(sizeof(int32_t) * num_reqs));
  p.move_stride = behind < keep ? behind : keep;
  const cudaError_t e = kvc::launch_evict(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc_status kvc_store(const void* x, int32_t x_dtype, int64_t x_row_stride, int64_t num_rows, uint8_t* kv_cache,
                     int32_t kv_format, int64_t num_kv_pages, const int64_t* slots, const int64_t* positions,
                     int64_t positions_row_stride, int64_t positions_axis_stride, int32_t num_axes,
                     const uint8_t* pair_axes, const float* cos_sin_cache, int64_t num_positions, void* stream) {
  if (num_rows < 0 || num_rows > kMaxRows || !format_ok(kv_format) ||
      (x_dtype != KVC_DTYPE_F32 && x_dtype != KVC_DTYPE_BF16))
    return KVC_ERR_INVALID_ARG;
  kvc::StoreParams p = {};
  if (num_axes != 0 && !rotation_ok(num_rows, positions, positions_row_stride, positions_axis_stride, num_axes, pair_axes, cos_sin_cache, num_positions,
                                    &p.rotation))
    return KVC_ERR_INVALID_ARG;
  if (num_axes == 0 && (positions != nullptr || pair_axes != nullptr)) return KVC_ERR_INVALID_ARG;
  if (num_rows == 0) return KVC_OK;
  p.x_f32 = x_dtype == KVC_DTYPE_F32;
  if (x == nullptr || kv_cache == nullptr || slots == nullptr || num_kv_pages <= 0 || num_kv_pages > INT32_MAX || !aligned(x, 16) ||
      !aligned(kv_cache, 16) || !aligned(slots, 8) || x_row_stride < 0 ||
      x_row_stride % (p.x_f32 ? 4 : 8) != 0)
    return KVC_ERR_INVALID_ARG;
  int sms = 0;
  long long wait_limit = 0;
  const kvc_status st = kvc::operator_device(&sms, &p.error, &wait_limit);
  if (st != KVC_OK) return st;
  p.x = x;
  p.x_row_stride = x_row_stride;
  p.num_rows = num_rows;
  p.kv_cache = kv_cache;
  p.num_pages = num_kv_pages;
  p.slots = slots;
  const cudaError_t e = kvc::launch_store(p, kv_format == KVC_FORMAT_4BIT, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc_status kvc_dequantize_format(const uint8_t* kv_cache, int32_t kv_format, int64_t num_kv_pages,
                                 const int64_t* slots, int64_t num_slots, void* out, int32_t out_dtype,
                                 void* stream) {
  if (!format_ok(kv_format)) return KVC_ERR_INVALID_ARG;
  if (kv_format == KVC_FORMAT_8BIT)
    return kvc_dequantize(kv_cache, num_kv_pages, slots, num_slots, out, out_dtype, stream);
  if (num_slots < 0 || num_slots > kMaxRows || (out_dtype != KVC_DTYPE_F32 && out_dtype != KVC_DTYPE_BF16))
    return KVC_ERR_INVALID_ARG;
  if (num_slots == 0) return KVC_OK;
  if (kv_cache == nullptr || slots == nullptr || out == nullptr || num_kv_pages <= 0 || num_kv_pages > INT32_MAX || !aligned(kv_cache, 16) ||
      !aligned(slots, 8) || !aligned(out, 16))
    return KVC_ERR_INVALID_ARG;
  int sms = 0;
  long long wait_limit = 0;
  uint32_t* error = nullptr;
  const kvc_status st = kvc::operator_device(&sms, &error, &wait_limit);
  if (st != KVC_OK) return st;
  const cudaError_t e = kvc::launch_dequantize4(kv_cache, num_kv_pages, slots, num_slots, out,
                                                out_dtype == KVC_DTYPE_BF16, error,
                                                static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

kvc_status kvc_rotate(const void* x, int32_t dtype, int64_t x_token_stride, int64_t x_head_stride, int64_t num_tokens,
                      int32_t num_heads, const int64_t* positions, int64_t positions_token_stride,
                      int64_t positions_axis_stride, int32_t num_axes, const uint8_t* pair_axes,
                      const float* cos_sin_cache, int64_t num_positions, int32_t inverse, void* out,
                      int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  if (num_tokens < 0 || num_heads < 0 || num_tokens > kMaxRows || num_heads > kMaxTurnedHeads ||
      (inverse != 0 && inverse != 1) || (dtype != KVC_DTYPE_F32 && dtype != KVC_DTYPE_BF16))
    return KVC_ERR_INVALID_ARG;
  kvc::RotateParams p = {};
  const bool none = num_tokens == 0 || num_heads == 0;
  if (!rotation_ok(none ? 0 : num_tokens, positions, positions_token_stride, positions_axis_stride, num_axes, pair_axes,
                   cos_sin_cache, num_positions, &p.rotation))
    return KVC_ERR_INVALID_ARG;
  if (none) return KVC_OK;
  p.f32 = dtype == KVC_DTYPE_F32;
  const int piece = p.f32 ? 4 : 8;  // elements in 16 bytes
  if (x == nullptr || out == nullptr || !aligned(x, 16) || !aligned(out, 16) || x_token_stride < 0 ||
      x_head_stride < 0 || out_token_stride < 0 || out_head_stride < 0 || x_token_stride % piece != 0 ||
      x_head_stride % piece != 0 || out_token_stride % piece != 0 || out_head_stride % piece != 0 ||
      !heads_apart(num_tokens, out_token_stride, num_heads, out_head_stride))
    return KVC_ERR_INVALID_ARG;
  if (num_tokens > INT32_MAX) return KVC_ERR_UNSUPPORTED;  // (a launch has no more CTAs)
  // in place, or apart: else rows would be read that others have been turned into
  const bool in_place = x == out && (num_tokens == 1 || x_token_stride == out_token_stride) &&
                        (num_heads == 1 || x_head_stride == out_head_stride);
  if (!in_place && kvc::rows_meet(x, {x_token_stride, x_head_stride}, out, {out_token_stride, out_head_stride}, num_tokens, num_heads,
                                  kvc::kRopeDim, p.f32 ? 4 : 2))
    return KVC_ERR_INVALID_ARG;
  int sms = 0;
  long long wait_limit = 0;
  const kvc_status st = kvc::operator_device(&sms, &p.error, &wait_limit);
  if (st != KVC_OK) return st;
  p.x = x;
  p.x_token_stride = x_token_stride;
  p.x_head_stride = x_head_stride;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.inverse = inverse;
  p.out = out;
  p.out_token_stride = out_token_stride;
  p.out_head_stride = out_head_stride;
  const cudaError_t e = kvc::launch_rotate(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? KVC_OK : KVC_ERR_CUDA;
}

}  // extern "C"
