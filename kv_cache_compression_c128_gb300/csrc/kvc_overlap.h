// Whether rows that are written share memory with rows that are read.  Host code.
#pragma once

#include <algorithm>
#include <cstdint>

namespace kvc {

// Rows (t, h) at t token_stride + h head_stride (elements, >= 0).
struct RowLayout {
  int64_t token_stride, head_stride;
};

namespace overlap {

using Wide = __int128;  // strides of any size, times as many rows

// Multiples lo .. hi of `step` bytes.
struct Axis {
  Wide step, lo, hi;
};

inline Wide floor_div(Wide a, Wide b) { return a / b - (a % b < 0); }  // b > 0

// Whether at + the sum of a multiple of each axis' step can come nearer to 0 than `size`.
// The axis of the largest step first: what the others add leaves few of its multiples.
inline bool near(Wide at, const Axis* axes, int count, Wide size) {
  if (count == 0) return -size < at && at < size;
  Wide least = 0, most = 0;  // what the others add
  for (int i = 1; i < count; ++i) {
    least += axes[i].step * axes[i].lo;
    most += axes[i].step * axes[i].hi;
  }
  const Axis& a = axes[0];
  const Wide from = std::max(a.lo, -floor_div(size - 1 + most + at, a.step));
  const Wide to = std::min(a.hi, floor_div(size - 1 - least - at, a.step));
  if (count == 1) return from <= to;
  for (Wide n = from; n <= to; ++n)
    if (near(at + a.step * n, axes + 1, count - 1, size)) return true;
  return false;
}

}  // namespace overlap

// Rows of `columns` elements of `element` bytes, t < tokens, h < heads (1 or more), at `x`
// and at `out`: whether a row of the one shares a byte with a row of the other.
inline bool rows_meet(const void* x, RowLayout of_x, const void* out, RowLayout of_out, int64_t tokens, int64_t heads,
                      int64_t columns, int64_t element) {
  using overlap::Axis;
  using overlap::Wide;
  const Wide size = Wide{columns} * element;
  const auto extent = [&](RowLayout l) {
    return (Wide{l.token_stride} * (tokens - 1) + Wide{l.head_stride} * (heads - 1)) * element + size;
  };
  const Wide begin_x = reinterpret_cast<uintptr_t>(x), begin_out = reinterpret_cast<uintptr_t>(out);
  if (begin_x + extent(of_x) <= begin_out || begin_out + extent(of_out) <= begin_x) return false;
  Axis axes[4];
  int count = 0;
  const auto add = [&](Wide stride, Wide lo, Wide hi) {
    const Wide step = stride * element;
    if (step == 0 || lo == hi) return;
    for (int i = 0; i < count; ++i)
      if (axes[i].step == step) {  // equal strides: only the difference counts
        axes[i].lo += lo;
        axes[i].hi += hi;
        return;
      }
    axes[count++] = Axis{step, lo, hi};
  };
  add(of_out.token_stride, 0, tokens - 1);
  add(of_out.head_stride, 0, heads - 1);
  add(of_x.token_stride, 1 - tokens, 0);
  add(of_x.head_stride, 1 - heads, 0);
  std::sort(axes, axes + count, [](const Axis& a, const Axis& b) { return a.step > b.step; });
  return overlap::near(begin_out - begin_x, axes, count, size);
}

}  // namespace kvc
