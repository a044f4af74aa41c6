// Ranges of bytes that a call's arguments take.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace pkv {

// Whether two ranges have a byte in common.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

using Wide = __int128;   // sums of any 64-bit strides

// [rows][heads] pieces of `len` bytes at these strides (bytes); none where `base` is null or a count is 0.
struct Rows {
  const void* base;
  int64_t rows, heads;
  Wide row_stride, head_stride;
  int64_t len;
  Wide lo, hi;   // from the first byte to behind the last one; equal where there is none

  Rows(const void* base, int64_t rows, int64_t heads, Wide row_stride, Wide head_stride, int64_t len)
      : base(base), rows(rows), heads(heads), row_stride(row_stride), head_stride(head_stride), len(len) {
    lo = hi = static_cast<Wide>(reinterpret_cast<uintptr_t>(base));
    if (!base || rows <= 0 || heads <= 0 || len <= 0) return;
    const Wide r = (rows - 1) * row_stride, h = (heads - 1) * head_stride;
    lo += (r < 0 ? r : 0) + (h < 0 ? h : 0);
    hi += (r > 0 ? r : 0) + (h > 0 ? h : 0) + len;
  }
  Rows(const void* base, int64_t bytes) : Rows(base, 1, 1, 0, 0, bytes) {}
  bool operator==(const Rows& o) const {
    return base == o.base && rows == o.rows && heads == o.heads && len == o.len &&
           (rows <= 1 || row_stride == o.row_stride) && (heads <= 1 || head_stride == o.head_stride);
  }
};

// Whether two such sets have a byte in common, decided exactly, so that parts of one projection's rows count as apart
// although their ranges overlap.  With x at X + sum i_d s_d and y at Y + sum j_d s_d they meet where
//   X - Y = sum j_d s_d - sum i_d s_d + r,   -len_x < r < len_y:
// counted from x's last byte down and y's first one up no term is negative, steps of equal size are one
// of both counts, and a step no longer than the range of r only makes that longer.  Two parts of the same rows
// leave at most two steps, and each a candidate or two.  `budget`: candidates looked at; a layout that needs more
// of them counts as meeting.
__attribute__((noinline)) inline bool meet_within(const Rows& x, const Rows& y, int budget) {
  struct Step {
    Wide n, s;
  } step[4];
  int steps = 0;
  Wide at = x.hi - 1 - y.lo;   // sum k_d s_d + r with 0 <= r < len, 0 <= k_d < n_d, all s_d > 0
  Wide len = static_cast<Wide>(x.len) + y.len - 1;
  auto add = [&](Wide n, Wide s) {
    if (n <= 1 || s == 0) return;
    if (s < 0) s = -s;
    for (int i = 0; i < steps; ++i)
      if (step[i].s == s) {
        step[i].n += n - 1;
        return;
      }
    step[steps++] = {n, s};
  };
  add(x.rows, x.row_stride);
  add(x.heads, x.head_stride);
  add(y.rows, y.row_stride);
  add(y.heads, y.head_stride);
  std::sort(step, step + steps, [](const Step& a, const Step& b) { return a.s < b.s; });
  int first = 0;
  for (; first < steps && step[first].s <= len; ++first) len += (step[first].n - 1) * step[first].s;
  Wide rest[4] = {};   // what the smaller steps come to
  for (int i = first + 1; i < steps; ++i) rest[i] = rest[i - 1] + (step[i - 1].n - 1) * step[i - 1].s;
  // the largest step first
  auto find = [&](auto self, int d, Wide to) -> bool {
    if (to < 0) return false;
    if (--budget < 0) return true;
    if (d < first) return to < len;
    const Wide s = step[d].s, low = to - len - rest[d] + 1;
    for (Wide k = std::min(step[d].n - 1, to / s); k >= 0 && k * s >= low; --k)
      if (self(self, d - 1, to - k * s)) return true;
    return false;
  };
  return find(find, steps - 1, at);
}
inline bool meet(const Rows& x, const Rows& y, int budget = 4096) {   // ranges that lie apart: nearly all
  return x.lo < y.hi && y.lo < x.hi && x.lo < x.hi && y.lo < y.hi && meet_within(x, y, budget);
}

}  // namespace pkv
