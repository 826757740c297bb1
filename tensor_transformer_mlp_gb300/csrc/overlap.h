// Whether tensors of one call share memory, by what they occupy: an output that is not to be another tensor of the call must
// not lie across one either. Tensors of heads are lattices of pieces, and those of one packed matrix interleave without
// touching, so extents alone do not tell. Plain C++, on the host.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

namespace tpmlp {

// `width` bytes at at + r * row + h * head for r < rows and h < heads. width 0: nothing (a null pointer).
struct Region {
  uintptr_t at;
  int64_t rows, row, heads, head, width;
};

using Wide = __int128;  // sums of offsets of valid strides may pass 64 bits

inline Region flat_region(const void* p, int64_t count, int64_t size) {
  const Wide bytes = p ? static_cast<Wide>(count) * size : 0;
  return {reinterpret_cast<uintptr_t>(p), 1, 1, 1, 1, static_cast<int64_t>(std::min<Wide>(bytes, INT64_MAX))};
}

inline bool same_region(const Region& a, const Region& b) {
  return a.at == b.at && a.row == b.row && a.head == b.head && a.rows == b.rows && a.heads == b.heads && a.width == b.width;
}

// Neighbouring pieces as one.
inline Region joined(Region r) {
  for (int i = 0; i < 2; ++i) {
    if (r.heads > 1 && r.head == r.width) r.width *= r.heads, r.heads = 1;
    if (r.rows > 1 && r.row == r.width) r.width *= r.rows, r.rows = 1;
  }
  return r;
}

// Whether some k in [lo, hi] puts a piece of wb bytes at d + k * stride across one of wa bytes at 0.
inline bool some_meet(Wide d, Wide wa, Wide wb, Wide stride, Wide lo, Wide hi) {
  const Wide first = -wb - d;  // the least k with d + k * stride > -wb
  const Wide k = std::max<Wide>(lo, (first >= 0 ? first / stride : -((-first + stride - 1) / stride)) + 1);
  return k <= hi && d + k * stride < wa;
}

// Exact, except that tensors of the same memory whose row strides and head strides both differ and which take more than 2^16
// comparisons are let pass.
inline bool overlap(Region a, Region b) {
  if (a.width == 0 || b.width == 0) return false;
  auto end = [](const Region& r) {
    return static_cast<Wide>(r.at) + static_cast<Wide>(r.rows - 1) * r.row + static_cast<Wide>(r.heads - 1) * r.head + r.width;
  };
  if (end(a) <= static_cast<Wide>(b.at) || end(b) <= static_cast<Wide>(a.at)) return false;
  a = joined(a);
  b = joined(b);
  // Where one of them has a single place its stride may be anything.
  if (a.rows == 1) a.row = b.row;
  if (b.rows == 1) b.row = a.row;
  if (a.heads == 1) a.head = b.head;
  if (b.heads == 1) b.head = a.head;
  // The rows in closed form, the heads one by one, or the other way round.
  if (a.row != b.row || (a.head == b.head && std::min(a.rows, b.rows) < std::min(a.heads, b.heads))) {
    std::swap(a.rows, a.heads);
    std::swap(a.row, a.head);
    std::swap(b.rows, b.heads);
    std::swap(b.row, b.head);
  }
  const Wide d = static_cast<Wide>(b.at) - static_cast<Wide>(a.at);
  constexpr int64_t kMost = 1 << 16;
  if (a.row == b.row && a.head == b.head) {
    for (int64_t h = 1 - a.heads; h < b.heads; ++h)
      if (some_meet(d + static_cast<Wide>(h) * a.head, a.width, b.width, a.row, 1 - a.rows, b.rows - 1)) return true;
    return false;
  }
  // One stride at least differs: the pieces of one of them, or of both, one by one.
  const bool rows_alike = a.row == b.row;
  if (static_cast<Wide>(a.heads) * b.heads * (rows_alike ? 1 : a.rows) > kMost) return false;
  for (int64_t h = 0; h < a.heads; ++h)
    for (int64_t g = 0; g < b.heads; ++g) {
      const Wide at = d + static_cast<Wide>(g) * b.head - static_cast<Wide>(h) * a.head;
      if (rows_alike) {
        if (some_meet(at, a.width, b.width, a.row, 1 - a.rows, b.rows - 1)) return true;
      } else {
        for (int64_t r = 0; r < a.rows; ++r)
          if (some_meet(at - static_cast<Wide>(r) * a.row, a.width, b.width, b.row, 0, b.rows - 1)) return true;
      }
    }
  return false;
}

// Whether one of `outputs` overlaps one of `others`, or another of `outputs`.
inline bool any_overlap(std::initializer_list<Region> outputs, std::initializer_list<Region> others) {
  for (const Region* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Region* p = outputs.begin(); p != o; ++p)
      if (overlap(*p, *o)) return true;
    for (const Region& p : others)
      if (overlap(p, *o)) return true;
  }
  return false;
}

}  // namespace tpmlp
