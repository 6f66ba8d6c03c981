// overlap.h -- whether operands of a call share memory, for the host's checks.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cstdlib>

namespace i8 {

// Memory of an operand: `rows` rows of `bytes`, `stride` bytes apart.
struct Extent {
  const void* base;
  int64_t bytes;
  int64_t rows = 1;
  int64_t stride = 0;
};

// Whether rows of `t` and the one row of `v` share a byte.
inline bool overlap(const Extent& t, const Extent& v) {
  if (!t.base || !v.base || t.bytes <= 0 || t.rows <= 0 || v.bytes <= 0) return false;
  const int64_t lo = static_cast<int64_t>(reinterpret_cast<uintptr_t>(v.base) - reinterpret_cast<uintptr_t>(t.base));
  const int64_t hi = lo + v.bytes;  // from t's base on
  if (hi <= 0) return false;
  // the first row that ends behind lo
  const int64_t row = lo < t.bytes ? 0 : t.rows == 1 ? 1 : (lo - t.bytes) / t.stride + 1;
  return row < t.rows && row * t.stride < hi;
}

// Whether a row of `a` shares a byte with another row of `b` (both of as many
// rows): a row may lie where the other's same row does.
inline bool rows_cross(const Extent& a, const Extent& b) {
  if (!a.base || !b.base || a.rows <= 1) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  if (d >= (a.rows - 1) * a.stride + a.bytes || d + (b.rows - 1) * b.stride + b.bytes <= 0) return false;
  if (a.stride != b.stride) {
    for (int64_t i = 0; i < b.rows; ++i) {
      const Extent row{static_cast<const char*>(b.base) + i * b.stride, b.bytes};
      const Extent before{a.base, a.bytes, i, a.stride};
      const Extent after{static_cast<const char*>(a.base) + (i + 1) * a.stride, a.bytes, a.rows - i - 1, a.stride};
      if (overlap(before, row) || overlap(after, row)) return true;
    }
    return false;
  }
  // row i + k of a begins d - k * stride before row i of b
  const int64_t k = d >= 0 ? d / a.stride : -((-d + a.stride - 1) / a.stride), r = d - k * a.stride;
  return (k != 0 && std::abs(k) < a.rows && r < a.bytes) ||
         (k + 1 != 0 && std::abs(k + 1) < a.rows && a.stride - r < b.bytes);
}

// Whether some row of `a` shares bytes with the same row of `b` (both of as many rows)
// and does not begin where it does.
inline bool rows_shifted(const Extent& a, const Extent& b) {
  if (!a.base || !b.base || a.rows <= 0) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.base) - reinterpret_cast<uintptr_t>(a.base));
  // row i of b begins d + i * drift behind row i of a: the rows i where that is small
  const int64_t drift = b.stride - a.stride;
  int64_t first = 0, last = 0;
  if (a.rows > 1 && drift != 0) {
    const int64_t middle = -d / drift, around = std::max(a.bytes, b.bytes) / std::abs(drift) + 1;
    first = std::max<int64_t>(0, middle - around);
    last = std::min(a.rows - 1, middle + around);
  }
  for (int64_t i = first; i <= last; ++i) {
    const int64_t at = d + i * drift;
    if (at != 0 && at < a.bytes && -at < b.bytes) return true;
  }
  return false;
}

// Whether rows [tokens, heads] of `dim` elements, these strides apart, share an
// element.
inline bool rows_overlap(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
  if ((tokens > 1 && token < dim) || (heads > 1 && head < dim)) return true;
  if (tokens <= 1 || heads <= 1) return false;
  if (token >= head * (heads - 1) + dim || head >= token * (tokens - 1) + dim) return false;
  // neither inside the other: the tokens nearest to each head's offset
  for (int64_t h = 1; h < heads; ++h)
    for (int64_t t = h * head / token; t <= h * head / token + 1 && t < tokens; ++t)
      if (std::abs(h * head - t * token) < dim) return true;
  return false;
}

}  // namespace i8
