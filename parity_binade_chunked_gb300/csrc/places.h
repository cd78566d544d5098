// The memory that a call reads and writes, on the host: what must lie apart.
#pragma once
#include <stdint.h>

#include <initializer_list>

namespace sq {
namespace loss {

// Rows of `width` bytes from `at` on, `stride` from one's start to the next, the last
// one up to `end`; no rows where there is nothing.  (Strides are the caller's: what
// they come to may pass 64 bits.)
struct Place {
  __int128 at, end;
  int64_t rows;
  __int128 stride;
  int64_t width;
};
inline Place place(__int128 at, int64_t rows, __int128 stride, int64_t width) {
  if (stride == 0 && rows > 1) rows = 1;
  return {at, at + (rows - 1) * stride + width, width > 0 ? rows : 0, stride, width};
}
inline Place place(const void *p, int64_t rows, __int128 stride, int64_t width) {
  return place((__int128) reinterpret_cast<uintptr_t>(p), p ? rows : 0, stride, width);
}
inline Place place(const void *p, int64_t bytes) { return place(p, 1, 0, bytes); }
inline bool overlap(const Place &a, const Place &b) {
  if (a.rows == 0 || b.rows == 0 || a.at >= b.end || b.at >= a.end) return false;
  if (a.rows > b.rows) return overlap(b, a);
  if (b.rows == 1) return true;
  // row k of b is the first that ends behind the start of a's one row
  if (a.rows == 1) {
    const __int128 k = a.at < b.at + b.width ? 0 : (a.at - b.at - b.width) / b.stride + 1;
    return k < b.rows && b.at + k * b.stride < a.end;
  }
  // of equal strides: the first row of a among all that b's rows are to a's
  if (a.stride == b.stride)
    return overlap(place(a.at, 1, 0, a.width), place(b.at - (a.rows - 1) * b.stride, a.rows + b.rows - 1, b.stride, b.width));
  for (int64_t k = 0; k < a.rows; k++)
    if (overlap(place(a.at + k * a.stride, 1, 0, a.width), b)) return true;
  return false;
}
// Whether what is written lies apart from what is read, and from what else is written.
inline bool apart(std::initializer_list<Place> written, std::initializer_list<Place> read) {
  for (const Place *w = written.begin(); w != written.end(); w++) {
    for (const Place *o = written.begin(); o != w; o++)
      if (overlap(*w, *o)) return false;
    for (const Place &r : read)
      if (overlap(*w, r)) return false;
  }
  return true;
}

}  // namespace loss
}  // namespace sq
