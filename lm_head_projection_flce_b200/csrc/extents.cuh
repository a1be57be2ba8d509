// extents.cuh - which bytes a call reads and writes, and whether two of its arguments
// share some (host only).
#pragma once

#include <algorithm>
#include <cstdint>

namespace flce {

// Bytes base + i stride[0] + j stride[1] + k stride[2] + [0, inner), i < count[0] and so on:
// rows, a state's beams.
struct Extent {
  uint64_t base, end;  // end: behind the last byte
  int64_t stride[3], count[3], inner;
  bool written;
};
static Extent make_extent(const void* base, const int64_t (&stride)[3], const int64_t (&count)[3],
                          int64_t inner, bool written) {
  Extent e{reinterpret_cast<uint64_t>(base), 0, {}, {}, inner, written};
  unsigned __int128 end = static_cast<unsigned __int128>(e.base) + uint64_t(inner);
  for (int d = 0; d < 3; ++d) {
    e.count[d] = stride[d] == 0 ? 1 : count[d];
    e.stride[d] = e.count[d] == 1 ? 0 : stride[d];
    end += static_cast<unsigned __int128>(e.count[d] - 1) * uint64_t(e.stride[d]);
  }
  e.end = end > UINT64_MAX ? UINT64_MAX : uint64_t(end);
  return e;
}
// Whether two of them have a byte in common.  Piece p of one and piece q of the other
// do when their distance, base - base' plus a multiple of every stride (those of the second
// one taken away), lies within their lengths.  Strides are tried from the largest
// down, and of each only the multiples that the smaller ones can still make good: one
// or two where both have the same strides.
struct ExtentStep {
  __int128 stride, low, high;  // multiples allowed
};
static bool extents_reach(const ExtentStep* step, int n, __int128 at, __int128 from, __int128 to) {
  if (n == 0) return at >= from && at <= to;
  __int128 least = 0, most = 0;  // what the smaller strides add
  for (int i = 1; i < n; ++i) {
    least += step[i].low * step[i].stride;
    most += step[i].high * step[i].stride;
  }
  auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0 ? 1 : 0); };
  const __int128 s = step[0].stride;
  const __int128 first = std::max(step[0].low, -floor_div(at + most - from, s));
  const __int128 last = std::min(step[0].high, floor_div(to - at - least, s));
  for (__int128 c = first; c <= last; ++c)
    if (extents_reach(step + 1, n - 1, at + c * s, from, to)) return true;
  return false;
}
static bool extents_overlap(const Extent& a, const Extent& b) {
  if (a.base >= b.end || b.base >= a.end) return false;
  ExtentStep step[6];
  int n = 0;
  for (int d = 0; d < 6; ++d) {
    const Extent& e = d < 3 ? a : b;
    if (e.count[d % 3] == 1) continue;
    const __int128 most = e.count[d % 3] - 1;
    ExtentStep one{e.stride[d % 3], d < 3 ? 0 : -most, d < 3 ? most : 0};
    int at = 0;
    while (at < n && step[at].stride > one.stride) ++at;
    if (at < n && step[at].stride == one.stride) {
      step[at].low += one.low;
      step[at].high += one.high;
      continue;
    }
    for (int i = n++; i > at; --i) step[i] = step[i - 1];
    step[at] = one;
  }
  return extents_reach(step, n, __int128(a.base) - __int128(b.base), -(__int128(a.inner) - 1),
                       __int128(b.inner) - 1);
}

}  // namespace flce
