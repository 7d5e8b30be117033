// Whether two arrays of a call share memory (host only).  The operators run
// their blocks in any order, so an output that shares an element with an input
// of the same call would be read before or after it is written, as it happens.
// The answer is exact: column slices of one buffer, whose rows interleave, do
// not overlap.
#pragma once

#include <cstdint>
#include <utility>

namespace svdq {

// n[0] x n[1] runs of `run` bytes, step[i] bytes apart along axis i; all of it
// lies in [lo, hi), which is empty for a null pointer and for no runs.
struct Extent {
  uintptr_t lo, hi;
  long long run;
  long long n[2];
  long long step[2];     // not negative
};

inline Extent extent(const void* p, long long run, long long n0, long long n1, long long step0, long long step1) {
  Extent e{reinterpret_cast<uintptr_t>(p), 0, run, {n0, n1}, {step0, step1}};
  if (!p || run <= 0 || n0 <= 0 || n1 <= 0) return e;
  const unsigned __int128 end = (unsigned __int128)e.lo + (unsigned __int128)(n0 - 1) * step0 +
                                (unsigned __int128)(n1 - 1) * step1 + run;
  e.hi = end > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end;
  return e;
}
inline Extent extent_flat(const void* p, long long bytes) { return extent(p, bytes, 1, 1, 0, 0); }
// Rows of `cols` elements of `esize` bytes, `ld` elements apart.
inline Extent extent_rows(const void* p, long long rows, long long cols, long long ld, int esize) {
  return extent(p, cols * esize, rows, 1, ld * esize, 0);
}

namespace overlap_detail {

using Wide = __int128;       // offsets of any count and stride

inline Wide floor_div(Wide a, Wide b) {      // b > 0
  const Wide q = a / b;
  return a % b < 0 ? q - 1 : q;
}

// The bytes from the first to the last of axes [axis, 2).
inline Wide hull(const Extent& e, int axis) {
  Wide h = e.run;
  for (int i = axis; i < 2; ++i) h += (Wide)(e.n[i] - 1) * e.step[i];
  return h;
}

// Axes [axis, 2) of a, and of b which begins d bytes behind it.
inline bool meet(const Extent& a, const Extent& b, int axis, Wide d) {
  if (d >= hull(a, axis) || d + hull(b, axis) <= 0) return false;
  if (axis == 2) return true;
  // the parts of a and b further in meet where -hb < their distance < ha
  const Wide ha = hull(a, axis + 1), hb = hull(b, axis + 1);
  // first and last j in [lo, hi] with -hb < from + j step < ha
  auto range = [&](Wide from, Wide step, Wide lo, Wide hi, Wide& first, Wide& last) {
    if (step == 0) {
      first = last = lo;
      return;
    }
    first = floor_div(-hb - from, step) + 1;
    last = floor_div(ha - 1 - from, step);
    if (first < lo) first = lo;
    if (last > hi) last = hi;
  };
  const long long na = a.n[axis], nb = b.n[axis];
  Wide first, last;
  if (na == 1 || nb == 1 || a.step[axis] == b.step[axis]) {
    // part i of a and part j of b: only j - i matters
    const Wide step = na == 1 ? b.step[axis] : a.step[axis];
    range(d, step, -(Wide)(na - 1), nb - 1, first, last);
    for (Wide k = first; k <= last; ++k)
      if (meet(a, b, axis + 1, d + k * step)) return true;
    return false;
  }
  for (long long i = 0; i < na; ++i) {
    const Wide di = d - (Wide)i * a.step[axis];
    range(di, b.step[axis], 0, nb - 1, first, last);
    for (Wide j = first; j <= last; ++j)
      if (meet(a, b, axis + 1, di + j * b.step[axis])) return true;
  }
  return false;
}

// Axes of one part and of no step go; the longer step comes first.
inline Extent in_order(Extent e) {
  for (int i = 0; i < 2; ++i) {
    if (e.step[i] == 0) e.n[i] = 1;
    if (e.n[i] == 1) e.step[i] = 0;
  }
  if (e.step[0] < e.step[1]) {
    std::swap(e.step[0], e.step[1]);
    std::swap(e.n[0], e.n[1]);
  }
  return e;
}

}  // namespace overlap_detail

// True if the two share a byte.
inline bool overlap(const Extent& a, const Extent& b) {
  using namespace overlap_detail;
  if (a.lo >= b.hi || b.lo >= a.hi) return false;      // as nearly always
  return meet(in_order(a), in_order(b), 0, (Wide)b.lo - (Wide)a.lo);
}

// An output's extent against the call's other arrays.
template <int N>
bool overlaps_any(const Extent& out, const Extent (&others)[N]) {
  for (const Extent& e : others)
    if (overlap(out, e)) return true;
  return false;
}

}  // namespace svdq
