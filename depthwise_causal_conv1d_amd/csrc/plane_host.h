// plane_host.h -- host-side checks of strided matrices: which elements a call
// touches, whether two buffers share memory, and launch limits.
#pragma once

#include "sconv_host.h"

namespace sconv {

// The runtime takes a launch of fewer than 2^32 threads in one dimension.
inline bool valid_grid(int64_t workgroups, int64_t threads) {
  return workgroups > 0 && workgroups <= INT32_MAX && workgroups * threads < (int64_t)1 << 32;
}

// A [nc, nt] matrix of es-byte elements at element strides (sc, st).  The
// stride of a dimension of one entry is never used, so it is set to what a
// dense matrix has.
struct Plane {
  const void* p;
  int64_t sc, st, nc, nt, es;

  bool empty() const { return nc == 0 || nt == 0; }
  bool readable() const { return sc >= 0 && st >= 0; }
  // From the first element's first byte to the last one's last.
  int64_t bytes() const { return empty() ? 0 : ((nc - 1) * sc + (nt - 1) * st + 1) * es; }
  // Elements along the dimension of the smaller stride: bytes from the
  // first to the last, and the step between two such runs.
  int64_t run() const { return ((sc <= st ? (nc - 1) * sc : (nt - 1) * st) + 1) * es; }
  int64_t step() const { return (sc <= st ? st : sc) * es; }
  // No two elements share memory (a run ends before the next begins).
  bool writable() const {
    if (empty()) return true;
    if (sc < 1 || st < 1) return false;
    return nc == 1 || nt == 1 || run() <= step();
  }
};

inline Plane plane(const void* p, int64_t sc, int64_t st, int64_t nc, int64_t nt, int64_t es) {
  Plane a = {p, sc, st, nc, nt, es};
  if (nc == 1) a.sc = st > 0 && nt > 1 ? st * nt : 1;
  if (nt == 1) a.st = a.sc > 0 && nc > 1 ? a.sc * nc : 1;
  return a;
}

inline bool same_plane(const Plane& a, const Plane& b) {
  return a.p == b.p && a.sc == b.sc && a.st == b.st && a.es == b.es;
}

// Whether two planes may share memory.  Planes of the same strides whose
// runs lie between each other's (columns of one wider matrix) do not;
// other planes are judged by their whole byte ranges.
inline bool planes_overlap(const Plane& a, const Plane& b) {
  if (!overlap(a.p, a.bytes(), b.p, b.bytes())) return false;
  if (a.sc != b.sc || a.st != b.st || a.es != b.es || a.nc != b.nc || a.nt != b.nt) return true;
  const int64_t step = a.step();
  if (step <= 0 || a.run() > step) return true;
  int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % step;
  if (d < 0) d += step;
  return d < a.run() || step - d < a.run();
}

}  // namespace sconv
