// sd_overlap.cuh -- host checks of whether the arrays of a call share memory.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace {

// Whether two arrays of na and nb bytes share any (NULL shares nothing).
inline bool share(const void* a, size_t na, const void* b, size_t nb) {
  return a && b && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// bf16 values [n][H][D] at i*ld + h*hs + d.
struct HeadRows {
  const void* p;
  long ld, hs;
  int H;
};

// Whether a value of one array is ever a value of the other: exact where the strides are alike, as those of
// slices of one array are; of others only the first values are compared. With alike strides the values'
// places differ by i*ld + j*hs + d for i within +-(n-1), j from -(b.H-1) to a.H-1, d within +-(D-1).
inline bool heads_share(const HeadRows& a, const HeadRows& b, int n, int D) {
  if ((n > 1 && a.ld != b.ld) || (a.H > 1 && b.H > 1 && a.hs != b.hs)) return a.p == b.p;
  struct Axis {
    long step, lo, hi;
  };
  Axis outer = {n > 1 ? a.ld : 0, 1L - n, n - 1L};
  Axis inner = {a.H > 1 ? a.hs : b.H > 1 ? b.hs : 0, 1L - b.H, a.H - 1L};
  if (outer.step < inner.step) {
    const Axis x = outer;
    outer = inner;
    inner = x;
  }
  // whether some step of an axis comes within a head of x
  auto down = [](long x, long y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };  // x / y, y > 0
  auto reaches = [&](long x, const Axis& s) {
    if (s.step == 0) return x > -D && x < D;
    const long from = -down(-(x - D + 1), s.step), to = down(x + D - 1, s.step);
    return (from > s.lo ? from : s.lo) <= (to < s.hi ? to : s.hi);
  };
  const long apart = ((intptr_t)b.p - (intptr_t)a.p) / 2;
  if (outer.step == 0) return apart > -D && apart < D;
  // the outer steps behind which an inner one can still do so: one or two where the inner steps lie
  // within an outer one
  long i = -down(-(apart - inner.hi * inner.step - D + 1), outer.step);
  long last = down(apart - inner.lo * inner.step + D - 1, outer.step);
  if (i < outer.lo) i = outer.lo;
  if (last > outer.hi) last = outer.hi;
  for (; i <= last; ++i)
    if (reaches(apart - i * outer.step, inner)) return true;
  return false;
}

// Whether values of one array lie on one another.
inline bool heads_overlap(const HeadRows& a, int n, int D) {
  if ((n > 1 && a.ld < D) || (a.H > 1 && a.hs < D)) return true;
  if (n == 1 || a.H == 1) return false;
  // rows (or heads) within one another's range: i*ld = j*hs + d for some i, j > 0
  const bool rows = a.ld >= a.hs;
  const long big = rows ? a.ld : a.hs, small = rows ? a.hs : a.ld;
  const long n_big = rows ? n : a.H, n_small = rows ? a.H : n;
  for (long i = 1; i < n_big && i * big < (n_small - 1) * small + D; ++i) {
    const long j = i * big / small, d = i * big - j * small;
    if (j < n_small && d < D) return true;
    if (j + 1 < n_small && small - d < D) return true;
  }
  return false;
}

}  // namespace
