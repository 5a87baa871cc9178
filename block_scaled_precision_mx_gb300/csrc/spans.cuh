// spans.cuh -- which tensors of a call share bytes, so that one whose outputs lie over its inputs is refused.
//
// Host only, and nothing else is included, so that it can be tested by itself.
#pragma once

#include <cstdint>

namespace mxgb {

// Rows of `bytes` bytes in up to two directions: n[0] x n[1] of them, step[0] >= step[1] >= 0 bytes apart; n = 1 and
// step = 0 where there is no direction.  Empty: n[0] = 0.
struct Span {
  uintptr_t at;
  int64_t bytes, n[2], step[2];
};

inline Span span(const void* at, int64_t bytes, int64_t n0 = 1, int64_t step0 = 0, int64_t n1 = 1, int64_t step1 = 0) {
  Span s{reinterpret_cast<uintptr_t>(at), bytes, {n0, n1}, {step0, step1}};
  if (!at || bytes <= 0 || n0 <= 0 || n1 <= 0) s.n[0] = 0;
  if (s.n[0] == 0) return s;
  for (int i = 0; i < 2; ++i) {
    if (s.n[i] > 1 && s.step[i] < 0) {  // (the same rows, from the other end)
      s.at += static_cast<uintptr_t>((s.n[i] - 1) * s.step[i]);
      s.step[i] = -s.step[i];
    }
    if (s.n[i] == 1 || s.step[i] == 0) s.n[i] = 1, s.step[i] = 0;
  }
  if (s.step[0] < s.step[1]) {
    const int64_t n = s.n[0], step = s.step[0];
    s.n[0] = s.n[1], s.step[0] = s.step[1];
    s.n[1] = n, s.step[1] = step;
  }
  return s;
}

inline int64_t span_reach(const Span& s) { return (s.n[0] - 1) * s.step[0] + (s.n[1] - 1) * s.step[1] + s.bytes; }

// a / b rounded down, and up, for b > 0
inline int64_t span_floor(int64_t a, int64_t b) { return a / b - (a % b < 0); }
inline int64_t span_ceil(int64_t a, int64_t b) { return a / b + (a % b > 0); }

// Whether rows of a and b share bytes that lie i step0 + j step1 + delta apart, for some i in [-(b.n[0] - 1), a.n[0] - 1]
// and j in [-(b.n[1] - 1), a.n[1] - 1]: the rows of both have the same steps.
inline bool spans_meet_in_step(const Span& a, const Span& b, int64_t step0, int64_t step1) {
  const int64_t delta = static_cast<int64_t>(a.at - b.at);
  const int64_t least = -a.bytes + 1, most = b.bytes - 1;  // of the distances at which two rows share a byte
  const int64_t lo1 = (a.n[1] - 1) * step1, hi1 = (b.n[1] - 1) * step1;
  int64_t i0 = 0, i1 = 0;
  if (step0) {
    i0 = span_ceil(least - lo1 - delta, step0);
    i1 = span_floor(most + hi1 - delta, step0);
    if (i0 < -(b.n[0] - 1)) i0 = -(b.n[0] - 1);
    if (i1 > a.n[0] - 1) i1 = a.n[0] - 1;
  }
  for (int64_t i = i0; i <= i1; ++i) {
    const int64_t x = delta + i * step0;
    if (!step1) {
      if (least <= x && x <= most) return true;
      continue;
    }
    int64_t j0 = span_ceil(least - x, step1), j1 = span_floor(most - x, step1);
    if (j0 < -(b.n[1] - 1)) j0 = -(b.n[1] - 1);
    if (j1 > a.n[1] - 1) j1 = a.n[1] - 1;
    if (j0 <= j1) return true;
  }
  return false;
}

// Whether rows of one tensor share no bytes with each other (n and steps as span takes them).
inline bool rows_apart(int64_t bytes, int64_t n0, int64_t step0, int64_t n1, int64_t step1) {
  if ((n0 > 1 && step0 == 0) || (n1 > 1 && step1 == 0)) return n0 < 1 || n1 < 1;
  const Span s = span(reinterpret_cast<const void*>(uintptr_t(1) << 62), bytes, n0, step0, n1, step1);
  if (s.n[0] == 0) return true;
  if (s.n[1] > 1 && s.step[1] < bytes) return false;
  const int64_t lo1 = (s.n[1] - 1) * s.step[1];
  for (int64_t i = 1; i < s.n[0] && i * s.step[0] - lo1 < bytes; ++i) {  // i rows on, and up to lo1 back
    if (i * s.step[0] < bytes) return false;
    if (s.n[1] > 1 && span_floor(i * s.step[0] + bytes - 1, s.step[1]) >= span_ceil(i * s.step[0] - bytes + 1, s.step[1])) {
      const int64_t j = span_ceil(i * s.step[0] - bytes + 1, s.step[1]);  // the least number of steps back that meets
      if (j <= s.n[1] - 1) return false;
    }
  }
  return true;
}

// Whether a and b share a byte.
inline bool spans_meet(const Span& a, const Span& b) {
  if (a.n[0] == 0 || b.n[0] == 0) return false;
  if (a.at >= b.at + static_cast<uintptr_t>(span_reach(b)) || b.at >= a.at + static_cast<uintptr_t>(span_reach(a))) return false;
  // Slices of one buffer lie between each other, with the same steps (where they have that direction at all).
  const bool same0 = a.n[0] == 1 || b.n[0] == 1 || a.step[0] == b.step[0];
  const bool same1 = a.n[1] == 1 || b.n[1] == 1 || a.step[1] == b.step[1];
  if (same0 && same1)
    return spans_meet_in_step(a, b, a.n[0] == 1 ? b.step[0] : a.step[0], a.n[1] == 1 ? b.step[1] : a.step[1]);
  // (rare) the one with fewer rows, row by row
  const bool swap = a.n[0] * a.n[1] < b.n[0] * b.n[1];
  const Span& many = swap ? b : a;
  const Span& few = swap ? a : b;
  for (int64_t i = 0; i < few.n[0]; ++i)
    for (int64_t j = 0; j < few.n[1]; ++j) {
      const Span row{few.at + static_cast<uintptr_t>(i * few.step[0] + j * few.step[1]), few.bytes, {1, 1}, {0, 0}};
      if (spans_meet_in_step(many, row, many.step[0], many.step[1])) return true;
    }
  return false;
}

}  // namespace mxgb
