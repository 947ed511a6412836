// Tensors that share memory: what an output may not do with an input (host).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sa {
namespace api {

// Rows of `row` bytes from ptr on, ext[i] of them str[i] bytes apart in dimension i.
struct Rows {
  uintptr_t ptr;
  long long ext[3], str[3], row, span;   // span: bytes from the first row's start to the last one's end, or 0
};
inline Rows rows_of(const void* ptr, int B, int S, int H, int n, int size, const long long str[3]) {
  Rows r = {reinterpret_cast<uintptr_t>(ptr), {B, S, H}, {}, (long long)n * size, 0};
  double span = 0;
  for (int i = 0; i < 3; ++i) {
    r.str[i] = r.ext[i] > 1 ? str[i] * size : 0;
    span += (double)(r.ext[i] - 1) * (double)r.str[i];
  }
  // (larger than any memory: nothing to compare, and nothing below overflows)
  if (span < 0x1p56) r.span = (r.ext[0] - 1) * r.str[0] + (r.ext[1] - 1) * r.str[1] + (r.ext[2] - 1) * r.str[2] + r.row;
  return r;
}
inline bool same(const Rows& a, const Rows& b) {
  return a.ptr == b.ptr && std::equal(a.str, a.str + 3, b.str) && std::equal(a.ext, a.ext + 3, b.ext) && a.row == b.row;
}

// Whether `at` plus a sum of multiples of steps[0..n), largest step first, each multiple in its range, can come to between
// -room and room.  steps_left bounds the search: slices of one buffer, whose steps lie within one another, take
// two or three tries a step.  (Undecided is taken for no.)
struct Step {
  long long by, lo, hi;
};
inline bool meets(const Step* steps, int n, long long at, long long room, int& steps_left) {
  if (n == 0) return -room < at && at < room;
  long long lo = 0, hi = 0;   // what the steps after this one can add
  for (int i = 1; i < n; ++i) {
    lo += steps[i].by * steps[i].lo;
    hi += steps[i].by * steps[i].hi;
  }
  auto down = [](long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); };
  const long long first = std::max(steps->lo, -down(at + hi + room - 1, steps->by));
  const long long last = std::min(steps->hi, down(room - 1 - at - lo, steps->by));
  for (long long x = first; x <= last; ++x) {
    if (--steps_left < 0) return false;
    if (meets(steps + 1, n - 1, at + x * steps->by, room, steps_left)) return true;
  }
  return false;
}

// Whether a row of a and a row of b (of one length) have a byte in common.
inline bool share_memory(const Rows& a, const Rows& b) {
  if (a.span == 0 || b.span == 0 || a.ptr + a.span <= b.ptr || b.ptr + b.span <= a.ptr) return false;
  Step steps[6];
  int n = 0;
  auto add = [&](long long by, long long lo, long long hi) {
    if (by == 0) return;
    int i = 0;
    while (i < n && steps[i].by != by) ++i;
    if (i == n) steps[n++] = {by, 0, 0};
    steps[i].lo += lo;
    steps[i].hi += hi;
  };
  for (int i = 0; i < 3; ++i) {
    add(a.str[i], 1 - a.ext[i], 0);
    add(b.str[i], 0, b.ext[i] - 1);
  }
  std::sort(steps, steps + n, [](const Step& x, const Step& y) { return x.by > y.by; });
  int steps_left = 10000;
  return meets(steps, n, (long long)(b.ptr - a.ptr), a.row, steps_left);
}

}  // namespace api
}  // namespace sa
