// Rows of bytes, and whether two such sets share one (host).
#pragma once
#include <algorithm>

namespace dsa {

// `n` rows of `bytes`, `step` bytes apart, from address `at` on.
struct Rows {
  long long at, n, step, bytes;
};

namespace rows_detail {
using Wide = __int128;  // strides come from the caller
// Rows with a step >= 0, and where the last one ends.
struct Run {
  Wide at, n, step, bytes, end;
};
inline Run run_of(Wide at, Wide n, Wide step, Wide bytes) {
  if (step < 0) at += (n - 1) * step, step = -step;
  if (step == 0 && n > 1) n = 1;
  return {at, n, step, bytes, at + (n - 1) * step + bytes};
}
inline bool empty(const Run& r) { return r.n <= 0 || r.bytes <= 0; }
inline bool apart(const Run& a, const Run& b) { return a.end <= b.at || b.end <= a.at; }
// Rows of one step: b's row j is d + (j - i) step bytes behind a's row i.
inline bool meet(const Run& a, const Run& b, Wide step) {
  auto floor_div = [](Wide p, Wide q) { return p / q - (p % q < 0); };
  const Wide d = b.at - a.at;
  const Wide lo = std::max(floor_div(-b.bytes - d, step) + 1, 1 - a.n);  // -b.bytes < d + k step
  const Wide hi = std::min(floor_div(a.bytes - d - 1, step), b.n - 1);   // d + k step < a.bytes
  return lo <= hi;
}
inline bool meet(const Run& a, const Run& b) {
  if (apart(a, b)) return false;
  if (a.n == 1 && b.n == 1) return true;
  if (a.n == 1 || b.n == 1 || a.step == b.step) return meet(a, b, a.n == 1 ? b.step : a.step);
  if (a.n > b.n) return meet(b, a);
  for (Wide i = 0; i < a.n; ++i)
    if (meet(run_of(a.at + i * a.step, 1, 0, a.bytes), b)) return true;
  return false;
}
}  // namespace rows_detail

// Whether x shares a byte with y, or with one of m copies of y, `gap` bytes from one to the next.
inline bool rows_meet(const Rows& x, const Rows& y, long long m = 1, long long gap = 0) {
  using namespace rows_detail;
  const Run a = run_of(x.at, x.n, x.step, x.bytes), first = run_of(y.at, y.n, y.step, y.bytes);
  if (empty(a) || empty(first) || m <= 0) return false;
  if (apart(a, run_of(first.at, m, gap, first.end - first.at))) return false;
  if (m > y.n) return rows_meet(x, {y.at, m, gap, y.bytes}, y.n, y.step);  // few long runs
  for (Wide i = 0; i < m; ++i)
    if (meet(a, run_of(y.at + i * gap, y.n, y.step, y.bytes))) return true;
  return false;
}

}  // namespace dsa
