// Whether two strided views share memory (host code, no HIP): outputs that do
// are refused, as the kernels' reads and writes would race.
#pragma once

#include <stdint.h>

namespace repro {

// Runs of `bytes` bytes, size[d] of them stride[d] >= 0 bytes apart along each
// of up to three dimensions.  Without bytes it holds nothing.
struct View {
  uintptr_t first = 0;
  int64_t bytes = 0;
  int dims = 0;
  int64_t size[3], stride[3];
  __int128 reach = 0;  // bytes from the first to one past the last

  View() = default;
  View(const void* p, int64_t run) : first(reinterpret_cast<uintptr_t>(p)), bytes(run), reach(run) {}
  void dimension(int64_t n, int64_t apart) {
    if (n <= 0) bytes = 0;
    if (n <= 1 || apart == 0) return;  // one place
    size[dims] = n;
    stride[dims++] = apart;
    reach += (__int128)(n - 1) * apart;
  }
};

// Whether some element of a list of sums lies in (low, high): value + the sum
// over t of step[t] * k, low[t] <= k <= high[t], steps in descending order.
struct Sums {
  struct Term {
    __int128 step, low, high;
  };
  Term term[6];
  __int128 least[7], most[7];  // of the sum of the terms from t on
  __int128 common[7];          // their greatest common divisor
  int terms = 0;
  __int128 low, high;
  int visits = 0;

  bool meets(int t, __int128 value) {
    // Multiples of the divisor of what is left to add: none may fall inside.
    if (common[t] > 0) {
      __int128 rest = value % common[t];
      if (rest < 0) rest += common[t];
      if (rest >= high && rest - common[t] <= low) return false;
    }
    if (t == terms) return low < value && value < high;
    if (++visits > kVisits) return true;
    // The k for which the terms after this one can still bring it inside.
    const Term& m = term[t];
    __int128 from = down(low - value - most[t + 1], m.step) + 1;
    __int128 to = -down(value + least[t + 1] - high, m.step) - 1;
    if (from < m.low) from = m.low;
    if (to > m.high) to = m.high;
    for (; from <= to; ++from)
      if (meets(t + 1, value + m.step * from)) return true;
    return false;
  }

  static __int128 down(__int128 a, __int128 b) { return a >= 0 ? a / b : -((-a + b - 1) / b); }
  // Views whose dimensions nest or share their strides take some tens of
  // visits; ones that cross so irregularly that these do not settle it count
  // as sharing memory.
  static constexpr int kVisits = 4096;
};

inline bool share_memory(const View& a, const View& b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  if (a.first + a.reach <= b.first || b.first + b.reach <= a.first) return false;
  // A run of a at distance x from a run of b touches it for -a.bytes < x <
  // b.bytes; the distances are sums over the dimensions, in which dimensions
  // of one stride count by the difference of their indexes alone.
  Sums s;
  for (int d = 0; d < a.dims; ++d) s.term[s.terms++] = {a.stride[d], 0, a.size[d] - 1};
  for (int d = 0; d < b.dims; ++d) {
    int t = 0;
    while (t < s.terms && s.term[t].step != b.stride[d]) ++t;
    if (t == s.terms) s.term[s.terms++] = {b.stride[d], 0, 0};
    s.term[t].low -= b.size[d] - 1;
  }
  for (int i = 1; i < s.terms; ++i)
    for (int j = i; j > 0 && s.term[j].step > s.term[j - 1].step; --j) {
      const Sums::Term other = s.term[j];
      s.term[j] = s.term[j - 1];
      s.term[j - 1] = other;
    }
  s.least[s.terms] = s.most[s.terms] = s.common[s.terms] = 0;
  for (int t = s.terms - 1; t >= 0; --t) {
    s.least[t] = s.least[t + 1] + s.term[t].step * s.term[t].low;
    s.most[t] = s.most[t + 1] + s.term[t].step * s.term[t].high;
    __int128 x = s.term[t].step, y = s.common[t + 1];
    while (y != 0) {
      const __int128 rest = x % y;
      x = y;
      y = rest;
    }
    s.common[t] = x;
  }
  s.low = -(__int128)a.bytes;
  s.high = b.bytes;
  return s.meets(0, (__int128)a.first - (__int128)b.first);
}

// Whether two views are one and the same.
inline bool same_view(const View& a, const View& b) {
  if (a.first != b.first || a.bytes != b.bytes || a.dims != b.dims) return false;
  for (int d = 0; d < a.dims; ++d)
    if (a.size[d] != b.size[d] || a.stride[d] != b.stride[d]) return false;
  return true;
}

}  // namespace repro
