// Whether two matrices in memory share a byte (host code).
#pragma once

#include <stdint.h>

namespace moe {

// `rows` rows of `len` bytes, `step` >= len bytes apart (one row: any positive
// step).
struct Rows {
  uintptr_t at;
  int64_t rows, len, step;
};

inline Rows rows_of(const void* p, int64_t rows, int64_t len, int64_t step) {
  return Rows{reinterpret_cast<uintptr_t>(p), rows, len, step};
}
inline Rows span_of(const void* p, int64_t bytes) { return rows_of(p, 1, bytes, bytes); }

// Ranges that do not meet decide at once, and so does one test for equal
// steps (column slices of one wider matrix).  Else each row of the matrix with
// fewer of them is compared with the first row of the other that ends behind
// its start.
inline bool rows_overlap(Rows a, Rows b) {
  const auto end = [](const Rows& m) { return m.at + (m.rows - 1) * m.step + m.len; };
  if (a.rows < 1 || b.rows < 1 || a.len < 1 || b.len < 1) return false;
  if (end(a) <= b.at || end(b) <= a.at) return false;
  if (a.rows > b.rows) {
    const Rows t = a;
    a = b;
    b = t;
  }
  int64_t n = a.rows;
  if (a.step == b.step) {
    // rows i and j meet as rows i - j and 0 (or 0 and j - i) do: the later
    // start's first row against all of the other
    if (a.at < b.at) {
      const Rows t = a;
      a = b;
      b = t;
    }
    n = 1;
  }
  for (int64_t i = 0; i < n; ++i) {
    const int64_t lo = static_cast<int64_t>(a.at - b.at) + i * a.step;  // row i, from b's start
    const int64_t j = lo < b.len ? 0 : (lo - b.len) / b.step + 1;       // first with its end > lo
    if (j < b.rows && j * b.step < lo + a.len) return true;
  }
  return false;
}

}  // namespace moe
