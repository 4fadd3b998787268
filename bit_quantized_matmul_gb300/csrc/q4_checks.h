// q4_checks.h — host checks of arguments that the cache and attention calls share.
#pragma once

#include <cmath>
#include <cstdint>

#include "q4mm_internal.h"

namespace q4 {

constexpr int64_t LIM = (int64_t)1 << 31;
// Row, position and request counts end here: kernels step past their end by up to a
// grid's worth (152 x 16 CTAs of 4 warps at most) in 32 bits.
constexpr int64_t MOST = LIM - (1 << 17);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int elem_bytes(int dtype) {
  return dtype == Q4_DTYPE_F32 ? 4 : (dtype == Q4_DTYPE_F16 || dtype == Q4_DTYPE_BF16) ? 2 : 0;
}

inline bool strides_ok(const int64_t* st) {
  return st && st[0] >= 0 && st[1] >= 0 && st[0] < (LIM << 28) && st[1] < (LIM << 28);
}

// Strides of rows x heads; one that is never taken may be anything.
inline bool strides_aligned(const int64_t* st, int eb, int64_t rows, int64_t heads) {
  return (rows == 1 || st[0] * eb % 16 == 0) && (heads == 1 || st[1] * eb % 16 == 0);
}

// Whether n bytes at p and m bytes at q have one in common.
inline bool meet(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && (a <= b ? b - a < (uintptr_t)n : a - b < (uintptr_t)m);
}

// Rows x heads x D values at p: a row of them is taken as one piece, its heads' gaps included.
struct Rows {
  const void* p;
  int64_t row, piece, rows;  // bytes from row to row and of a row
  Rows(const void* p, const int64_t* st, int64_t rows, int64_t heads, int64_t d, int eb)
      : p(p), row(rows > 1 ? st[0] * eb : 0), piece(((heads > 1 ? (heads - 1) * st[1] : 0) + d) * eb), rows(rows) {}
  bool meets(const void* out, int64_t bytes) const {
    const char* base = static_cast<const char*>(p);
    if (row == 0) return rows > 0 && meet(base, piece, out, bytes);
    // the first row that ends after `out` begins
    const int64_t before = static_cast<const char*>(out) - base - piece;
    const int64_t t = before < 0 ? 0 : before / row + 1;
    return t < rows && meet(base + t * row, piece, out, bytes);
  }
  // the very rows, packed
  bool same(const void* out, int64_t heads, int64_t d, int eb) const {
    return p == out && piece == heads * d * eb && (rows == 1 || row == piece);
  }
};

// A positive factor that stays finite in units of log2.
inline bool scale_ok(float scale) { return scale > 0.0f && std::isfinite(scale * 1.4427f); }

}  // namespace q4
