// Whether tensors of the C-ABI entry points lie on each other: host code, on addresses alone.
#pragma once

#include <stdint.h>

namespace mxg {
namespace host {

// Rows of a tensor: `rows` of `bytes` bytes each, `step` bytes apart, which is not less than `bytes` unless there is one row.
struct RowsAt {
  const void* at;
  int64_t rows, bytes, step;
};

inline RowsAt rows_at(const void* at, int64_t rows, int64_t columns, int64_t ld, int64_t elem) { return {at, rows, columns * elem, ld * elem}; }
// Contiguous bytes.
inline RowsAt flat(const void* at, int64_t bytes) { return {at, 1, bytes, bytes}; }

// Whether two tensors share a byte.  Where their rows are equally far apart, the first rows that could meet decide (the
// halves of one matrix's columns lie apart); others are compared row by row as far as the tensors reach into each other.
inline bool overlap(const RowsAt& a, const RowsAt& b) {
  if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.bytes <= 0 || b.bytes <= 0) return false;
  const int64_t sa = a.rows > 1 ? a.step : a.bytes, sb = b.rows > 1 ? b.step : b.bytes;
  // in bytes behind a's first
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  const int64_t end = (a.rows - 1) * sa + a.bytes;
  if (d >= end || d + (b.rows - 1) * sb + b.bytes <= 0) return false;
  // b's row j from the first that ends past a's begin, while it begins before a's end
  for (int64_t j = d + b.bytes > 0 ? 0 : (-d - b.bytes) / sb + 1; j < b.rows && d + j * sb < end; ++j) {
    const int64_t from = d + j * sb, last = (from + b.bytes - 1) / sa;
    const int64_t i = last < a.rows ? last : a.rows - 1;  // the last row of a that begins before b's row ends
    if (i * sa + a.bytes > from) return true;
    if (sa == sb) return false;
  }
  return false;
}

// Whether two tensors with rows of one length are the same one.
inline bool same(const RowsAt& a, const RowsAt& b) { return a.at == b.at && (a.rows <= 1 || a.step == b.step); }

}  // namespace host
}  // namespace mxg
