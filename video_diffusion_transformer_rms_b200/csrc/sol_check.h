// Host-side argument checks shared by the C ABI's translation units: status
// and message of the calling thread's last error, alignment, byte ranges.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sol.h"

namespace sol {

// Record the calling thread's last error and return its status.
sol_status fail(sol_status s, const char *fmt, ...);
sol_status cuda_fail(cudaError_t e, const char *what);
// Clear it.
sol_status ok();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int esize_of(sol_dtype dt) { return dt == SOL_F32 ? 4 : 2; }

// Byte range [begin, end) touched by `rows` rows of `width` bytes, `ld`
// bytes apart, starting at p.
struct Span {
  uintptr_t begin, end;
};
inline Span span_of(const void *p, int64_t rows, int64_t ld, int64_t width) {
  uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return Span{b, b + static_cast<uintptr_t>((rows - 1) * ld + width)};
}
inline bool spans_overlap(Span a, Span b) { return a.begin < b.end && b.begin < a.end; }

// True if the strided blocks A (base a, width wa) and B (base b, width wb),
// both `rows` rows with the same row pitch `ld`, share no byte.  With equal
// pitches, B's columns sit at offset c = (b - a) mod ld inside A's rows and
// the blocks are disjoint when wa <= c <= ld - wb.
inline bool strided_disjoint(const void *a, int64_t wa, const void *b, int64_t wb, int64_t rows,
                             int64_t lda, int64_t ldb) {
  if (!spans_overlap(span_of(a, rows, lda, wa), span_of(b, rows, ldb, wb))) return true;
  if (lda != ldb) return false;
  const int64_t off = static_cast<int64_t>(reinterpret_cast<intptr_t>(b) -
                                           reinterpret_cast<intptr_t>(a));
  int64_t c = off % lda;
  if (c < 0) c += lda;
  return wa <= c && c <= lda - wb;
}

// Identical or disjoint, for two contiguous [rows, width] tensors.
inline bool same_or_disjoint(const void *a, const void *b, int64_t bytes) {
  if (a == b) return true;
  return !spans_overlap(span_of(a, 1, 0, bytes), span_of(b, 1, 0, bytes));
}

}  // namespace sol
