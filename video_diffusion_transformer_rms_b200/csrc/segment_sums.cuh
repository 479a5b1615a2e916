// Contiguous shares of token rows and the (sample, modality) keys they meet,
// shared by the kernels that sum over rows and by the kernel that joins the
// sums (sol_train.h, Segments).
#pragma once

#include <stdint.h>

#include "sol_train.h"

namespace sol {

// First row of CTA c's share; c = ctas gives the row count.  With ctas <=
// rows every share has a row.
__host__ __device__ __forceinline__ int64_t share_begin(const Segments &s, int64_t c) {
  return s.rows * c / s.ctas;
}
// The CTA whose share holds `row`: the largest c with rows * c / ctas <= row.
__host__ __device__ __forceinline__ int share_of(const Segments &s, int64_t row) {
  return static_cast<int>(((row + 1) * s.ctas - 1) / s.rows);
}
__host__ __device__ __forceinline__ int key_of(const Segments &s, int64_t row) {
  if (s.keys == 1) return 0;
  const int64_t b = row / s.L;
  return static_cast<int>(2 * b + (row - b * s.L >= s.n_video ? 1 : 0));
}
// Rows [begin, end) of a key; empty if the modality has no rows.
__host__ __device__ __forceinline__ void key_rows(const Segments &s, int key, int64_t *begin,
                                                  int64_t *end) {
  if (s.keys == 1) {
    *begin = 0;
    *end = s.rows;
    return;
  }
  const int64_t base = static_cast<int64_t>(key >> 1) * s.L;
  *begin = base + ((key & 1) ? s.n_video : 0);
  *end = base + ((key & 1) ? s.L : s.n_video);
}

}  // namespace sol
