// Contiguous shares of token rows and the (sample, modality) keys they meet,
// shared by the kernels that sum over rows and by the kernel that joins the
// sums (sol_train.h, Segments).  Row numbers are below 2^31.
#pragma once

#include <stdint.h>

#include "sol_train.h"

namespace sol {

// First row of CTA c's share; c = ctas gives the row count.
__device__ __forceinline__ int64_t share_begin(const Segments &s, int c) {
  return static_cast<int64_t>(c) * s.share + (c < s.longer ? c : s.longer);
}
// The CTA whose share holds `row`.
__device__ __forceinline__ int share_of(const Segments &s, int64_t row) {
  const unsigned r = static_cast<unsigned>(row), n = static_cast<unsigned>(s.share);
  const unsigned head = static_cast<unsigned>(s.longer) * (n + 1);  // <= rows
  return static_cast<int>(r < head ? r / (n + 1) : s.longer + (r - head) / n);
}
__device__ __forceinline__ int key_of(const Segments &s, int64_t row) {
  if (s.keys == 1) return 0;
  const unsigned b = static_cast<unsigned>(row) / static_cast<unsigned>(s.L);
  const unsigned r = static_cast<unsigned>(row) - b * static_cast<unsigned>(s.L);
  return static_cast<int>(2 * b + (r >= static_cast<unsigned>(s.n_video) ? 1 : 0));
}
// Rows [begin, end) of a key; empty if the modality has no rows.
__device__ __forceinline__ void key_rows(const Segments &s, int key, int64_t *begin,
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
