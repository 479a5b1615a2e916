// Host-side interface between the C ABI of the training operators
// (sol_abi_train.cu) and their launchers.  Internal to libsol: arguments
// arrive here already validated.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sol.h"
#include "sol_launch.h"

namespace sol {

// ---- layer norm, forward ---------------------------------------------------

struct LnArgs {
  const void *x;
  void *y;
  float *mean;        // [rows], with rstd, or null
  float *rstd;
  const void *gamma;  // may be null
  const void *beta;   // may be null
  const void *scale;  // with shift, or null: then L = n_video = rows (one key)
  const void *shift;
  int64_t rows;       // B * L
  int L;
  int n_video;
  int nvec;           // 16-byte vectors per row
  int D;
  float eps;
};
cudaError_t launch_layer_norm(const LnArgs &a, int dtype, cudaStream_t stream);

// ---- sums over the rows of each (sample, modality) ---------------------------

// Rows [0, rows) in CTAs' contiguous shares, the first `longer` of them `share`
// + 1 rows, the others `share`.  Key of a row = 2 * sample + modality,
// non-decreasing along the rows.  A CTA writes the sums over its rows of key k
// to slot `cta + k` of the workspace: (cta, key) pairs walk a staircase, so no
// two share a slot and ctas + keys slots are enough.
struct Segments {
  int64_t rows;  // < 2^31
  int L;         // rows per sample (rows, if the sums have one key)
  int n_video;   // first rows of a sample: key 2b; the others: key 2b + 1
  int keys;      // 2 * samples, or 1
  int ctas;      // shares the rows are cut into, at most `rows`
  int share;
  int longer;
};
inline void cut_shares(Segments *s, int64_t ctas) {
  s->ctas = static_cast<int>(ctas);
  s->share = static_cast<int>(s->rows / ctas);
  s->longer = static_cast<int>(s->rows % ctas);
}
// Bound on `ctas`: four CTAs on each of 148 SMs.
constexpr int kMaxSumCtas = 592;
// Slots of the workspace: shares and keys.
inline int64_t sum_slots(int64_t rows, int64_t keys) {
  return (rows < kMaxSumCtas ? rows : kMaxSumCtas) + keys;
}

struct SumArgs {
  Segments seg;
  const float *partial;  // [slot][sums][D]
  int sums;              // 1: S1 only; 2: S1, then S0
  int D;
  const void *scale;     // vectors of the I/O type, or null
  const void *gamma;
  const void *beta;
  float *dscale;         // [keys][D]: gamma * S1 + beta * S0, or null
  float *dshift;         // [keys][D]: S0, or null
  float *dgamma;         // [D]: sum over keys of (1 + scale) * S1, or null
  float *dbeta;          // [D]: sum over keys of (1 + scale) * S0, or null
  float mult;            // applied to S1
};
cudaError_t launch_segment_sums(const SumArgs &a, int dtype, cudaStream_t stream);

// ---- norm, backward ----------------------------------------------------------

struct NormBwdArgs {
  const void *dy;
  const void *x;
  const float *mean;   // layer norm only
  const float *rstd;
  const void *gamma;   // may be null
  const void *scale;   // may be null: one key
  const void *dres;    // may be null: added to dx
  void *dx;
  float *partial;      // workspace, or null: no vector gradients wanted
  Segments seg;        // shares cut by the launcher
  int nvec;
  int D;
  float eps;           // RMS only
  bool rms;
};
// Cuts the shares of a.seg and enqueues the kernel.
cudaError_t launch_norm_backward(NormBwdArgs &a, int dtype, cudaStream_t stream);

// ---- dropout in front of the gated residual ----------------------------------

struct DropArgs {
  const void *h;        // forward: may be null
  const void *branch;   // forward: the dropped input; backward: its value
  const void *gate;     // may be null in the forward kernel
  const void *dout;     // backward only
  void *out;            // out, or dbranch
  const uint64_t *rng;  // device: seed, offset
  uint64_t site;
  uint32_t drop_max;    // a word <= this is dropped
  bool drop;            // false: nothing is dropped, rng is not read
  float keep_scale;     // 1 / (1 - p), 0 for p = 1
  float *partial;       // backward: workspace
  Segments seg;         // backward: shares cut by the launcher
  int nvec;
  int D;
};
cudaError_t launch_dropout_residual(const DropArgs &a, int dtype, cudaStream_t stream);
cudaError_t launch_dropout_backward(DropArgs &a, int dtype, cudaStream_t stream);

// ---- rotary positions with several axes --------------------------------------

struct HeadsArg {
  void *data;          // null: absent
  int64_t sb, sr, sh;  // strides in bytes
};

struct RopeArgs {
  HeadsArg x[2];       // q, k: forward input; backward: forward input (norm only)
  HeadsArg g[2];       // backward: gradients of the outputs
  HeadsArg out[2];     // forward: outputs; backward: gradients of the inputs
  int heads[2];
  const void *gamma[2];
  const void *pos;
  int64_t pos_stride_axis, pos_stride_b;  // elements
  int pos_type;        // sol_pos_type
  int L;
  int64_t rows;
  int head_dim, rot_dim;
  float eps;
  float inv_hd;
  float *partial;      // backward with norm: [cta][2][head_dim], or null
  uint8_t axis[128];   // of each rotary pair
  double freq[128];    // radians per position; 0 beyond rot_dim / 2
};
enum RopeMode { kRotate = 0, kNormRotate = 1, kRotateBack = 2, kNormRotateBack = 3 };
// `ctas` receives the grid (the partial slots written).
cudaError_t launch_rope_axes_bf16(RopeArgs &a, RopeMode mode, bool half, cudaStream_t stream,
                                  int *ctas);
cudaError_t launch_rope_axes_f32(RopeArgs &a, RopeMode mode, bool half, cudaStream_t stream,
                                 int *ctas);
// dgamma_q and dgamma_k (either may be null) from `ctas` partial slots.
cudaError_t launch_rope_dgamma(const float *partial, int ctas, int head_dim, float *dgamma_q,
                               float *dgamma_k, cudaStream_t stream);
constexpr int kMaxRopeCtas = 148 * 8;
constexpr int64_t kMaxRopeHeads = 1024;

}  // namespace sol
