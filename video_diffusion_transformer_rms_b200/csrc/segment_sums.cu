// Joins the row sums that the CTAs of a backward kernel left in their
// workspace slots into the gradients of the vectors:
//   dscale[key] = gamma * S1[key] + beta * S0[key],   dshift[key] = S0[key],
//   dgamma = sum_key (1 + scale[key]) * S1[key],
//   dbeta  = sum_key (1 + scale[key]) * S0[key].
//
// A CTA owns 32 channels, a lane each, and reads their slots once.  With few
// keys its warps share the slots of every key and are joined through shared
// memory; with many, where a key has few slots, a warp takes a whole key, and
// the keys are spread over blockIdx.x; the last blockIdx.x then goes over all of
// them again for dgamma and dbeta, if these are wanted.
// Sums are fp64 and their order is fixed by the sizes, so results repeat bit for
// bit.
//
// Bound by latency: at most 592 + 2B slots of 8*D bytes, read from L2, 16 loads
// in flight per thread.  16 warps per CTA, so that two fit an SM: with 32 the 160
// CTAs of D = 5120 took two rounds of the 148 SMs.
#include "segment_sums.cuh"
#include "sol_device.cuh"

namespace sol {
namespace {

constexpr int kCols = 32, kGroups = 16;

template <typename T>
__device__ __forceinline__ float widen(const void *p, int64_t i);
template <>
__device__ __forceinline__ float widen<float>(const void *p, int64_t i) {
  return static_cast<const float *>(p)[i];
}
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(const void *p, int64_t i) {
  return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}

// Keys whose sums fit the shared memory of the first form.
constexpr int kSharedKeys = 4;

template <typename T>
__global__ void __launch_bounds__(kCols *kGroups, 2) segment_sums_kernel(const SumArgs a) {
  __shared__ double red[kSharedKeys][2][kGroups][kCols];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int c = blockIdx.y * kCols + lane;
  const bool ok = c < a.D;
  const Segments &s = a.seg;
  const int64_t slot_stride = static_cast<int64_t>(a.sums) * a.D;
  const float *base = a.partial + (ok ? c : 0);

  // Sums over slots first, first + step, ... of key k, in guarded batches: a
  // remainder loop would wait for its loads one by one.
  auto add_slots = [&](int k, int first, int step, double &s1, double &s0) {
    constexpr int BATCH = 8;
    double t1 = 0.0, t0 = 0.0;
    int64_t r0, r1;
    key_rows(s, k, &r0, &r1);
    if (r0 < r1) {
      const int w0 = share_of(s, r0) + first;
      const float *p = base + (w0 + static_cast<int64_t>(k)) * slot_stride;
      const int64_t jump = step * slot_stride;
      for (int left = share_of(s, r1 - 1) - w0; left >= 0; left -= BATCH * step) {
        float v1[BATCH], v0[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          v1[i] = v0[i] = 0.f;
          if (i * step <= left) {
            v1[i] = p[i * jump];
            if (a.sums == 2) v0[i] = p[i * jump + a.D];
          }
        }
        p += BATCH * jump;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          t1 += v1[i];
          t0 += v0[i];
        }
      }
    }
    s1 = t1;
    s0 = t0;
  };
  double g1 = 0.0, g0 = 0.0;  // this warp's part of dgamma and dbeta
  // the sums of key k are complete
  auto finish_key = [&](int k, double s1, double s0) {
    s1 *= a.mult;
    const int64_t o = static_cast<int64_t>(k) * a.D + c;
    const double fac = a.scale ? 1.0 + widen<T>(a.scale, o) : 1.0;
    g1 += fac * s1;
    g0 += fac * s0;
    if (a.dshift) a.dshift[o] = static_cast<float>(s0);
    if (a.dscale) {
      if (a.gamma) s1 *= widen<T>(a.gamma, c);
      if (a.beta) s1 += s0 * widen<T>(a.beta, c);
      a.dscale[o] = static_cast<float>(s1);
    }
  };

  if (s.keys <= kSharedKeys) {
    for (int k = 0; k < s.keys; ++k)
      add_slots(k, group, kGroups, red[k][0][group][lane], red[k][1][group][lane]);
    __syncthreads();
    if (group < s.keys && ok) {
      double s1 = 0.0, s0 = 0.0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        s1 += red[group][0][g][lane];
        s0 += red[group][1][g][lane];
      }
      finish_key(group, s1, s0);
    }
    __syncthreads();
  } else if (static_cast<int64_t>(blockIdx.x) * kGroups < s.keys) {
    const int k = blockIdx.x * kGroups + group;
    if (k < s.keys) {
      double s1, s0;
      add_slots(k, 0, 1, s1, s0);
      if (ok) finish_key(k, s1, s0);
    }
    return;
  } else {
    for (int k = group; k < s.keys; k += kGroups) {
      double s1, s0;
      add_slots(k, 0, 1, s1, s0);
      const double fac =
          a.scale && ok ? 1.0 + widen<T>(a.scale, static_cast<int64_t>(k) * a.D + c) : 1.0;
      g1 += fac * s1 * a.mult;
      g0 += fac * s0;
    }
  }
  if (a.dgamma || a.dbeta) {
    red[0][0][group][lane] = g1;
    red[0][1][group][lane] = g0;
    __syncthreads();
    if (group == 0 && ok) {
      g1 = g0 = 0.0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        g1 += red[0][0][g][lane];
        g0 += red[0][1][g][lane];
      }
      if (a.dgamma) a.dgamma[c] = static_cast<float>(g1);
      if (a.dbeta) a.dbeta[c] = static_cast<float>(g0);
    }
  }
}

}  // namespace

cudaError_t launch_segment_sums(const SumArgs &a, int dtype, cudaStream_t stream) {
  if (!a.dscale && !a.dshift && !a.dgamma && !a.dbeta) return cudaSuccess;
  const bool vectors = a.dgamma || a.dbeta;
  const unsigned blocks =
      a.seg.keys <= kSharedKeys
          ? 1
          : static_cast<unsigned>((a.seg.keys + kGroups - 1) / kGroups) + (vectors ? 1 : 0);
  const dim3 grid(blocks, static_cast<unsigned>((a.D + kCols - 1) / kCols));
  if (dtype == 0)
    segment_sums_kernel<float><<<grid, kCols * kGroups, 0, stream>>>(a);
  else
    segment_sums_kernel<__nv_bfloat16><<<grid, kCols * kGroups, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sol
