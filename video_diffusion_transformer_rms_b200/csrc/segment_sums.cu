// Joins the row sums that the CTAs of a backward kernel left in their
// workspace slots into the gradients of the vectors:
//   dscale[key] = gamma * S1[key] + beta * S0[key],   dshift[key] = S0[key],
//   dgamma = sum_key (1 + scale[key]) * S1[key],
//   dbeta  = sum_key (1 + scale[key]) * S0[key].
//
// A CTA owns 32 channels of one output (blockIdx.y: a key, or one past the
// last key for dgamma and dbeta); its 32 warps take the slots in turn, a lane
// per channel, and are joined through shared memory.  Sums are fp64 and their
// order is fixed by the sizes, so results repeat bit for bit.
//
// Bound by latency: at most 592 + 2B slots of 8*D bytes, read once from L2.
// 32 warps per CTA leave each lane about 10 loads at one full wave of slots.
#include "segment_sums.cuh"
#include "sol_device.cuh"

namespace sol {
namespace {

constexpr int kCols = 32, kGroups = 32;

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

template <typename T>
__global__ void __launch_bounds__(kCols *kGroups) segment_sums_kernel(const SumArgs a, int y0) {
  __shared__ double red[2][kGroups][kCols];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int c = blockIdx.x * kCols + lane;
  const bool ok = c < a.D;
  const Segments &s = a.seg;
  const int64_t slot_stride = static_cast<int64_t>(a.sums) * a.D;
  const int key = y0 + static_cast<int>(blockIdx.y);
  const bool vectors = key == s.keys;  // dgamma and dbeta

  double s1 = 0.0, s0 = 0.0;
  if (ok && s.rows > 0) {
    if (!vectors) {
      int64_t r0, r1;
      key_rows(s, key, &r0, &r1);
      if (r0 < r1) {
        const int last = share_of(s, r1 - 1);
#pragma unroll 4
        for (int w = share_of(s, r0) + group; w <= last; w += kGroups) {
          const float *p = a.partial + (w + static_cast<int64_t>(key)) * slot_stride + c;
          s1 += p[0];
          if (a.sums == 2) s0 += p[a.D];
        }
      }
    } else if (s.keys == 1) {
#pragma unroll 4
      for (int w = group; w < s.ctas; w += kGroups) {
        const float *p = a.partial + w * slot_stride + c;
        s1 += p[0];
        if (a.sums == 2) s0 += p[a.D];
      }
    } else {
      for (int w = group; w < s.ctas; w += kGroups) {
        const int k1 = key_of(s, share_begin(s, w + 1) - 1);
        for (int k = key_of(s, share_begin(s, w)); k <= k1; ++k) {
          int64_t r0, r1;
          key_rows(s, k, &r0, &r1);
          if (r0 == r1) continue;
          const double fac = 1.0 + widen<T>(a.scale, static_cast<int64_t>(k) * a.D + c);
          const float *p = a.partial + (w + static_cast<int64_t>(k)) * slot_stride + c;
          s1 += fac * p[0];
          if (a.sums == 2) s0 += fac * p[a.D];
        }
      }
    }
  }
  red[0][group][lane] = s1;
  red[1][group][lane] = s0;
  __syncthreads();
  if (group == 0 && ok) {
    s1 = 0.0;
    s0 = 0.0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      s1 += red[0][g][lane];
      s0 += red[1][g][lane];
    }
    s1 *= a.mult;
    s0 *= a.mult;
    if (vectors) {
      if (a.dgamma) a.dgamma[c] = static_cast<float>(s1);
      if (a.dbeta) a.dbeta[c] = static_cast<float>(s0);
    } else {
      const int64_t o = static_cast<int64_t>(key) * a.D + c;
      if (a.dshift) a.dshift[o] = static_cast<float>(s0);
      if (a.dscale) {
        double v = s1;
        if (a.gamma) v *= widen<T>(a.gamma, c);
        if (a.beta) v += s0 * widen<T>(a.beta, c);
        a.dscale[o] = static_cast<float>(v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_segment_sums(const SumArgs &a, int dtype, cudaStream_t stream) {
  const bool keyed = a.dscale || a.dshift, vectors = a.dgamma || a.dbeta;
  const int ny = (keyed ? a.seg.keys : 0) + (vectors ? 1 : 0);
  if (ny == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((a.D + kCols - 1) / kCols), static_cast<unsigned>(ny));
  const int y0 = keyed ? 0 : a.seg.keys;
  if (dtype == 0)
    segment_sums_kernel<float><<<grid, kCols * kGroups, 0, stream>>>(a, y0);
  else
    segment_sums_kernel<__nv_bfloat16><<<grid, kCols * kGroups, 0, stream>>>(a, y0);
  return cudaGetLastError();
}

}  // namespace sol
