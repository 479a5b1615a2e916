// fp32 instantiations of the multi-axis rotary kernels, and the join of the
// CTAs' dgamma partials.
#include "rope_axes.cuh"

namespace sol {

cudaError_t launch_rope_axes_f32(RopeArgs &a, RopeMode mode, bool half, cudaStream_t stream,
                                 int *ctas) {
  return half ? dispatch_mode<float, true>(a, mode, stream, ctas)
              : dispatch_mode<float, false>(a, mode, stream, ctas);
}

namespace {

// One CTA per 32 channels of q (blockIdx.y = 0) or k (1); 32 warps take the
// partial rows in turn, a lane per channel, and are joined in a fixed order.
__global__ void __launch_bounds__(1024) rope_dgamma_kernel(const float *partial, int ctas,
                                                           int head_dim, float *dq, float *dk) {
  __shared__ double red[32][32];
  const int lane = threadIdx.x & 31, group = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float *out = blockIdx.y == 0 ? dq : dk;
  double s = 0.0;
  if (c < head_dim && out) {
    const float *p = partial + static_cast<int64_t>(blockIdx.y) * head_dim + c;
#pragma unroll 4
    for (int w = group; w < ctas; w += 32) s += p[static_cast<int64_t>(w) * 2 * head_dim];
  }
  red[group][lane] = s;
  __syncthreads();
  if (group == 0 && c < head_dim && out) {
    s = 0.0;
#pragma unroll
    for (int g = 0; g < 32; ++g) s += red[g][lane];
    out[c] = static_cast<float>(s);
  }
}

}  // namespace

cudaError_t launch_rope_dgamma(const float *partial, int ctas, int head_dim, float *dgamma_q,
                               float *dgamma_k, cudaStream_t stream) {
  if (!dgamma_q && !dgamma_k) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((head_dim + 31) / 32), 2);
  rope_dgamma_kernel<<<grid, 1024, 0, stream>>>(partial, ctas, head_dim, dgamma_q, dgamma_k);
  return cudaGetLastError();
}

}  // namespace sol
